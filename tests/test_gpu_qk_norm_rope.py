"""vda_qk_norm_rope and its gradient on the GPU against the float64 oracle.

Tolerances, from the arithmetic, before the first run.  u is half a step of
the output type (bf16 2^-8, fp32 2^-24); everything else is fp32: the sum of
squares, its root and two products are off by at most 2^-20 together (8
channels a lane and four shuffle steps at 2^-24 each, rsqrt 2 ulp); cos and
sin by 2^-22 (the angle, at most half a turn, is rounded to 24 bits once:
pi 2^-24, plus 2^-23 of the functions).  A rotated value is a sum of two such
products, so |error| <= u |y| + 2^-19 (|z_i| + |z_j|).  The gradient adds a
mean of d products and a difference: 2^-18 of the magnitudes that go in.  A
weight gradient adds at most 64 terms a lane in sequence here, and 2^-24 each
for the joining of lanes, warps and blocks: 2^-17 of the summed magnitudes."""

import numpy as np
import pytest

from oracle import softmax_ref as ref

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _api():
    from frame_wise_delta_vda_b200 import api
    return api


def _np(t):
    return t.detach().double().cpu().numpy()


def _case(N, Hq, Hk, d, dtype, rot, axes=1, start=0, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float32)  # noqa: E731
    api = _api()
    half = rot // 2
    sections = [half] if axes == 1 else [half - 2 * (half // 3), half // 3, half // 3]
    freq, axis = api.rope_frequencies(rot, 10000.0, sections, device=device)
    pos = (start + torch.randint(0, 1000, (N, axes), generator=g)).to(torch.int32)
    qkv = r(N, (Hq + 2 * Hk) * d).to(dtype).to(device)
    c = dict(q=qkv[:, :Hq * d].view(N, Hq, d), k=qkv[:, Hq * d:(Hq + Hk) * d].view(N, Hk, d),
             q_weight=(1 + 0.2 * r(d)).to(device), k_weight=(1 + 0.2 * r(d)).to(device), positions=pos.to(device),
             frequencies=freq, axis=axis)
    return c, qkv[:, (Hq + Hk) * d:].view(N, Hk, d), g


def _phi(c):
    return ref.angles(c["positions"].cpu().numpy(), c["frequencies"].cpu().numpy(), c["axis"].cpu().numpy())


def _near(got, x, w, phi, interleaved, dtype, eps=1e-6):
    x, w = _np(x), _np(w) if w is not None else 1.0
    want = ref.norm_rope(x, w, phi, interleaved, eps)
    z = ref.norm(x, eps)[0] * w
    tol = U[dtype] * np.abs(want) + 2.0 ** -19 * ref.paired_magnitude(z, 2 * phi.shape[1], interleaved) + 1e-30
    bad = np.abs(_np(got) - want) / tol
    assert bad.max() <= 1.0, bad.max()


CASES = [   # N, Hq, Hk, d, rot, axes, start, interleaved
    (1, 1, 1, 16, 16, 1, 0, False),
    (1, 32, 8, 128, 128, 1, 100_000, False),
    (37, 3, 1, 64, 64, 3, 0, False),
    (37, 5, 5, 128, 64, 1, 2_000_000_000, True),
    (5, 2, 7, 32, 16, 1, 77, True),
    (130, 9, 3, 64, 32, 3, -500, False),
    (3, 2, 2, 128, 0, 1, 0, False),
    (4000, 12, 4, 128, 128, 3, 0, False),
]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,Hq,Hk,d,rot,axes,start,inter", CASES)
def test_forward(N, Hq, Hk, d, rot, axes, start, inter, dtype):
    c, _, _ = _case(N, Hq, Hk, d, dtype, rot, axes, start)
    qo, ko = _api().vda_qk_norm_rope(**c, interleaved=inter)
    phi = _phi(c)
    _near(qo, c["q"], c["q_weight"], phi, inter, dtype)
    _near(ko, c["k"], c["k_weight"], phi, inter, dtype)


@gpu
def test_far_positions_keep_their_angle():
    """The largest positions, where radians in 32 bits have no digit left."""
    c, _, _ = _case(64, 2, 1, 64, torch.float32, 64)
    c["positions"] = (2 ** 31 - 1 - torch.arange(64, dtype=torch.int32, device="cuda")).view(64, 1)
    qo, _ = _api().vda_qk_norm_rope(**c)
    # the angle itself, in extended integers: position * frequency in turns
    freq = c["frequencies"].cpu().numpy()
    turns = [int(round((f / (2 * np.pi)) * 2 ** 64)) for f in freq]
    pos = c["positions"].cpu().numpy()[:, 0]
    phi = np.array([[((int(p) * t) % 2 ** 64) / 2.0 ** 64 * 2 * np.pi for t in turns] for p in pos])
    z = ref.norm(_np(c["q"]), 1e-6)[0] * _np(c["q_weight"])
    tol = 2.0 ** -18 * ref.paired_magnitude(z, 64)   # 2^31 * 2^-55 turns more than the angles above
    assert (np.abs(_np(qo) - ref.rotate(z, phi)) <= tol).all()


@gpu
def test_no_weights_no_rotation_and_an_axis_that_does_not_exist():
    api = _api()
    c, _, _ = _case(9, 3, 2, 64, torch.float32, 64)
    qo, ko = api.vda_qk_norm_rope(c["q"], c["k"])
    none = np.zeros((9, 0))
    _near(qo, c["q"], None, none, False, torch.float32)
    _near(ko, c["k"], None, none, False, torch.float32)
    c["axis"][::2] = 1
    c["axis"][1] = -3
    qo, _ = api.vda_qk_norm_rope(**c)
    _near(qo, c["q"], c["q_weight"], _phi(c), False, torch.float32)


@gpu
def test_zero_rows_and_infinite_rows_stay_in_their_rows():
    api = _api()
    c, _, _ = _case(6, 4, 1, 128, torch.bfloat16, 128)
    clean, _ = api.vda_qk_norm_rope(**c)
    c["q"][2, 1] = 0
    c["q"][3, 2, 5] = float("inf")
    c["q"][4, 0, 7] = float("nan")
    qo, _ = api.vda_qk_norm_rope(**c)
    assert (qo[2, 1] == 0).all()
    touched = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    touched[2, 1] = touched[3, 2] = touched[4, 0] = True
    assert torch.equal(qo[~touched], clean[~touched])
    assert qo[4, 0].isnan().all()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_append_writes_only_the_slots(dtype):
    api = _api()
    N, Hq, Hk, d, page, P = 45, 6, 3, 64, 16, 5
    c, v, g = _case(N, Hq, Hk, d, dtype, 64, start=10)
    kc = torch.randn(P, Hk, page, d, generator=g).to(dtype).cuda()
    vc = torch.randn(P, Hk, page, d, generator=g).to(dtype).cuda()
    kw, vw = kc.clone(), vc.clone()
    slots = torch.randperm(P * page, generator=g)[:N]
    slots[7], slots[8], slots[9] = -1, P * page, 2 ** 60
    k_out = torch.empty(N, Hk, d, dtype=dtype, device="cuda")
    qo, ko = api.vda_qk_norm_rope(**c, v=v, k_cache=kc, v_cache=vc, slots=slots.cuda(), k_out=k_out)
    _near(qo, c["q"], c["q_weight"], _phi(c), False, dtype)
    _near(ko, c["k"], c["k_weight"], _phi(c), False, dtype)
    for t in range(N):
        s = int(slots[t])
        if 0 <= s < P * page:
            kw[s // page, :, s % page], vw[s // page, :, s % page] = ko[t], v[t]
    assert torch.equal(kc, kw) and torch.equal(vc, vw)
    kc2 = kc.clone().zero_()
    qo2, none = api.vda_qk_norm_rope(**c, v=v, k_cache=kc2, v_cache=vc, slots=slots.cuda())
    assert none is None and torch.equal(qo2, qo)


@gpu
def test_strides_of_inputs_and_outputs():
    api = _api()
    c, _, _ = _case(33, 4, 2, 128, torch.bfloat16, 128)
    want = api.vda_qk_norm_rope(**c)
    major = {n: c[n].transpose(0, 1).contiguous().transpose(0, 1) for n in "qk"}     # head-major
    assert all(torch.equal(x, y) for x, y in zip(want, api.vda_qk_norm_rope(**{**c, **major})))
    qo = torch.full((4, 33, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")       # into every other row
    out, _ = api.vda_qk_norm_rope(**c, q_out=qo[:, :, 0].transpose(0, 1))
    assert torch.equal(out, want[0]) and (qo[:, :, 1] == 7).all()
    one = c["k"][:1].expand(33, 2, 128)                                              # broadcast over tokens
    assert torch.equal(api.vda_qk_norm_rope(**{**c, "k": one})[1], api.vda_qk_norm_rope(**{**c, "k": one.contiguous()})[1])


def _grad_near(got, gotw, dy, x, w, phi, inter, dtype, eps=1e-6):
    dy, x = _np(dy), _np(x)
    wn = _np(w) if w is not None else np.ones(x.shape[-1])
    dx, dw = ref.norm_rope_backward(dy, x, wn, phi, inter, eps)
    u, inv = ref.norm(x, eps)
    m = ref.paired_magnitude(dy, 2 * phi.shape[1], inter)
    size = inv * (m * np.abs(wn) + np.abs(u) * (m * np.abs(wn * u)).mean(-1, keepdims=True))
    bad = np.abs(_np(got) - dx) / (U[dtype] * np.abs(dx) + 2.0 ** -18 * size + 1e-30)
    assert bad.max() <= 1.0, bad.max()
    if gotw is not None:
        bad = np.abs(_np(gotw) - dw) / (2.0 ** -17 * (m * np.abs(u)).sum((0, 1)) + 1e-30)
        assert bad.max() <= 1.0, bad.max()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,Hq,Hk,d,rot,axes,start,inter", CASES)
def test_backward(N, Hq, Hk, d, rot, axes, start, inter, dtype):
    c, _, g = _case(N, Hq, Hk, d, dtype, rot, axes, start)
    dq, dk = (torch.randn(N, h, d, generator=g).to(dtype).cuda() for h in (Hq, Hk))
    gq, gk, wq, wk = _api().vda_qk_norm_rope_backward(dq, dk, **c, interleaved=inter)
    phi = _phi(c)
    _grad_near(gq, wq, dq, c["q"], c["q_weight"], phi, inter, dtype)
    _grad_near(gk, wk, dk, c["k"], c["k_weight"], phi, inter, dtype)
    again = _api().vda_qk_norm_rope_backward(dq, dk, **c, interleaved=inter)
    assert all(torch.equal(x, y) for x, y in zip((gq, gk, wq, wk), again))


@gpu
def test_backward_broadcast_gradients_strided_results_and_no_weights():
    api = _api()
    c, _, g = _case(21, 4, 2, 64, torch.float32, 64)
    dq = torch.randn(21, 1, 64, generator=g).cuda().expand(21, 4, 64)
    dk = torch.randn(1, 1, 64, generator=g).cuda().expand(21, 2, 64)
    joint = torch.full((21, 8 * 64), 3.0, device="cuda")
    into = dict(dq=joint[:, :256].view(21, 4, 64), dk=joint[:, 256:384].view(21, 2, 64))
    gq, gk, wq, wk = api.vda_qk_norm_rope_backward(dq, dk, **c, **into)
    _grad_near(gq, wq, dq, c["q"], c["q_weight"], _phi(c), False, torch.float32)
    _grad_near(gk, wk, dk, c["k"], c["k_weight"], _phi(c), False, torch.float32)
    assert (joint[:, 384:] == 3).all()
    c["q_weight"] = c["k_weight"] = None
    gq, gk, wq, wk = api.vda_qk_norm_rope_backward(dq, dk, **c)
    assert wq is None and wk is None
    _grad_near(gq, None, dq, c["q"], None, _phi(c), False, torch.float32)


@gpu
def test_backward_against_differences_of_the_forward():
    api = _api()
    c, _, g = _case(4, 2, 1, 32, torch.float32, 32)
    dq, dk = torch.randn(4, 2, 32, generator=g).cuda(), torch.zeros(4, 1, 32, device="cuda")
    gq, _, wq, _ = api.vda_qk_norm_rope_backward(dq, dk, **c)
    loss = lambda c: float((dq.double() * api.vda_qk_norm_rope(**c)[0].double()).sum())  # noqa: E731
    h = 2.0 ** -7
    # central differences: h^2 / 6 of a third derivative of order 10, and 2^-19 of the summed magnitudes over 2 h
    tol = 10 * h * h + 2.0 ** -19 * float(dq.abs().sum()) * 4 / (2 * h)
    for idx in [(0, 0, 0), (1, 1, 17), (3, 0, 31)]:
        e = torch.zeros(4, 2, 32, device="cuda")
        e[idx] = h
        d = (loss({**c, "q": c["q"] + e}) - loss({**c, "q": c["q"] - e})) / (2 * h)
        assert abs(d - float(gq[idx])) <= tol
    e = torch.zeros(32, device="cuda")
    e[5] = h
    d = (loss({**c, "q_weight": c["q_weight"] + e}) - loss({**c, "q_weight": c["q_weight"] - e})) / (2 * h)
    assert abs(d - float(wq[5])) <= tol


@gpu
def test_empty_batch():
    api = _api()
    c, v, _ = _case(0, 4, 2, 64, torch.bfloat16, 64)
    qo, ko = api.vda_qk_norm_rope(**c)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)
    z = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    qo, ko = api.vda_qk_norm_rope(**c, v=v, k_cache=z, v_cache=z.clone(),
                                  slots=torch.empty(0, dtype=torch.int64, device="cuda"))
    assert ko is None and (z == 0).all()
    _, _, wq, wk = api.vda_qk_norm_rope_backward(qo, c["k"], **c)
    assert (wq == 0).all() and (wk == 0).all()


@gpu
def test_side_stream_and_graph_replay():
    api = _api()
    c, _, g = _case(50, 4, 2, 128, torch.bfloat16, 128)
    dq, dk = (torch.randn(50, h, 128, generator=g).to(torch.bfloat16).cuda() for h in (4, 2))
    fwd, bwd = api.vda_qk_norm_rope(**c), api.vda_qk_norm_rope_backward(dq, dk, **c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f2 = api.vda_qk_norm_rope(**c)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(fwd, f2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f3, b3 = api.vda_qk_norm_rope(**c), api.vda_qk_norm_rope_backward(dq, dk, **c)
    for _ in range(2):
        for t in (*f3, *b3):
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*fwd, *bwd), (*f3, *b3)))
