"""The Softmax branch's operators as they run together: each step norms and
rotates the new tokens' queries and keys, appends keys and values to the paged
cache and attends over it.  Against the float64 oracle of the same steps.

Tolerance, before the first run: the oracle reads the cache and the queries as
the GPU stored them, so the attention's own bound holds (see
test_gpu_paged_attention), and the stored values are held to the norm's (see
test_gpu_qk_norm_rope)."""

import numpy as np
import pytest

from oracle import softmax_ref as ref
from test_gpu_paged_attention import _check
from test_gpu_qk_norm_rope import _near, _np

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _api():
    from frame_wise_delta_vda_b200 import api
    return api


class Branch:
    """A paged cache for B sequences with pages handed out as they are needed."""

    def __init__(self, B, Hq, Hk, d, page, dtype, pages, axes=1, seed=0):
        g = self.g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hk, self.d, self.page, self.dtype, self.axes = Hq, Hk, d, page, dtype, axes
        sections = None if axes == 1 else [d // 2 - 2 * (d // 6), d // 6, d // 6]
        self.freq, self.axis = _api().rope_frequencies(d, sections=sections)
        self.wq, self.wk = (1 + 0.1 * torch.randn(d, generator=g)).cuda(), (1 + 0.1 * torch.randn(d, generator=g)).cuda()
        self.kc = torch.full((pages, Hk, page, d), float("nan"), dtype=dtype, device="cuda")
        self.vc = self.kc.clone()
        self.free = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((B, pages), -1, dtype=torch.int32)
        self.len = [0] * B
        self.kept = [[] for _ in range(B)]      # the projections and positions of all tokens

    def step(self, new, positions=None, check=True, **mask):
        """new[b] tokens of each sequence; positions default to the places in the sequence."""
        api, B = _api(), len(new)
        N, C = sum(new), (self.Hq + 2 * self.Hk) * self.d
        qkv = torch.randn(N, C, generator=self.g).to(self.dtype).cuda()
        slots, pos = [], []
        for b, n in enumerate(new):
            for i in range(self.len[b], self.len[b] + n):
                if i % self.page == 0:
                    self.table[b, i // self.page] = self.free.pop()
                slots.append(int(self.table[b, i // self.page]) * self.page + i % self.page)
                pos.append([i] * self.axes if positions is None else positions(b, i))
            self.len[b] += n
        q = qkv[:, :self.Hq * self.d].view(N, self.Hq, self.d)
        k = qkv[:, self.Hq * self.d:(self.Hq + self.Hk) * self.d].view(N, self.Hk, self.d)
        v = qkv[:, (self.Hq + self.Hk) * self.d:].view(N, self.Hk, self.d)
        pos = torch.tensor(pos, dtype=torch.int32).view(N, self.axes).cuda()
        slots = torch.tensor(slots, dtype=torch.int64).cuda()
        start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
        kv_len = torch.tensor(self.len, dtype=torch.int32).cuda()
        qo, _ = api.vda_qk_norm_rope(q, k, self.wq, self.wk, pos, self.freq, self.axis, v=v, k_cache=self.kc,
                                     v_cache=self.vc, slots=slots)
        out, lse = api.vda_paged_attention(qo, self.kc, self.vc, self.table.cuda(), kv_len, start, return_lse=True, **mask)
        if check:
            phi = ref.angles(pos.cpu().numpy(), self.freq.cpu().numpy(), self.axis.cpu().numpy())
            _near(qo, q, self.wq, phi, False, self.dtype)
            stored = self.kc[slots // self.page, :, slots % self.page]
            _near(stored, k, self.wk, phi, False, self.dtype)
            assert torch.equal(self.vc[slots // self.page, :, slots % self.page], v)
            c = dict(q=qo, k_cache=self.kc, v_cache=self.vc, block_table=self.table, kv_len=kv_len, q_start=start)
            _check(c, out, lse, mask.get("block", 1), mask.get("window_blocks", -1), mask.get("anchors", 0))
        return qkv, out


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 32)],
                         ids=["bf16-128", "bf16-64", "f32-32"])
def test_prompts_then_single_tokens(dtype, d):
    """Prompts of different lengths, one in two chunks, then steps of a ragged batch."""
    b = Branch(3, 8, 2, d, 16, dtype, pages=60)
    b.step([200, 17, 1])
    b.step([133, 0, 5])
    for _ in range(4):
        b.step([1, 1, 1])
    b.step([0, 3, 1])


def test_video_chunks_with_anchor_and_window():
    """Livestream form: an anchor frame, then chunks of two frames that see
    themselves, one chunk before and the anchor; frame/row/column positions."""
    U = 45                                         # a latent frame of 5 x 9 tokens
    at = lambda b, i: [i // U, i % U // 9, i % 9]  # noqa: E731
    b = Branch(1, 4, 4, 128, 16, torch.bfloat16, pages=60, axes=3)
    mask = dict(block=2 * U, window_blocks=1, anchors=U)
    b.step([U], positions=at, **mask)
    for _ in range(5):
        b.step([2 * U], positions=at, **mask)


def test_a_prompt_in_chunks_equals_the_prompt_at_once():
    """The same tokens through one call and through three: the same cache bits,
    and outputs that differ by the order of the sums alone."""
    outs = []
    for parts in ([300], [100, 77, 123]):
        b = Branch(1, 4, 2, 64, 16, torch.bfloat16, pages=30, seed=5)
        gen = torch.Generator().manual_seed(9)
        whole = torch.randn(300, 8 * 64, generator=gen)
        rows, at = [], 0
        for n in parts:
            b.g = _Replay(whole[at:at + n])
            rows.append(b.step([n], check=False)[1])
            at += n
        pages = b.table[0, :19].long()
        outs.append((torch.cat(rows), b.kc[pages].cpu(), b.vc[pages].cpu()))
    assert torch.equal(outs[0][1].view(torch.int16), outs[1][1].view(torch.int16))
    assert torch.equal(outs[0][2].view(torch.int16), outs[1][2].view(torch.int16))
    a, c = _np(outs[0][0]), _np(outs[1][0])
    # both within 2^-8 (the result) + 2^-8 (the weights) of a mean of |v| <= 5
    assert np.abs(a - c).max() <= 2 * (2.0 ** -8 + 2.0 ** -8) * 5


class _Replay:
    def __init__(self, rows):
        self.rows = rows


_randn = torch.randn


@pytest.fixture(autouse=True)
def _replay(monkeypatch):
    """`torch.randn(..., generator=_Replay(rows))` gives those rows."""
    def randn(*shape, generator=None, **kw):
        return generator.rows.clone() if isinstance(generator, _Replay) else _randn(*shape, generator=generator, **kw)
    monkeypatch.setattr(torch, "randn", randn)


def test_two_streams_at_once_and_two_graphs():
    """Calls that overlap have workspaces of their own: two streams, and two
    captured graphs replayed at the same time."""
    api = _api()
    from test_gpu_paged_attention import _case
    cases = [_case([40, 1], [3000, 5000], 8, 2, 128, 64, torch.bfloat16, seed=s) for s in (1, 2)]
    want = [api.vda_paged_attention(**c, return_lse=True) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for _ in range(20):
        for i, (s, c) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                got[i] = api.vda_paged_attention(**c, return_lse=True)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))
    graphs = [torch.cuda.CUDAGraph() for _ in cases]
    for i, c in enumerate(cases):
        with torch.cuda.graph(graphs[i]):
            got[i] = api.vda_paged_attention(**c, return_lse=True)
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))
    assert api.vda_device_status() == 0


def test_linear_and_softmax_branch_on_one_stream():
    """The block's two halves one after the other: the linear branch's result is what it is alone."""
    from frame_wise_delta_vda_b200 import inputs as gen
    from _helpers import to_torch
    api = _api()
    wl = gen.custom("block", H=2, T=10, U=40, d=128, chunk=5, window_chunks=0, dtype="bf16", seed=4)
    t = {k: to_torch(v, "cuda") for k, v in gen.make_inputs(wl).items()}
    run = lambda: api.vda_forward(t["q"], t["k"], t["v"], t["beta"], t["gate"], t["rms_weight"], chunk=5, window_chunks=0)  # noqa: E731
    alone = run()
    b = Branch(1, 2, 2, 128, 16, torch.bfloat16, pages=40)
    b.step([400])
    for _ in range(3):
        out = run()
        b.step([1])
        assert torch.equal(out, alone)
    assert api.vda_device_status() == 0
