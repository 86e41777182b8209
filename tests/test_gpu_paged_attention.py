"""vda_paged_attention on the GPU against the float64 oracle.

Tolerances, from the arithmetic, before the first run.  u is half a step of
the output type.  Scores are fp32 sums of d exact products (or of d rounded
ones in fp32): off by at most (d + 2) 2^-24 sum |q k| scale, here s_err.
A weight's relative error is then at most 2 s_err + 2^-21 (two exponentials
of a difference and, over several parts, of the joining), an output's
2 s_err + 2^-21 + n 2^-24 of sum_j p_j |v_j|, n the number of keys, and the
tensor cores' P in bf16 adds 2^-8 of the same sum.  lse: s_err + 2^-20 (1 +
|lse|)."""

import numpy as np
import pytest

from oracle import softmax_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _api():
    from frame_wise_delta_vda_b200 import api
    return api


def _np(t):
    return t.detach().double().cpu().numpy()


def _case(new, length, Hq, Hk, d, page, dtype, seed=0, spare=3, peak=2.0, behind=0):
    """Caches whose unused places hold NaN, a shuffled table whose unused
    entries are out of range, and `behind` tokens after the last sequence."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-m // page) for m in length]
    P = sum(need) + spare
    N = sum(new) + behind
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q = (peak * r(N, Hq, d)).to(dtype)
    kc = torch.full((P, Hk, page, d), float("nan"), dtype=dtype)
    vc = kc.clone()
    order = torch.randperm(P, generator=g)
    table = torch.full((len(new), max(max(need), 1) + 1), 2 ** 30, dtype=torch.int32)
    at = 0
    for b, m in enumerate(length):
        for i in range(need[b]):
            p = int(order[at])
            at += 1
            table[b, i] = p
            n = min(page, m - i * page)
            kc[p, :, :n] = r(Hk, n, d).to(dtype)
            vc[p, :, :n] = r(Hk, n, d).to(dtype)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    dev = lambda t: t.cuda()  # noqa: E731
    return dict(q=dev(q), k_cache=dev(kc), v_cache=dev(vc), block_table=dev(table),
                kv_len=torch.tensor(length, dtype=torch.int32).cuda(), q_start=dev(start))


def _check(c, out, lse, block=1, window=-1, anchors=0, scale=None):
    q, kc, vc = _np(c["q"]), _np(c["k_cache"]), _np(c["v_cache"])
    table, length, start = (c[n].cpu().numpy() for n in ("block_table", "kv_len", "q_start"))
    N, Hq, d = q.shape
    P, Hk, page, _ = kc.shape
    G = Hq // Hk
    scale = d ** -0.5 if scale is None else scale
    tc = c["q"].dtype == torch.bfloat16 and d >= 64
    out, lse = _np(out), _np(lse)
    worst = 0.0
    for b in range(len(length)):
        t0, t1, L = int(start[b]), int(start[b + 1]), int(length[b])
        if t0 == t1:
            continue
        pages = table[b].astype(np.int64)[np.arange(L) // page]
        absent = np.flatnonzero((pages < 0) | (pages >= P))
        at, off = np.clip(pages, 0, P - 1), np.arange(L) % page
        see = ref.visible(np.arange(L - (t1 - t0), L), L, block, window, anchors, absent)[:, None]     # [n, 1, L]
        for h in range(Hk):
            K, V = np.nan_to_num(kc[at, h, off]), np.nan_to_num(vc[at, h, off])
            Q = q[t0:t1, h * G:(h + 1) * G]
            s = np.where(see, scale * (Q @ K.T), -np.inf)
            m = s.max(-1, keepdims=True, initial=-np.inf)
            none = np.isneginf(m)
            p = np.exp(s - np.where(none, 0.0, m))
            tot = p.sum(-1, keepdims=True)
            p = p / np.where(none, 1.0, tot)
            want = p @ V
            z = np.where(none, -np.inf, m + np.log(np.where(none, 1.0, tot)))[..., 0]
            s_err = ((d + 2) * 2.0 ** -24 * scale * np.where(see, np.abs(Q) @ np.abs(K).T, 0.0)).max(-1, initial=0.0)
            got, gz = out[t0:t1, h * G:(h + 1) * G], lse[t0:t1, h * G:(h + 1) * G]
            assert (got[none[..., 0]] == 0).all()
            np.testing.assert_array_equal(np.isneginf(gz), none[..., 0])
            n = see.sum(-1)
            rel = 2 * s_err + 2.0 ** -21 + n * 2.0 ** -24 + (2.0 ** -8 if tc else 0.0)
            tol = U[c["q"].dtype] * np.abs(want) * (1 + 2.0 ** -7) + rel[..., None] * (p @ np.abs(V)) + 1e-30
            bad = (np.abs(got - want) / tol).max(initial=0.0)
            assert np.isfinite(got).all() and bad <= 1.0, (b, h, bad)
            worst = max(worst, bad)
            ok = ~none[..., 0]
            bad = np.abs(gz - np.where(ok, z, 0.0))[ok] / (s_err + 2.0 ** -20 * (1 + np.abs(np.where(ok, z, 0.0))))[ok]
            assert bad.max(initial=0.0) <= 1.0, (b, h, bad.max())
    return worst


TYPES = [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64), (torch.float32, 128), (torch.bfloat16, 32),
         (torch.float32, 16)]
IDS = ["bf16-128", "bf16-64", "f32-64", "f32-128", "bf16-32", "f32-16"]


@pytest.mark.parametrize("dtype,d", TYPES, ids=IDS)
@pytest.mark.parametrize("new,length,Hq,Hk,page", [
    ([1], [1], 1, 1, 16),
    ([1], [1000], 8, 2, 16),
    ([1, 1, 1], [127, 128, 129], 4, 4, 16),
    ([1, 0, 3, 1], [40, 5, 3, 600], 10, 2, 32),
    ([5], [700], 24, 3, 64),
    ([100], [100], 2, 1, 16),
    ([33, 257, 64], [500, 257, 64], 6, 2, 128),
    ([300], [1300], 8, 8, 64),
    ([7, 1, 130], [70, 900, 130], 15, 5, 16),
], ids=str)
def test_causal_by_token(new, length, Hq, Hk, page, dtype, d):
    c = _case(new, length, Hq, Hk, d, page, dtype)
    out, lse = _api().vda_paged_attention(**c, return_lse=True)
    print("worst", _check(c, out, lse))


@pytest.mark.parametrize("dtype,d", TYPES[:3], ids=IDS[:3])
@pytest.mark.parametrize("block,window,anchors", [
    (0, -1, 0), (1, 0, 0), (1, 50, 0), (1, 127, 4), (1, 200, 150), (48, -1, 0), (48, 0, 0), (48, 2, 48), (100, 1, 7),
    (1 << 30, 0, 0), (7, 2 ** 31 - 1, 300), (1, 5, 1 << 30)])
def test_masks(block, window, anchors, dtype, d):
    c = _case([90, 1, 260], [90, 800, 700], 6, 3, d, 16, dtype, seed=block % 97)
    out, lse = _api().vda_paged_attention(**c, block=block, window_blocks=window, anchors=anchors, return_lse=True)
    _check(c, out, lse, block, window, anchors)


@pytest.mark.parametrize("dtype,d", TYPES[:3], ids=IDS[:3])
def test_rows_that_see_nothing(dtype, d):
    """More new tokens than keys, a sequence without keys, one whose every
    page is gone, and tokens of no sequence."""
    c = _case([30, 5, 40, 2], [20, 0, 60, 50], 4, 2, d, 16, dtype, behind=9)
    c["block_table"][2, :] = -1
    c["block_table"][3, 1] = 10 ** 6
    out = torch.full_like(c["q"], 7.0)
    lse = torch.full(out.shape[:2], 7.0, device="cuda")
    got, z = _api().vda_paged_attention(**c, out=out, lse=lse, return_lse=True)
    assert got is out and z is lse
    _check(c, out, lse)
    assert (out[-9:] == 7).all() and (lse[-9:] == 7).all()
    assert (out[:10] == 0).all() and (out[30:75] == 0).all()


@pytest.mark.parametrize("dtype,d", TYPES[:3], ids=IDS[:3])
def test_stale_and_infinite_places_do_not_matter(dtype, d):
    """NaN already fills what no sequence uses; here also keys that the window has left."""
    c = _case([40], [500], 4, 2, d, 16, dtype)
    table = c["block_table"][0].tolist()
    want = _api().vda_paged_attention(**c, window_blocks=63, anchors=3)
    # windows of 64 of positions 460.. begin at key 397 or later: 3 .. 396 are unseen
    for i in range(1, 24):
        c["k_cache"][table[i]] = float("nan")
        c["v_cache"][table[i]] = float("inf")
    c["v_cache"][table[0], :, 3:] = float("nan")
    c["v_cache"][table[24], :, :397 - 384] = float("-inf")
    got = _api().vda_paged_attention(**c, window_blocks=63, anchors=3)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,d", TYPES[:3], ids=IDS[:3])
def test_a_growing_maximum_and_lowest_values(dtype, d):
    """Scores that rise along the keys by hundreds, and some of the type's lowest value."""
    c = _case([20, 200], [900, 700], 4, 1, d, 64, dtype, peak=1.0)
    c["k_cache"].nan_to_num_(0.0)
    c["v_cache"].nan_to_num_(0.0)
    c["q"].abs_()
    for b, L in enumerate((900, 700)):
        for j in range(0, L, 40):
            p = int(c["block_table"][b, j // 64])
            c["k_cache"][p, 0, j % 64] = 0.02 * j / d ** 0.5
            c["k_cache"][p, 0, (j + 1) % 64] = torch.finfo(dtype).min / 2 ** 20
    out, lse = _api().vda_paged_attention(**c, return_lse=True)
    _check(c, out, lse)


@pytest.mark.parametrize("dtype,d", TYPES[:3], ids=IDS[:3])
def test_scale_strides_and_a_table_that_is_a_slice(dtype, d):
    api = _api()
    c = _case([50, 3], [333, 200], 6, 2, d, 32, dtype)
    want, lse = api.vda_paged_attention(**c, scale=0.3, return_lse=True)
    _check(c, want, lse, scale=0.3)
    N = c["q"].shape[0]
    joint = torch.zeros(N, 10 * d, dtype=dtype, device="cuda")
    joint[:, 2 * d:8 * d] = c["q"].flatten(1)
    into = torch.full((6, N, 2, d), 5.0, dtype=dtype, device="cuda")
    table = torch.full((2, 40), -7, dtype=torch.int32, device="cuda")
    table[:, 3:3 + c["block_table"].shape[1]] = c["block_table"]
    c2 = {**c, "q": joint[:, 2 * d:8 * d].view(N, 6, d), "block_table": table[:, 3:3 + c["block_table"].shape[1]]}
    got = api.vda_paged_attention(**c2, scale=0.3, out=into[:, :, 0].transpose(0, 1))
    assert torch.equal(got, want) and (into[:, :, 1] == 5).all()
    major = c["q"].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(api.vda_paged_attention(**{**c, "q": major}, scale=0.3), want)


@pytest.mark.parametrize("page", [8, 256, 48, 1, 7])
def test_page_sizes(page):
    for dtype, d in TYPES[:2]:
        c = _case([60, 1, 1], [300, 77, 513], 4, 2, d, page, dtype)
        out, lse = _api().vda_paged_attention(**c, return_lse=True)
        _check(c, out, lse, block=1)


@pytest.mark.parametrize("Hq,Hk", [(128, 1), (64, 1), (3, 1), (71, 1), (40, 8), (100, 2)])
def test_groups(Hq, Hk):
    for dtype, d in TYPES[:3]:
        if Hq // Hk > 64 and dtype == torch.float32:
            continue
        c = _case([3, 1, 20], [300, 77, 20], Hq, Hk, d, 16, dtype)
        out, lse = _api().vda_paged_attention(**c, return_lse=True)
        _check(c, out, lse)


def test_many_sequences():
    """More sequences than are counted at once, most with one token, some with none or many."""
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.choice([0, 1, 1, 1, 2, 70], 333)]
    length = [max(n, int(rng.integers(1, 90))) for n in new]
    for dtype, d in TYPES[:3]:
        c = _case(new, length, 4, 2, d, 16, dtype)
        out, lse = _api().vda_paged_attention(**c, return_lse=True)
        _check(c, out, lse)


def test_empty_batches():
    api = _api()
    c = _case([0, 0], [30, 5], 4, 2, 64, 16, torch.bfloat16, behind=3)
    out = torch.full_like(c["q"], 2.0)
    api.vda_paged_attention(**c, out=out)
    assert (out == 2).all()
    c = _case([0], [30], 4, 2, 64, 16, torch.bfloat16)
    assert api.vda_paged_attention(**c).shape == (0, 4, 64)


def test_the_same_bits_every_time_on_a_side_stream_and_in_a_graph():
    api = _api()
    for dtype, d in TYPES[:3]:
        c = _case([50, 1, 400], [1500, 3000, 900], 8, 2, d, 64, dtype)
        want = api.vda_paged_attention(**c, return_lse=True)
        for _ in range(3):
            assert all(torch.equal(x, y) for x, y in zip(want, api.vda_paged_attention(**c, return_lse=True)))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = api.vda_paged_attention(**c, return_lse=True)
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = api.vda_paged_attention(**c, return_lse=True)
        c["kv_len"] -= 10      # a replay follows the lengths
        graph.replay()
        torch.cuda.synchronize()
        _check(c, *got)
