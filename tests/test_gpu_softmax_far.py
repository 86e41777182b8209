"""The Softmax branch's operators where element offsets pass 32 bits: pages at
the end of a cache of 2^32 elements, tokens 2^31 elements apart.  The same bits
as from a small cache and from contiguous rows, which are held to the oracle
elsewhere.  d = 128 runs on the tensor cores, d = 32 on the SIMT kernel."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [128, 32])
def test_far_pages_and_far_tokens(d):
    from frame_wise_delta_vda_b200 import api
    Hq, Hk, page, N = 8, 2, 64, 3
    per = Hk * page * d
    pages = (1 << 32) // per + 3
    if torch.cuda.mem_get_info()[0] < 3 * 2 * per * pages:
        pytest.skip("needs 26 GB of device memory")
    g = torch.Generator().manual_seed(d)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    used = [pages - 1, 0, (1 << 31) // per, pages - 3, (1 << 31) // per - 1]   # in the order of the keys
    keys = 64 * len(used) - 5
    small_k, small_v = rand(len(used), Hk, page, d), rand(len(used), Hk, page, d)
    big_k, big_v = (torch.empty(pages, Hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i, p in enumerate(used):
        big_k[p], big_v[p] = small_k[i], small_v[i]

    # rows 2^31 elements apart
    far = torch.empty((N - 1) * (1 << 31) + 2 * Hq * d, dtype=torch.bfloat16, device="cuda")
    at = lambda first, heads: far.as_strided((N, heads, d), (1 << 31, d, 1), first * d)
    q, k, v = rand(N, Hq, d), rand(N, Hk, d), rand(N, Hk, d)
    far_q, far_out = at(0, Hq), at(Hq, Hq)
    far_q.copy_(q)
    freq, axis = api.rope_frequencies(d)
    pos = torch.arange(keys - N, keys, dtype=torch.int32, device="cuda").view(N, 1)
    last = [(keys - N + i) // page for i in range(N)], [(keys - N + i) % page for i in range(N)]
    slots = lambda ids: torch.tensor([ids[p] * page + o for p, o in zip(*last)], dtype=torch.int64, device="cuda")

    q_small, _ = api.vda_qk_norm_rope(q, k, None, None, pos, freq, axis, v=v, k_cache=small_k, v_cache=small_v,
                                      slots=slots(range(len(used))))
    api.vda_qk_norm_rope(far_q, k, None, None, pos, freq, axis, v=v, k_cache=big_k, v_cache=big_v, slots=slots(used),
                         q_out=far_out)
    assert torch.equal(far_out, q_small)
    for i, p in enumerate(used):
        assert torch.equal(big_k[p], small_k[i]) and torch.equal(big_v[p], small_v[i])

    kv_len = torch.tensor([keys], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    table = lambda ids: torch.tensor([list(ids)], dtype=torch.int32, device="cuda")
    want = api.vda_paged_attention(q_small, small_k, small_v, table(range(len(used))), kv_len, start)
    far_q.copy_(q_small)
    api.vda_paged_attention(far_q, big_k, big_v, table(used), kv_len, start, out=far_out)
    assert torch.equal(far_out, want)

    dq, dk, _, _ = api.vda_qk_norm_rope_backward(want, k, q, k, None, None, pos, freq, axis)
    far_dq = at(0, Hq)
    api.vda_qk_norm_rope_backward(far_out, k, q, k, None, None, pos, freq, axis, dq=far_dq)
    assert torch.equal(far_dq, dq)
    del big_k, big_v, far, far_q, far_out, far_dq
    torch.cuda.empty_cache()
