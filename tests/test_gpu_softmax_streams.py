"""The Softmax branch's calls on a stream that is not the current one."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _api():
    from frame_wise_delta_vda_b200 import api
    return api


def _calls():
    """Calls on a stream, with results or a workspace of more MB than the allocator splits off."""
    api = _api()
    g = torch.Generator().manual_seed(5)
    N, Hq, Hk, d, page = 8192, 16, 4, 128, 64
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    q, k = rand(N, Hq, d), rand(N, Hk, d)
    kc, vc = rand(20, Hk, page, d), rand(20, Hk, page, d)
    w = torch.ones(d, device="cuda")
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(1, 20)
    kv_len = torch.tensor([1200], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 512], dtype=torch.int32, device="cuda")
    return {
        "norm": lambda s: api.vda_qk_norm_rope(q, k, w, w, stream=s),
        "gradient": lambda s: api.vda_qk_norm_rope_backward(q, k, q, k, w, w, stream=s),
        "attention": lambda s: api.vda_paged_attention(q[:512], kc, vc, table, kv_len, start, return_lse=True, stream=s),
    }


@pytest.mark.parametrize("name", ["norm", "gradient", "attention"])
def test_results_and_workspaces_belong_to_the_given_stream(name):
    """Memory that the current stream has let go of may still be in use there:
    a call on another stream leaves it alone (bits as they were), and gives
    the same bits as on the current stream."""
    call = _calls()[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    free = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (64 << 20, 24 << 20, 1 << 20, 512, 512)]
    at = [t.data_ptr() for t in free]
    sizes = [t.numel() for t in free]
    torch.cuda.synchronize()
    del free
    got = call(s)
    s.synchronize()
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    assert sorted(t.data_ptr() for t in again) == sorted(at)
    assert all(bool((t == 0x5A).all()) for t in again)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.cuda.current_stream() != s
