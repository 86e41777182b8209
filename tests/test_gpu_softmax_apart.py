"""Results beside inputs in one tensor are taken, results on inputs refused."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 33])
def test_results_in_other_columns_of_the_inputs_tensor(N):
    from frame_wise_delta_vda_b200 import api
    H, Hk, d = 4, 2, 64
    g = torch.Generator().manual_seed(N)
    joint = torch.randn(N, (2 * H + 2 * Hk) * d, generator=g).to(torch.bfloat16).cuda()
    cols = lambda a, n: joint[:, a * d:(a + n) * d].view(N, n, d)  # noqa: E731
    q, k, qo, ko = cols(0, H), cols(H, Hk), cols(H + Hk, H), cols(2 * H + Hk, Hk)
    want = api.vda_qk_norm_rope(q.clone(), k.clone())
    got = api.vda_qk_norm_rope(q, k, q_out=qo, k_out=ko)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # heads in turn: [N, H, 2, d] holds q and its result
    two = torch.randn(N, H, 2, d, generator=g).to(torch.bfloat16).cuda()
    want = api.vda_qk_norm_rope(two[:, :, 0].clone(), k.clone())[0]
    assert torch.equal(api.vda_qk_norm_rope(two[:, :, 0], k, q_out=two[:, :, 1])[0], want)
    grad = api.vda_qk_norm_rope_backward(two[:, :, 0], k, qo, ko)
    into = torch.empty(N, H, 2, d, dtype=torch.bfloat16, device="cuda")
    into[:, :, 1] = two[:, :, 0]
    got = api.vda_qk_norm_rope_backward(into[:, :, 1], k, qo, ko, dq=into[:, :, 0])
    assert torch.equal(got[0], grad[0]) and torch.equal(got[1], grad[1])
    # attention: one page, the output beside the queries
    cache = torch.randn(2, Hk, 64, d, generator=g).to(torch.bfloat16).cuda()
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (cache, cache, ints(1).view(1, 1), ints(50), ints(0, N))
    want = api.vda_paged_attention(two[:, :, 0].clone(), *args)
    assert torch.equal(api.vda_paged_attention(two[:, :, 0], *args, out=two[:, :, 1]), want)


def test_results_on_inputs_are_refused():
    from frame_wise_delta_vda_b200 import api
    q, k = (torch.randn(5, h, 64, device="cuda") for h in (4, 2))
    qw = q.clone()
    cache = torch.zeros(2, 2, 16, 64, device="cuda")
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(api.VdaError):
        api.vda_qk_norm_rope(q, k, q_out=q)
    with pytest.raises(api.VdaError):
        api.vda_qk_norm_rope(q, k, q_out=q[:, [0]].expand(5, 4, 64))
    with pytest.raises(api.VdaError):
        api.vda_qk_norm_rope_backward(q, k, qw, k, dq=q)
    with pytest.raises(api.VdaError):
        api.vda_paged_attention(q, cache, cache, ints(0, 1).view(1, 2), ints(30), ints(0, 5), out=q)
    torch.cuda.synchronize()
    assert torch.equal(q, qw)
