"""Items whose keys so many shares took that their parts are joined in several
groups of 32, against the float64 oracle (tolerances: test_gpu_paged_attention)."""

import pytest

from test_gpu_paged_attention import _case, _check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64), (torch.float32, 128),
                                     (torch.bfloat16, 32), (torch.float32, 16)],
                         ids=["bf16-128", "bf16-64", "f32-64", "f32-128", "bf16-32", "f32-16"])
@pytest.mark.parametrize("new,length,Hq,Hk", [
    ([1], [8000], 1, 1),             # one item: 63 tiles of 128 keys or 125 of 64, a share each
    ([1], [40_000], 4, 1),           # every CTA has a part
    ([1], [9001], 8, 2),
    ([3, 1], [12_000, 300], 5, 1),
    ([70], [20_000], 2, 1),          # two row tiles
], ids=str)
def test_parts_joined_in_several_groups(new, length, Hq, Hk, dtype, d):
    from frame_wise_delta_vda_b200 import api
    c = _case(new, length, Hq, Hk, d, 16, dtype, seed=len(new) + Hq)
    out, lse = api.vda_paged_attention(**c, return_lse=True)
    _check(c, out, lse)
    # the largest score in one of the last groups, then in the first
    for key in (length[0] - 5, 3):
        p = int(c["block_table"][0, key // 16])
        c["k_cache"][p, :, key % 16] = 3 * c["q"][0, 0] / d ** 0.25
        out, lse = api.vda_paged_attention(**c, return_lse=True)
        _check(c, out, lse)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64)], ids=["bf16-128", "f32-64"])
def test_only_one_part_has_keys(dtype, d):
    """All pages but one are gone: every other part sees nothing."""
    from frame_wise_delta_vda_b200 import api
    c = _case([1], [9000], 4, 1, d, 16, dtype)
    keep = int(c["block_table"][0, 400])
    c["block_table"][0] = -1
    for at in (400, 0, 562):
        c["block_table"][0, at] = keep
        out, lse = api.vda_paged_attention(**c, return_lse=True)
        c["k_cache"].nan_to_num_(0.0)
        c["v_cache"].nan_to_num_(0.0)
        _check(c, out, lse)
        c["block_table"][0, at] = -1
