"""Empty batches through the binding: no sequences, or no pages yet."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,max_pages", [(0, 0), (0, 4), (3, 0), (3, 4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_attention_of_no_tokens(B, max_pages, dtype):
    from frame_wise_delta_vda_b200 import api
    q = torch.empty(0, 4, 64, dtype=dtype, device="cuda")
    cache = torch.zeros(5, 2, 16, 64, dtype=dtype, device="cuda")
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = api.vda_paged_attention(q, cache, cache, ints(B, max_pages), ints(B), ints(B + 1), return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    torch.cuda.synchronize()
