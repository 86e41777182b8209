"""vda_paged_attention over the longest sequences, with most pages absent.

Tolerances as in test_gpu_paged_attention, for n the keys that are there:
an output is off by at most 2 s_err + 2^-21 + n 2^-24 (and 2^-8 for the tensor
cores' weights) of sum_j p_j |v_j| and half a step of its own, lse by
s_err + 2^-20 (1 + |lse|), with s_err = (d + 2) 2^-24 max sum |q k| scale."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _near(out, lse, q, K, V, dtype, d):
    """q [G, d], K and V [keys, d] that are seen, on the GPU."""
    q, K, V = q.double(), K.double(), V.double()
    s = q @ K.T * d ** -0.5
    s_err = (d + 2) * 2.0 ** -24 * d ** -0.5 * (q.abs() @ K.abs().T).max(-1).values
    z = torch.logsumexp(s, -1)
    p = torch.exp(s - z[:, None])
    want, size = p @ V, p @ V.abs()
    rel = 2 * s_err + 2.0 ** -21 + K.shape[0] * 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    tol = U[dtype] * (1 + 2.0 ** -7) * want.abs() + rel[:, None] * size
    assert float(((out.double() - want).abs() / tol).max()) <= 1.0
    assert float(((lse.double() - z).abs() / (s_err + 2.0 ** -20 * (1 + z.abs()))).max()) <= 1.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("L", [2 ** 31 - 1, 2 ** 31 - 200])
def test_keys_at_the_end_of_31_bits(dtype, L):
    """A table of 2^31 places of which three pages are there, the first and the last among them."""
    from frame_wise_delta_vda_b200 import api
    d, G, page = 64, 4, 1 << 16
    g = torch.Generator().manual_seed(7)
    rand = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    kc, vc = rand(3, 1, page, d), rand(3, 1, page, d)
    q = 2 * rand(1, G, d)
    table = torch.full((1, 1 << 15), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, 1 << 14], table[0, (1 << 15) - 1] = 1, 2, 0
    end = L - (2 ** 31 - page)                 # keys in the last page
    kc[0, 0, end:] = float("nan")
    vc[0, 0, end:] = float("nan")
    kv_len = torch.tensor([L], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")

    out, lse = api.vda_paged_attention(q, kc, vc, table, kv_len, start, block=0, return_lse=True)
    pick = lambda c: torch.cat([c[1, 0], c[2, 0], c[0, 0, :end]])  # noqa: E731
    _near(out[0], lse[0], q[0], pick(kc), pick(vc), dtype, d)

    out, lse = api.vda_paged_attention(q, kc, vc, table, kv_len, start, window_blocks=199, anchors=70, return_lse=True)
    pick = lambda c: torch.cat([c[1, 0, :70], c[0, 0, end - 200:end]])  # noqa: E731
    _near(out[0], lse[0], q[0], pick(kc), pick(vc), dtype, d)
    assert api.vda_device_status() == 0
