"""The Softmax branch of a clip: every chunk of frames sees itself, the chunks
around it and the anchor frames at both ends, through one row of the block table
a chunk (block = 0), with pages that the rows share.  Against a dense mask over
the frames (tolerances: test_gpu_paged_attention)."""

import numpy as np
import pytest

from oracle import softmax_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def chunk_tables(T, U, chunk, window, page, first=1):
    """(block_table, kv_len, q_start) of the T interior frames of a clip whose
    cache holds its T + 2 frames of U tokens one after the other, page 0 on."""
    assert U % page == 0, "a frame fills whole pages"
    per = U // page
    frame = lambda f: list(range(f * per, (f + 1) * per))  # noqa: E731
    rows, lens, start = [], [], [0]
    for t0 in range(0, T, chunk):
        lo, hi = max(0, t0 - window * chunk), min(T, t0 + (window + 1) * chunk)
        frames = [0, *range(first + lo, first + hi), T + 1]
        rows.append(sum((frame(f) for f in frames), []))
        lens.append(len(frames) * U)
        start.append(start[-1] + min(chunk, T - t0) * U)
    width = max(map(len, rows))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return ints([r + [-1] * (width - len(r)) for r in rows]), ints(lens), ints(start)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)],
                         ids=["bf16-128", "bf16-64", "f32-64"])
@pytest.mark.parametrize("T,U,chunk,window", [(11, 48, 2, 1), (10, 32, 5, 1), (7, 16, 3, 0), (6, 48, 1, 2)])
def test_own_chunk_the_chunks_around_it_and_anchors_at_both_ends(T, U, chunk, window, dtype, d):
    from frame_wise_delta_vda_b200 import api
    H, page = 3, 16
    g = torch.Generator().manual_seed(T * U)
    n = (T + 2) * U
    rand = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    q, k, v = rand(n, H, d), rand(n, H, d), rand(n, H, d)
    w = torch.ones(d, device="cuda")
    grid = U // 8
    at = torch.arange(n, device="cuda")
    pos = torch.stack([at // U, at % U // grid, at % grid], 1).to(torch.int32)
    freq, axis = api.rope_frequencies(d, sections=[d // 2 - 2 * (d // 6), d // 6, d // 6])
    kc = torch.full((n // page, H, page, d), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    ko = torch.empty_like(k)
    qo, _ = api.vda_qk_norm_rope(q, k, w, w, pos, freq, axis, v=v, k_cache=kc, v_cache=vc, slots=at, k_out=ko)
    table, kv_len, start = chunk_tables(T, U, chunk, window, page)
    out, lse = api.vda_paged_attention(qo[U:-U], kc, vc, table, kv_len, start, block=0, return_lse=True)

    frame = np.arange(n) // U
    c = (frame - 1) // chunk
    inside = (frame >= 1) & (frame <= T)
    see = (np.abs(c[:, None] - c[None]) <= window) & inside[None] | ~inside[None]
    see = see[U:-U]
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    for h in range(H):
        Q, K, V = f64(qo[U:-U, h]), f64(ko[:, h]), f64(v[:, h])
        want, z = ref.attend(Q[:, None], K, V, see, d ** -0.5)
        size, _ = ref.attend(Q[:, None], K, np.abs(V), see, d ** -0.5)
        s_err = ((d + 2) * 2.0 ** -24 * d ** -0.5 * (np.abs(Q) @ np.abs(K).T)).max(-1)
        rel = 2 * s_err + 2.0 ** -21 + see.sum(-1) * 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
        tol = u * (1 + 2.0 ** -7) * np.abs(want[:, 0]) + rel[:, None] * size[:, 0]
        assert (np.abs(f64(out[:, h]) - want[:, 0]) <= tol).all()
        assert (np.abs(f64(lse[:, h]) - z[:, 0]) <= s_err + 2.0 ** -20 * (1 + np.abs(z[:, 0]))).all()
