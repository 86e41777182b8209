"""Torch-facing binding of libvda.so, with the C ABI's names.

Argument marshalling only: shape/dtype/device checks, pointer extraction and
the current CUDA stream.  Every step of the computation runs in the library's
CUDA kernels; there is no PyTorch or CPU implementation here.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from ._lib import (VDA_BF16, VDA_F32, VDA_SCAN_AUTO, VDA_SCAN_CHUNKS, VDA_SCAN_FRAMES, VdaArgs,  # noqa: F401
                   VdaError, VdaPrepArgs, check, lib, pack_attn, pack_qk, pack_qk_grad)

_SCAN_FORMS = {"auto": VDA_SCAN_AUTO, "frames": VDA_SCAN_FRAMES, "chunks": VDA_SCAN_CHUNKS}

_DTYPES = {torch.bfloat16: VDA_BF16, torch.float32: VDA_F32}

_F32_TINY, _F32_MAX = 2.0 ** -149, (2.0 - 2.0 ** -23) * 2.0 ** 127   # the positive float32's


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check_tensor(name, t, dtype=None, shape=None, device=None, allow_none=False, on_host=False):
    if t is None:
        if allow_none:
            return
        raise ValueError(f"{name} is required")
    if on_host:
        if t.is_cuda:
            raise ValueError(f"{name} must be a host tensor")
    elif not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def make_args(q, k, v, beta, gate, rms_weight, S0_fwd, S0_rev, out, chunk, window_chunks,
              eps=1e-6, stream=None, check_device=True, alpha=None, scan_form="auto"):
    """Build the C `vda_args` block from tensors (device or host)."""
    if q.dim() != 5:
        raise ValueError("q must be [B, H, T, U, d_k]")
    Bn, Hn, T, U, d_k = q.shape
    d_v = v.shape[-1]
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype} (bf16 or float32)")
    dev = q.device
    # host tensors (vda_forward_host) get the same shape and dtype checks
    chk = _check_tensor if check_device else (lambda *a, **k: _check_tensor(*a[:4], None, **k, on_host=True))
    chk("q", q, q.dtype, (Bn, Hn, T, U, d_k), dev)
    chk("k", k, q.dtype, (Bn, Hn, T, U, d_k), dev)
    chk("v", v, q.dtype, (Bn, Hn, T, U, d_v), dev)
    chk("gate", gate, q.dtype, (Bn, Hn, T, U, d_v), dev)
    chk("out", out, q.dtype, (Bn, Hn, T, U, d_v), dev)
    chk("beta", beta, torch.float32, (Bn, Hn, T, U), dev)
    chk("rms_weight", rms_weight, torch.float32, (d_v,), dev)
    chk("S0_fwd", S0_fwd, torch.float32, (Bn, Hn, d_v, d_k), dev, allow_none=True)
    chk("S0_rev", S0_rev, torch.float32, (Bn, Hn, d_v, d_k), dev, allow_none=True)
    chk("alpha", alpha, torch.float32, (Bn, Hn, T, d_k), dev, allow_none=True)
    a = VdaArgs()
    a.dtype = dt
    a.q, a.k, a.v, a.beta, a.gate = (t.data_ptr() for t in (q, k, v, beta, gate))
    a.rms_weight = rms_weight.data_ptr()
    a.S0_fwd = S0_fwd.data_ptr() if S0_fwd is not None else None
    a.S0_rev = S0_rev.data_ptr() if S0_rev is not None else None
    a.out = out.data_ptr()
    a.B, a.H, a.T, a.U, a.d_k, a.d_v = Bn, Hn, T, U, d_k, d_v
    a.chunk, a.window_chunks = int(chunk), int(window_chunks)
    a.eps = float(eps)
    a.stream = _stream(stream).value if check_device else None
    a.alpha = alpha.data_ptr() if alpha is not None else None
    if scan_form not in _SCAN_FORMS:
        raise ValueError(f"scan_form must be one of {sorted(_SCAN_FORMS)}")
    a.scan_form = _SCAN_FORMS[scan_form]
    return a


def vda_workspace_bytes(B, H, T, U, d_k, d_v, chunk, dtype=torch.bfloat16):
    return int(lib().vda_workspace_bytes(B, H, T, U, d_k, d_v, chunk, _DTYPES[dtype]))


def workspace_for(q, v, chunk):
    """A device workspace tensor sized for these inputs (uint8, 256-aligned)."""
    Bn, Hn, T, U, d_k = q.shape
    n = vda_workspace_bytes(Bn, Hn, T, U, d_k, v.shape[-1], chunk, q.dtype)
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def vda_forward(q, k, v, beta, gate, rms_weight, S0_fwd=None, S0_rev=None, chunk=5,
                window_chunks=1, out=None, workspace=None, states_out=None, stats_out=None,
                eps=1e-6, stream=None, alpha=None, scan_form="auto"):
    """Bidirectional VDA forward (see include/vda.h).  Returns `out`.

    Without `workspace`, `states_out`, `stats_out`, `alpha` or a `scan_form`
    other than "auto" this calls `vda_forward` / `vda_forward_f32`
    (stream-ordered workspace); otherwise `vda_forward_ex`.  `alpha`
    [B, H, T, d_k] float32 adds the decay gate; `scan_form` ("auto", "frames",
    "chunks") selects the scan form of the tensor-core path.
    """
    if out is None:
        out = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    a = make_args(q, k, v, beta, gate, rms_weight, S0_fwd, S0_rev, out, chunk, window_chunks, eps, stream,
                  alpha=alpha, scan_form=scan_form)
    L = lib()
    if (workspace is None and states_out is None and stats_out is None and eps == 1e-6 and alpha is None
            and scan_form == "auto"):
        fn = L.vda_forward if a.dtype == VDA_BF16 else L.vda_forward_f32
        rc = fn(a.q, a.k, a.v, a.beta, a.gate, a.rms_weight, a.S0_fwd, a.S0_rev,
                a.B, a.H, a.T, a.U, a.d_k, a.d_v, a.chunk, a.window_chunks, a.out, a.stream)
        check(rc, "vda_forward")
        return out
    if workspace is None:
        workspace = workspace_for(q, v, chunk)
    for name, t in (("states_out", states_out), ("stats_out", stats_out)):
        if t is not None:
            _check_tensor(name, t, torch.float32, None, q.device)
    rc = L.vda_forward_ex(ctypes.byref(a), _ptr(workspace), workspace.numel(),
                          _ptr(states_out), _ptr(stats_out))
    check(rc, "vda_forward_ex")
    return out


def vda_prep(q_in, k_in, v_in, wk_s, wk_t, wv_s, wv_t, Hl, Wl, q_out=None, k_out=None, v_out=None,
             eps=1e-6, stream=None):
    """Feature preparation of the linear branch (see include/vda.h):
    q_in, k_in, v_in [B, T, U, H, d] bf16 (U = Hl * Wl) -> q', k', v'
    [B, H, T, U, d] bf16 with q' = L2(q), k' = L2(SiLU(conv(k))),
    v' = SiLU(conv(v)); filters wk_s, wv_s [H, d, 5, 5], wk_t, wv_t [H, d, 5]
    float32.  Returns (q_out, k_out, v_out)."""
    if q_in.dim() != 5:
        raise ValueError("q_in must be [B, T, U, H, d]")
    Bn, T, U, Hn, d = q_in.shape
    if U != Hl * Wl:
        raise ValueError(f"U = {U} is not Hl * Wl = {Hl} * {Wl}")
    dev = q_in.device
    for name, t in (("q_in", q_in), ("k_in", k_in), ("v_in", v_in)):
        _check_tensor(name, t, torch.bfloat16, (Bn, T, U, Hn, d), dev)
    for name, t in (("wk_s", wk_s), ("wv_s", wv_s)):
        _check_tensor(name, t, torch.float32, (Hn, d, 5, 5), dev)
    for name, t in (("wk_t", wk_t), ("wv_t", wv_t)):
        _check_tensor(name, t, torch.float32, (Hn, d, 5), dev)
    outs = []
    for name, t in (("q_out", q_out), ("k_out", k_out), ("v_out", v_out)):
        if t is None:
            t = torch.empty((Bn, Hn, T, U, d), dtype=torch.bfloat16, device=dev)
        _check_tensor(name, t, torch.bfloat16, (Bn, Hn, T, U, d), dev)
        outs.append(t)
    a = VdaPrepArgs()
    a.q_in, a.k_in, a.v_in = q_in.data_ptr(), k_in.data_ptr(), v_in.data_ptr()
    a.wk_s, a.wk_t, a.wv_s, a.wv_t = wk_s.data_ptr(), wk_t.data_ptr(), wv_s.data_ptr(), wv_t.data_ptr()
    a.q_out, a.k_out, a.v_out = (t.data_ptr() for t in outs)
    a.B, a.H, a.T, a.Hl, a.Wl, a.d = Bn, Hn, T, int(Hl), int(Wl), d
    a.eps = float(eps)
    a.stream = _stream(stream).value
    check(lib().vda_prep(ctypes.byref(a)), "vda_prep")
    return tuple(outs)


# ---------------------------------------------------------------------------
# Softmax branch: norm and rotation of queries and keys, paged cache, attention.
#
# A serving step makes these calls once a layer on a handful of tokens, where
# the kernel takes a few microseconds: a tensor that is as it should be is
# looked at once, and only one that is not goes through the checks that say why.
def _call(index, fn, *args):
    """fn(*args) with device `index` current, as the library launches there."""
    if torch._C._cuda_getDevice() == index:
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def _on(stream, fn, given):
    """fn with the arguments `given` (their `stream` among them) and that stream
    current: what the call allocates then belongs to the stream that uses it,
    and is not handed out on another one while the kernels run."""
    t = given["q"]
    if t.is_cuda and stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, q on {t.device}")
    with torch.cuda.stream(stream):
        return fn(**{**given, "stream": None})


def _pack(pack, *fields):
    try:
        return pack(*fields)
    except struct.error as e:   # a size that its C type does not hold
        raise ValueError(f"argument out of range: {e}") from None


def _at(name, t, dtype, shape, index):
    """Address of a contiguous tensor on device `index`."""
    if t is not None and t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _check_tensor(name, t, dtype, shape, torch.device("cuda", index))
    return t.data_ptr()


def _rows(name, t, dtype, shape, index):
    """(address, token stride, head stride) of [N, heads, d] with contiguous
    channels and any token and head strides."""
    if t is not None and t.dtype is dtype and t.get_device() == index and t.shape == shape:
        st = t.stride()
        if st[2] == 1:
            return t.data_ptr(), st[0], st[1]
        raise ValueError(f"{name} must have contiguous channels")
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _workspace(t, index):
    """(address, bytes) of a workspace that the caller keeps, or of none."""
    if t is None:
        return 0, 0
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{index}")
    return t.data_ptr(), t.numel() * t.element_size()


def rope_frequencies(rot, theta=10000.0, sections=None, device="cuda"):
    """The (frequencies, axis) arguments of `vda_qk_norm_rope`: radians per
    position theta ** (-2 i / c) of the i-th pair of each axis, the c = 2 *
    pairs channels of the axes side by side.  `sections` lists the pairs of
    each axis (default: one axis with all rot / 2)."""
    if rot % 2:
        raise ValueError("rot must be even")
    sections = [rot // 2] if sections is None else list(sections)
    if sum(sections) != rot // 2 or min(sections, default=0) < 0:
        raise ValueError(f"sections {sections} must add up to rot / 2 = {rot // 2}")
    freq = [theta ** (-i / c) for c in sections for i in range(c)]
    axis = [a for a, c in enumerate(sections) for _ in range(c)]
    return (torch.tensor(freq, dtype=torch.float64, device=device),
            torch.tensor(axis, dtype=torch.int32, device=device))


def _rotation(N, positions, frequencies, axis, index):
    """(positions, frequencies, axis, axes, rot) of the argument block."""
    if frequencies is None:
        if positions is not None or axis is not None:
            raise ValueError("positions and axis need frequencies")
        return 0, 0, 0, 0, 0
    half = frequencies.numel()
    if positions is None or positions.dim() != 2:
        raise ValueError("positions must be [N, axes]")
    axes = positions.shape[1]
    return (_at("positions", positions, torch.int32, (N, axes), index),
            _at("frequencies", frequencies, torch.float64, (half,), index),
            _at("axis", axis, torch.int32, (half,), index), axes, 2 * half)


def _weight(name, w, d, index):
    return 0 if w is None else _at(name, w, torch.float32, (d,), index)


def _qk_shapes(q, k, eps):
    if not _F32_TINY <= eps <= _F32_MAX:   # what rounds to 0 would select the default
        raise ValueError(f"eps must be a positive float32, got {eps}")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [N, heads, d]")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype} (bf16 or float32)")
    N, Hq, d = q.shape
    return N, Hq, k.shape[1], d, dt


def _cache(k_cache, v_cache, dtype, Hk, d, index):
    """(k_cache, v_cache, pages, page_size) of [pages, Hk, page_size, d], contiguous."""
    if k_cache is None or v_cache is None or k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [pages, Hk, page_size, d]")
    shape = (k_cache.shape[0], Hk, k_cache.shape[2], d)
    return (_at("k_cache", k_cache, dtype, shape, index), _at("v_cache", v_cache, dtype, shape, index), shape[0], shape[2])


def vda_qk_norm_rope(q, k, q_weight=None, k_weight=None, positions=None, frequencies=None, axis=None,
                     interleaved=False, eps=1e-6, v=None, k_cache=None, v_cache=None, slots=None, q_out=None,
                     k_out=None, stream=None):
    """RMS norm of each head of q [N, Hq, d] and k [N, Hk, d] (weights [d]
    float32) and the rotation of its first 2 * len(frequencies) channels by
    positions [N, axes] int32 (see include/vda.h and `rope_frequencies`);
    `eps` is positive.  q, k and v may be strided over tokens and heads (slices
    of a joint projection).  With `slots` [N] int64, k's result and v [N, Hk, d]
    go to those places of k_cache and v_cache [pages, Hk, page_size, d] (slot =
    page * page_size + offset; -1: not stored).  Results must not lie on inputs
    (not in place).  Returns (q_out, k_out); k_out is None when only the cache
    receives k.  Autograd does not see the call: its gradient is
    `vda_qk_norm_rope_backward`."""
    if stream is not None:
        return _on(stream, vda_qk_norm_rope, locals())
    N, Hq, Hk, d, dt = _qk_shapes(q, k, eps)
    dtype, i = q.dtype, q.get_device()
    rows_q, rows_k, rows_v, rows_ko = _rows("q", q, dtype, (N, Hq, d), i), _rows("k", k, dtype, (N, Hk, d), i), (0, 0, 0), (0, 0, 0)
    pos, freq, ax, axes, rot = _rotation(N, positions, frequencies, axis, i)
    at_slots = at_kc = at_vc = pages = page = 0
    if slots is not None:
        at_slots = _at("slots", slots, torch.int64, (N,), i)
        at_kc, at_vc, pages, page = _cache(k_cache, v_cache, dtype, Hk, d, i)
        rows_v = _rows("v", v, dtype, (N, Hk, d), i)
    elif k_cache is not None or v_cache is not None or v is not None:
        raise ValueError("v, k_cache and v_cache need slots")
    if q_out is None:
        q_out = q.new_empty((N, Hq, d))
    if k_out is None and slots is None:
        k_out = q.new_empty((N, Hk, d))
    if k_out is not None:
        rows_ko = _rows("k_out", k_out, dtype, (N, Hk, d), i)
    args = _pack(
        pack_qk, dt, *rows_q, *rows_k, *rows_v, *_rows("q_out", q_out, dtype, (N, Hq, d), i), *rows_ko,
        _weight("q_weight", q_weight, d, i), _weight("k_weight", k_weight, d, i), pos, freq, ax,
        at_slots, at_kc, at_vc, N, Hq, Hk, d, axes, rot, 1 if interleaved else 0, pages, page, eps,
        torch._C._cuda_getCurrentRawStream(i))
    check(_call(i, lib().vda_qk_norm_rope, args), "vda_qk_norm_rope")
    return q_out, k_out


def vda_qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight=None, k_weight=None, positions=None, frequencies=None,
                              axis=None, interleaved=False, eps=1e-6, dq=None, dk=None, workspace=None, stream=None):
    """Gradient of `vda_qk_norm_rope`: from the gradients of its results
    [N, heads, d] (strided, or broadcast with stride 0, as they come) and its
    inputs, returns (dq, dk, dq_weight, dk_weight); the weight gradients are
    float32 [d], sums in a fixed order (None for a weight that is None)."""
    if stream is not None:
        return _on(stream, vda_qk_norm_rope_backward, locals())
    N, Hq, Hk, d, dt = _qk_shapes(q, k, eps)
    dtype, i = q.dtype, q.get_device()
    pos, freq, ax, axes, rot = _rotation(N, positions, frequencies, axis, i)
    if dq is None:
        dq = q.new_empty((N, Hq, d))
    if dk is None:
        dk = q.new_empty((N, Hk, d))
    rows = (*_rows("dq_out", dq_out, dtype, (N, Hq, d), i), *_rows("dk_out", dk_out, dtype, (N, Hk, d), i),
            *_rows("q", q, dtype, (N, Hq, d), i), *_rows("k", k, dtype, (N, Hk, d), i),
            *_rows("dq", dq, dtype, (N, Hq, d), i), *_rows("dk", dk, dtype, (N, Hk, d), i))
    L = lib()
    dwq, dwk = torch.empty((2, d), dtype=torch.float32, device=q.device).unbind(0)
    if q_weight is None:
        dwq = None
    if k_weight is None:
        dwk = None
    at_wq, at_wk = _weight("q_weight", q_weight, d, i), _weight("k_weight", k_weight, d, i)
    if workspace is None and (at_wq or at_wk):
        workspace = torch.empty(L.vda_qk_grad_workspace_bytes(d), dtype=torch.uint8, device=q.device)
    args = _pack(
        pack_qk_grad, dt, *rows, at_wq, at_wk, dwq.data_ptr() if at_wq else 0, dwk.data_ptr() if at_wk else 0, pos, freq, ax,
        N, Hq, Hk, d, axes, rot, 1 if interleaved else 0, eps, torch._C._cuda_getCurrentRawStream(i))
    check(_call(i, L.vda_qk_norm_rope_backward, args, *_workspace(workspace, i)), "vda_qk_norm_rope_backward")
    return dq, dk, dwq, dwk


def vda_paged_attention_workspace_bytes(N, B, Hq, Hk, d, page_size, dtype=torch.bfloat16):
    return int(lib().vda_paged_attention_workspace_bytes(_DTYPES[dtype], N, B, Hq, Hk, d, page_size))


def vda_paged_attention(q, k_cache, v_cache, block_table, kv_len, q_start, block=1, window_blocks=-1, anchors=0,
                        scale=None, out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """Attention of the new tokens q [N, Hq, d] of B sequences over the paged
    cache k_cache, v_cache [pages, Hk, page_size, d], which holds their keys
    already (see include/vda.h).  block_table [B, max_pages], kv_len [B] and
    q_start [B + 1] are int32 on the device; sequence b's new tokens are rows
    q_start[b] .. q_start[b + 1] and its last positions.  `block` 1 is causal
    by token, n >= 2 by blocks of n tokens, 0 sees every key; `window_blocks`
    blocks before a token's own are seen (-1: all), and those of the first
    `anchors` keys that lie before the end of its own block; blocks are counted
    from the end of the anchors.  Other sets of keys, such as a window on both
    sides of a clip's chunk, are given by the table: a sequence per chunk with
    block 0, whose row lists the (shared, full) pages it sees.  `scale` defaults to 1 / sqrt(d).  Returns out [N, Hq, d], or
    (out, lse [N, Hq] float32) with return_lse.  Calls that may overlap need
    workspaces of their own (the default is a new one)."""
    if stream is not None:
        return _on(stream, vda_paged_attention, locals())
    if scale is None:
        scale = 0.0
    elif not _F32_TINY <= scale < 1e30:   # what rounds to 0 would select the default
        raise ValueError(f"scale must be at least 2 ** -149 and below 1e30, got {scale}")
    if q.dim() != 3:
        raise ValueError("q must be [N, Hq, d]")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dtype, i = q.dtype, q.get_device()
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {dtype} (bf16 or float32)")
    N, Hq, d = q.shape
    rows_q = _rows("q", q, dtype, (N, Hq, d), i)
    if k_cache is None or k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [pages, Hk, page_size, d]")
    Hk = k_cache.shape[1]
    at_kc, at_vc, pages, page = _cache(k_cache, v_cache, dtype, Hk, d, i)
    if block_table is None or block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    if block_table.get_device() != i or block_table.dtype is not torch.int32:
        raise ValueError(f"block_table must be int32 on cuda:{i}")
    table_stride, one = block_table.stride()
    if max_pages > 1 and one != 1:
        raise ValueError("block_table must have contiguous rows")
    if out is None:
        out = q.new_empty((N, Hq, d))
    if lse is None:
        if return_lse:
            lse = torch.empty((N, Hq), dtype=torch.float32, device=q.device)
            at_lse = lse.data_ptr()
        else:
            at_lse = 0
    else:
        at_lse = _at("lse", lse, torch.float32, (N, Hq), i)
    L = lib()
    args = _pack(
        pack_attn, dt, *rows_q, at_kc, at_vc, block_table.data_ptr(), _at("kv_len", kv_len, torch.int32, (B,), i),
        _at("q_start", q_start, torch.int32, (B + 1,), i), *_rows("out", out, dtype, (N, Hq, d), i), at_lse, table_stride,
        N, B, Hq, Hk, d, pages, page, max_pages, block, window_blocks, anchors, scale,
        torch._C._cuda_getCurrentRawStream(i))
    if workspace is None:
        n = _call(i, L.vda_paged_attention_workspace_bytes, dt, N, B, Hq, Hk, d, page)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    check(_call(i, L.vda_paged_attention, args, *_workspace(workspace, i)), "vda_paged_attention")
    return (out, lse) if return_lse else out


def vda_text_state(k_text, v_text, beta_text, S_out=None, workspace=None, stream=None):
    """S = B'(I + A')^{-1} per (b, h) from L prompt tokens (one frame-wise
    update of the zero state).  k_text [B,H,L,d_k], v_text [B,H,L,d_v],
    beta_text [B,H,L] float32.  Returns S [B,H,d_v,d_k] float32."""
    Bn, Hn, Lt, d_k = k_text.shape
    d_v = v_text.shape[-1]
    dt = _DTYPES[k_text.dtype]
    _check_tensor("k_text", k_text, k_text.dtype, (Bn, Hn, Lt, d_k))
    _check_tensor("v_text", v_text, k_text.dtype, (Bn, Hn, Lt, d_v), k_text.device)
    _check_tensor("beta_text", beta_text, torch.float32, (Bn, Hn, Lt), k_text.device)
    if S_out is None:
        S_out = torch.empty((Bn, Hn, d_v, d_k), dtype=torch.float32, device=k_text.device)
    _check_tensor("S_out", S_out, torch.float32, (Bn, Hn, d_v, d_k), k_text.device)
    L = lib()
    n = int(L.vda_text_state_workspace_bytes(Bn, Hn, Lt, d_k, d_v, dt))
    if workspace is None:
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=k_text.device)
    rc = L.vda_text_state(dt, _ptr(k_text), _ptr(v_text), _ptr(beta_text), Bn, Hn, Lt, d_k, d_v,
                          _ptr(S_out), _ptr(workspace), workspace.numel(), _stream(stream))
    check(rc, "vda_text_state")
    return S_out


def vda_forward_host_bytes(q, v, chunk):
    Bn, Hn, T, U, d_k = q.shape
    return int(lib().vda_forward_host_bytes(Bn, Hn, T, U, d_k, v.shape[-1], chunk, _DTYPES[q.dtype]))


def vda_forward_host(q, k, v, beta, gate, rms_weight, S0_fwd, S0_rev, out, chunk, window_chunks,
                     device_buffer, eps=1e-6, alpha=None):
    """End-to-end forward from host (CPU, ideally pinned) tensors; copies in,
    computes on the current CUDA device and copies `out` back (synchronous)."""
    for name, t in (("q", q), ("k", k), ("v", v), ("beta", beta), ("gate", gate),
                    ("rms_weight", rms_weight), ("out", out), ("S0_fwd", S0_fwd), ("S0_rev", S0_rev),
                    ("alpha", alpha)):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous host tensor")
    a = make_args(q, k, v, beta, gate, rms_weight, S0_fwd, S0_rev, out, chunk, window_chunks, eps,
                  check_device=False, alpha=alpha)
    if not device_buffer.is_cuda:
        raise ValueError("device_buffer must be a CUDA tensor")
    rc = lib().vda_forward_host(ctypes.byref(a), _ptr(device_buffer), device_buffer.numel())
    check(rc, "vda_forward_host")
    return out


def vda_forward_noalloc(q, k, v, beta, gate, rms_weight, S0_fwd=None, S0_rev=None, chunk=5,
                        window_chunks=1, out=None, eps=1e-6, stream=None, alpha=None):
    """Forward through `vda_forward_noalloc`: the library uses its fixed
    internal scratch array instead of any allocation (sizes must fit in
    NOALLOC_SCRATCH_BYTES of workspace).  The caller passes a preallocated
    `out`: this route exists for callers that cannot allocate, so it never
    creates a tensor itself."""
    if out is None:
        raise ValueError("vda_forward_noalloc needs a preallocated `out` (this route allocates nothing)")
    a = make_args(q, k, v, beta, gate, rms_weight, S0_fwd, S0_rev, out, chunk, window_chunks, eps, stream,
                  alpha=alpha)
    check(lib().vda_forward_noalloc(ctypes.byref(a)), "vda_forward_noalloc")
    return out


def vda_device_status(stream=None):
    """Synchronise and return the library's device error status (0 = OK)."""
    return int(lib().vda_device_status(_stream(stream)))


def vda_launches_per_forward(B, H, T, U, d_k, d_v, chunk, dtype=torch.bfloat16):
    return int(lib().vda_launches_per_forward(B, H, T, U, d_k, d_v, chunk, _DTYPES[dtype]))


class StageTimer:
    """Per-stage device time (stats, inverse, scan, readout) of the next
    `max_calls` forward calls, from CUDA events the library records on the
    launching stream."""

    NAMES = ("stats", "inverse", "scan", "readout")

    def __init__(self, max_calls):
        check(lib().vda_timing_enable(int(max_calls)), "vda_timing_enable")

    def read(self):
        ms = (ctypes.c_float * 4)()
        calls = ctypes.c_int(0)
        check(lib().vda_timing_read(ms, 4, ctypes.byref(calls)), "vda_timing_read")
        return {n: float(ms[i]) for i, n in enumerate(self.NAMES)}, int(calls.value)
