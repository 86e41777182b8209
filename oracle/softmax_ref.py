"""float64 oracle of the Softmax branch's operators, in NumPy, written from
their definitions: the norm and rotation of queries and keys with its
gradient, the paged cache, and the attention of new tokens over it."""

from __future__ import annotations

import numpy as np


def _pairs(rot, interleaved):
    p = np.arange(rot // 2)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)


def angles(positions, frequencies, axis):
    """[N, rot / 2] radians; a pair whose axis does not exist is not turned."""
    positions = np.asarray(positions)
    axis = np.asarray(axis)
    known = (axis >= 0) & (axis < positions.shape[1])
    pos = positions[:, np.where(known, axis, 0)].astype(np.float64)
    return np.where(known, pos * np.asarray(frequencies, np.float64), 0.0)


def rotate(z, phi, interleaved=False):
    """z [N, H, d], phi [N, rot / 2]."""
    i, j = _pairs(2 * phi.shape[1], interleaved)
    c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
    y = z.copy()
    y[..., i] = z[..., i] * c - z[..., j] * s
    y[..., j] = z[..., j] * c + z[..., i] * s
    return y


def norm(x, eps):
    """(x / rms, 1 / rms) of the last axis."""
    inv = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * inv, inv


def norm_rope(x, w, phi, interleaved=False, eps=1e-6):
    return rotate(norm(x, eps)[0] * w, phi, interleaved)


def norm_rope_backward(dy, x, w, phi, interleaved=False, eps=1e-6):
    """(dx, dw) of norm_rope."""
    u, inv = norm(x, eps)
    g = rotate(dy, -phi, interleaved)
    dw = (g * u).sum((0, 1))
    gw = g * w
    return inv * (gw - u * (gw * u).mean(-1, keepdims=True)), dw


def paired_magnitude(z, rot, interleaved=False):
    """|z_i| + |z_j| of each channel's pair (|z_i| where it is not rotated)."""
    m = np.abs(z)
    i, j = _pairs(rot, interleaved)
    out = m.copy()
    out[..., i] = out[..., j] = m[..., i] + m[..., j]
    return out


def visible(pos, length, block, window, anchors, absent=()):
    """[len(pos), length] truth values: key j is seen from position pos."""
    pos = np.asarray(pos, np.int64)[:, None]
    j = np.arange(length, dtype=np.int64)[None]
    see = (pos >= 0) & (j >= 0)
    if block > 0:
        b = (pos - anchors) // block
        see &= j < (b + 1) * block + anchors
        if window >= 0:
            see &= (j >= (b - window) * block + anchors) | (j < anchors)
    for k in absent:
        see[:, k] = False
    return see


def attend(q, k, v, see, scale):
    """q [n, G, d], k, v [L, d], see [n, L]: (o [n, G, d], lse [n, G])."""
    n, G, d = q.shape
    o, lse = np.zeros((n, G, v.shape[1])), np.full((n, G), -np.inf)
    for i in range(n):
        at = np.flatnonzero(see[i])
        if at.size:
            s = scale * (q[i] @ k[at].T)
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            t = e.sum(-1, keepdims=True)
            o[i] = (e / t) @ v[at]
            lse[i] = (m + np.log(t))[:, 0]
    return o, lse


def paged_attention(q, k_cache, v_cache, block_table, kv_len, q_start, scale=None, block=1, window=-1, anchors=0):
    """q [N, Hq, d], caches [pages, Hk, page, d]: (out, lse), rows behind the
    last sequence zero.  A key whose page does not exist is not seen."""
    N, Hq, d = q.shape
    P, Hk, page, _ = k_cache.shape
    G = Hq // Hk
    scale = d ** -0.5 if scale is None else scale
    out, lse = np.zeros((N, Hq, d)), np.full((N, Hq), -np.inf)
    for b in range(len(kv_len)):
        t0, t1, L = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        if t1 <= t0:
            continue
        pages = np.asarray(block_table[b], np.int64)[np.arange(L) // page]
        absent = np.flatnonzero((pages < 0) | (pages >= P))
        at = np.clip(pages, 0, P - 1)
        off = np.arange(L) % page
        see = visible(np.arange(L - (t1 - t0), L), L, block, window, anchors, absent)
        for h in range(Hk):
            o, z = attend(q[t0:t1, h * G:(h + 1) * G], k_cache[at, h, off], v_cache[at, h, off], see, scale)
            out[t0:t1, h * G:(h + 1) * G], lse[t0:t1, h * G:(h + 1) * G] = o, z
    return out, lse
