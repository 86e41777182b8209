"""Operators of the Softmax side of the hybrid attention block: the norm and position rotation of the queries and keys
of each head (with the cache append of a serving step, and its gradient), and the attention of new tokens over a
paged cache.

``listed()`` and ``draw()`` give the cases, ``prepare()`` their inputs on the GPU, ``run()`` one pass, ``exact()`` the
same outputs from the definitions in 64 bits, and ``work()`` the bytes and operations that a pass cannot do without.
``own`` selects the calls of this package (true) or the operators' plain form in elementary torch operations (false).

The formulas.  A head's vector x of d channels, weight w, angles phi_p = position[axis_p] * frequency_p:

    x^ = x / sqrt(mean(x^2) + eps),   z = w * x^,   (y_i, y_j) = (z_i cos - z_j sin, z_j cos + z_i sin)

for each rotated pair p = (i, j): (p, p + rot / 2), or (2 p, 2 p + 1) when interleaved; channels from rot on are not
rotated.  The gradient of y gives g = R^T dy, dw = sum of g x^ and dx = (g w - x^ mean(g w x^)) / sqrt(mean(x^2) + eps).

Query i of the n new tokens of a sequence of `len` cached keys stands at position p = len - n + i.  With `block` >= 1
positions fall into blocks floor((p - anchors) / block), and the query sees the keys of its own block and of the
`window` blocks before it (all blocks before it when window < 0), and the first `anchors` keys; with block = 0 it sees
every key.  o = softmax(scale q K^T) V over the keys it sees, lse = log of the sum of exponents; o = 0 and lse = -inf
where it sees none.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
GRID = (24, 42)          # rows and columns of a latent frame: 1008 tokens
FRAME = GRID[0] * GRID[1]


def _rope(name, op, tokens, heads, kv_heads, dim, dtype, rot, axes, start, interleaved=False, append=False, page=16):
    return dict(name=name, op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, rot=rot, axes=axes,
                start=start, interleaved=interleaved, append=append, page=page)


def _attend(name, seqs, new, ctx, heads, kv_heads, dim, dtype, page, block, window, anchors, ragged):
    return dict(name=name, op="attend", seqs=seqs, new=new, ctx=ctx, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                page=page, block=block, window=window, anchors=anchors, ragged=ragged)


def listed():
    return [
        # one serving step of a batch of eight: every sequence's new token is normed, rotated and put into the cache
        _rope("norm-rotate step of 8", "rope", 8, 32, 8, 128, "bf16", 128, 1, 100_000, append=True, page=16),
        # a prompt's chunk on its way into the cache, grouped heads
        _rope("norm-rotate prompt 4099", "rope", 4099, 32, 8, 128, "bf16", 128, 1, 0, append=True, page=64),
        # a whole clip of 60 latent frames of 24 x 42 tokens, 48 heads, frame/row/column rotation
        _rope("norm-rotate clip", "rope", 60 * FRAME, 48, 48, 128, "bf16", 128, 3, 0),
        # float32 checking of a small model: a partial, interleaved rotation at far positions
        _rope("norm-rotate f32", "rope", 1337, 16, 4, 64, "f32", 32, 1, 1_000_000, interleaved=True),
        # the gradient in a training step on 20 latent frames
        _rope("norm-rotate gradient clip", "rope_grad", 20 * FRAME, 48, 48, 128, "bf16", 128, 3, 0),
        # the gradient in float32, grouped heads, a token count that fills no tile
        _rope("norm-rotate gradient f32", "rope_grad", 777, 16, 4, 64, "f32", 64, 1, 5000),
        # the smallest serving step: one new token of one sequence
        _attend("attend 1 token", 1, 1, 1000, 32, 8, 128, "bf16", 16, 1, -1, 0, False),
        # a serving batch of 64 sequences of very different lengths, one new token each
        _attend("attend step of 64", 64, 1, 8200, 32, 8, 128, "bf16", 64, 1, -1, 0, True),
        # two sequences with long caches
        _attend("attend long cache", 2, 1, 131_000, 32, 8, 128, "bf16", 128, 1, -1, 0, False),
        # a chunk of a long prompt over what is cached of it
        _attend("attend prompt chunk", 1, 4096, 16_400, 32, 8, 128, "bf16", 64, 1, -1, 0, False),
        # livestream video, one of eight head shards: the new chunk of five frames sees itself, the two chunks before it
        # and the anchor frame
        _attend("attend video chunk", 1, 5 * FRAME, 26 * FRAME, 6, 6, 128, "bf16", 16, 5 * FRAME, 2, FRAME, False),
        # float32 checking of ragged prompts with a sliding window of 128 tokens and four anchors
        _attend("attend f32 window", 5, 333, 1111, 8, 2, 64, "f32", 16, 1, 127, 4, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    dim = rng.choice([64, 128, 128])
    kv = _log(rng, 1, 48)
    if rng.random() < 0.5:
        heads, kv = (kv, kv) if rng.random() < 0.3 else (max(1, kv // 6) * rng.choice([1, 2, 4, 5, 8]), max(1, kv // 6))
        most = 60 * FRAME * 96 * 128 // ((heads + kv) * dim)
        axes = rng.choice([1, 1, 3])
        op = rng.choice(["rope", "rope", "rope_grad"])
        if op == "rope_grad":
            most //= 3
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return _rope("", op, _log(rng, 1, min(most // (2 if dtype == "f32" else 1), 70_000)), heads, kv, dim, dtype,
                     rng.choice([dim, dim, dim // 2]), axes, rng.choice([0, _log(rng, 1, 1_000_000)]),
                     interleaved=rng.random() < 0.3, append=op == "rope" and axes == 1 and rng.random() < 0.5,
                     page=rng.choice([16, 32, 64, 128]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
    kv = max(1, kv // 6)
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    f32 = dtype == "f32"
    if rng.random() < 0.5:   # serving steps
        seqs = _log(rng, 1, 128)
        ctx = _log(rng, 1, max(2, min(131_000, (60_000 if f32 else 1_000_000) * 8 // (seqs * kv))))
        new = rng.choice([1, 1, 1, 2, 5])
    else:                    # prompts and chunks
        seqs = _log(rng, 1, 6)
        most = 4096 * 16_400 * 32 // (16 if f32 else 1)
        new = _log(rng, 2, min(4096, max(2, int(math.sqrt(most / (seqs * heads))))))
        ctx = _log(rng, new, max(new, min(40_000, most // (seqs * heads * new))))
    block = rng.choice([1, 1, 1, 0, _log(rng, 2, 5000)])
    return _attend("", seqs, new, ctx, heads, kv, dim, dtype, rng.choice([16, 32, 64, 128]), block,
                   -1 if block == 0 else rng.choice([-1, -1, _log(rng, 1, 2000) if block == 1 else 2]),
                   rng.choice([0, 0, _log(rng, 1, 1008)]), rng.random() < 0.7)


def _lengths(case):
    """New tokens and cached keys (the new ones among them) of each sequence: the case says them, not the seed."""
    new, length = [], []
    for b in range(case["seqs"]):
        if case["ragged"]:
            u = (0.55 + 0.6180339887 * b) % 1.0
            n = max(1, int(case["new"] * (1.0 - 0.9 * ((0.31 + 0.4142135623 * b) % 1.0)))) if case["new"] > 1 else 1
            if case["seqs"] >= 4 and b == 2:
                n = 0                                  # a sequence that has nothing new in this step
            length.append(max(n, 1, int(case["ctx"] * (0.03 + 0.97 * u * u))))
        else:
            n = case["new"]
            length.append(max(n, case["ctx"]))
        new.append(n)
    return new, length


def _spans(case):
    """For each new token (numpy, all sequences in order): its sequence, the end of the keys it sees, the start of its
    window and the keys of the anchors that it sees."""
    new, length = _lengths(case)
    seq = np.repeat(np.arange(len(new)), new)
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(new, length)]) if seq.size else np.zeros(0, np.int64)
    m = np.asarray(length)[seq]
    g, w, a = case["block"], case["window"], case["anchors"]
    if g == 0:
        return seq, m, np.zeros_like(pos), np.zeros_like(pos)
    blk = (pos - a) // g
    end = np.minimum(m, (blk + 1) * g + a)
    first = np.maximum(0, (blk - w) * g + a) if w >= 0 else np.zeros_like(pos)
    first = np.minimum(first, end)
    return seq, end, first, np.minimum(np.minimum(a, end), first)


def work(case):
    size = torch.finfo(DTYPES[case["dtype"]]).bits // 8
    if case["op"] != "attend":
        rows = case["tokens"] * (case["heads"] + case["kv_heads"])
        one = rows * case["dim"] * size
        extra = case["tokens"] * case["axes"] * 4
        if case["op"] == "rope_grad":
            return {"bytes": 3 * one + extra, "flops": 20 * rows * case["dim"]}
        moved = 2 * one + (2 * case["tokens"] * case["kv_heads"] * case["dim"] * size if case["append"] else 0)
        return {"bytes": moved + extra, "flops": 9 * rows * case["dim"]}
    new, _ = _lengths(case)
    seq, end, first, anchor = _spans(case)
    pairs = int((end - first + anchor).sum())
    keys = 0
    for b in range(case["seqs"]):
        at = seq == b
        if at.any():
            keys += int(end[at].max() - first[at].min()) + int(min(anchor[at].max(), first[at].min()))
    rows = sum(new) * case["heads"]
    return {"bytes": 2 * rows * case["dim"] * size + 4 * rows + 2 * keys * case["kv_heads"] * case["dim"] * size,
            "flops": 4 * pairs * case["heads"] * case["dim"]}


def _frequencies(case):
    """Radians per position of each rotated pair and its axis; three axes share the pairs as frame : row : column."""
    half = case["rot"] // 2
    counts = [half] if case["axes"] == 1 else [half - 2 * (half // 3), half // 3, half // 3]
    freq = np.concatenate([10000.0 ** (-np.arange(c, dtype=np.float64) / c) for c in counts])
    axis = np.concatenate([np.full(c, a, np.int32) for a, c in enumerate(counts)])
    return torch.from_numpy(freq).cuda(), torch.from_numpy(axis).cuda()


def _randn(gen, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda", dtype=dtype).mul_(scale) if scale != 1.0 else
            torch.randn(*shape, generator=gen, device="cuda", dtype=dtype))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype, H, Hk, d = DTYPES[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]
    if case["op"] != "attend":
        N = case["tokens"]
        s = {"op": case["op"], "interleaved": case["interleaved"], "rot": case["rot"]}
        # the projections come as one matrix [q | k | v] per token
        qkv = _randn(gen, N, (H + 2 * Hk) * d, dtype=dtype)
        s["q"], s["k"] = qkv[:, : H * d].view(N, H, d), qkv[:, H * d: (H + Hk) * d].view(N, Hk, d)
        s["q_weight"] = 1 + _randn(gen, d, dtype=torch.float32, scale=0.1)
        s["k_weight"] = 1 + _randn(gen, d, dtype=torch.float32, scale=0.1)
        s["frequencies"], s["axis"] = _frequencies(case)
        t = torch.arange(N, device="cuda", dtype=torch.int32)
        if case["axes"] == 3:
            u = t % FRAME
            s["positions"] = torch.stack([t // FRAME + case["start"], u // GRID[1], u % GRID[1]], 1).contiguous()
        else:
            s["positions"] = (t + case["start"]).view(N, 1)
        if case["append"]:
            page = case["page"]
            P = -(-N // page) + 3
            s["v"] = qkv[:, (H + Hk) * d:].view(N, Hk, d)
            s["k_cache"] = _randn(gen, P, Hk, page, d, dtype=dtype)
            s["v_cache"] = _randn(gen, P, Hk, page, d, dtype=dtype)
            order = torch.randperm(P, generator=gen, device="cuda")
            at = torch.arange(N, device="cuda") + 5        # the first new token falls into a page in use
            s["slots"] = order[at // page] * page + at % page
            s["stored"] = N - 3 if N > 16 else N           # a padded batch: its last tokens go nowhere
            s["slots"][s["stored"]:] = -1
        if case["op"] == "rope_grad":
            s["dq"], s["dk"] = _randn(gen, N, H, d, dtype=dtype), _randn(gen, N, Hk, d, dtype=dtype)
        return s
    new, length = _lengths(case)
    B, page = case["seqs"], case["page"]
    need = [-(-m // page) for m in length]
    P = sum(need) + 2
    s = {"op": "attend", "block": case["block"], "window": case["window"], "anchors": case["anchors"],
         "max_new": max(new), "max_len": max(length)}
    # keys and queries as the norm and rotation leave them; queries twice as long, for scores that differ
    s["q"] = _randn(gen, sum(new), H, d, dtype=dtype, scale=2.0)
    s["k_cache"] = _randn(gen, P, Hk, page, d, dtype=dtype)
    s["v_cache"] = _randn(gen, P, Hk, page, d, dtype=dtype)
    order = torch.randperm(P, generator=gen, device="cuda").to(torch.int32)
    begin = np.concatenate([[0], np.cumsum(need)])[:-1]
    col = np.arange(max(need))
    where = begin[:, None] + np.minimum(col[None, :], np.asarray(need)[:, None] - 1)
    s["block_table"] = order[torch.from_numpy(where).cuda()].contiguous()
    s["kv_len"] = torch.tensor(length, dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------- one pass
def _turn(x, cos, sin, rot, interleaved):
    """Rotates the pairs of the first `rot` channels of x [N, H, d] by the angles' cos and sin [N, 1, rot / 2]."""
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _angles(s):
    # far positions lose their angle in 32 bits
    phi = (s["positions"].double()[:, s["axis"].long()] * s["frequencies"])[:, None, :]
    return phi.cos().float(), phi.sin().float()


def _plain_rope(s):
    cos, sin = _angles(s)

    def one(x, w):
        f = x.float()
        z = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w
        return _turn(z, cos, sin, s["rot"], s["interleaved"]).to(x.dtype)

    q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
    if "slots" not in s:
        return q, k
    n, page = s["stored"], s["k_cache"].shape[2]
    at = s["slots"][:n]
    s["k_cache"][at // page, :, at % page] = k[:n]
    s["v_cache"][at // page, :, at % page] = s["v"][:n]
    return q, s["k_cache"], s["v_cache"]


def _plain_rope_grad(s):
    cos, sin = _angles(s)

    def one(x, w, dy):
        f = x.float()
        r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
        xh = f * r
        g = _turn(dy.float(), cos, -sin, s["rot"], s["interleaved"])
        gw = g * w
        return (r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(x.dtype), (g * xh).sum((0, 1))

    dq, dwq = one(s["q"], s["q_weight"], s["dq"])
    dk, dwk = one(s["k"], s["k_weight"], s["dk"])
    return dq, dk, dwq, dwk


def _plain_attend(s):
    q, kc, vc, table = s["q"], s["k_cache"], s["v_cache"], s["block_table"].long()
    N, H, d = q.shape
    Hk, page = kc.shape[1], kc.shape[2]
    B, M, L = table.shape[0], s["max_new"], s["max_len"]
    G = H // Hk
    start, length = s["q_start"].long(), s["kv_len"].long()
    count = start[1:] - start[:-1]
    j = torch.arange(L, device=q.device)
    pages, off = table[:, j // page], j % page                                        # [B, L], [L]
    K = kc[pages, :, off[None]].permute(0, 2, 1, 3).float()                           # [B, Hk, L, d]
    V = vc[pages, :, off[None]].permute(0, 2, 1, 3).float()
    V = torch.where((j[None] < length[:, None])[:, None, :, None], V, 0.0)
    i = torch.arange(M, device=q.device)
    row = (start[:-1, None] + i[None]).clamp(max=max(N - 1, 0))                       # [B, M]
    Q = q[row].float().view(B, M, Hk, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * M, d)
    pos = length[:, None] - count[:, None] + i[None]                                  # [B, M]
    seen = (j[None, None] < length[:, None, None]) & (pos >= 0)[..., None]            # [B, M, L]
    g, w, a = s["block"], s["window"], s["anchors"]
    if g > 0:
        blk = torch.div(pos - a, g, rounding_mode="floor")[..., None]
        seen &= j < (blk + 1) * g + a
        if w >= 0:
            seen &= (j >= (blk - w) * g + a) | (j < a)
    x = (Q @ K.transpose(-1, -2)).mul_(d ** -0.5).view(B, Hk, G, M, L)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(B, Hk, G * M, L) @ V).view(B, Hk, G, M, d) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).squeeze(-1)
    # token t of the batch: sequence b, number i
    t = torch.arange(N, device=q.device)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    n = t - start[b]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, M, H, d)[b, n].to(q.dtype)
    return out, lse.permute(0, 3, 1, 2).reshape(B, M, H)[b, n]


def run(s):
    if own:
        from frame_wise_delta_vda_b200 import api
        if s["op"] == "attend":
            return api.vda_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_len"], s["q_start"],
                                           block=s["block"], window_blocks=s["window"], anchors=s["anchors"], return_lse=True)
        how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], positions=s["positions"], frequencies=s["frequencies"],
                   axis=s["axis"], interleaved=s["interleaved"], eps=EPS)
        if s["op"] == "rope_grad":
            return api.vda_qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], **how)
        if "slots" not in s:
            return api.vda_qk_norm_rope(s["q"], s["k"], **how)
        q, _ = api.vda_qk_norm_rope(s["q"], s["k"], v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"], **how)
        return q, s["k_cache"], s["v_cache"]
    if s["op"] == "attend":
        return _plain_attend(s)
    return _plain_rope_grad(s) if s["op"] == "rope_grad" else _plain_rope(s)


# ------------------------------------------------------------------------------------------------- 64 bits
def _exact_rope(case, s):
    d, rot, half = case["dim"], case["rot"], case["rot"] // 2
    phi = s["positions"].double()[:, s["axis"].long()] * s["frequencies"]
    c, n = torch.cos(phi), torch.sin(phi)
    p = torch.arange(half, device=phi.device)
    first, second = (2 * p, 2 * p + 1) if case["interleaved"] else (p, p + half)

    def norm(x):
        x = x.double()
        inv = 1.0 / torch.sqrt((x * x).sum(-1) / d + EPS)
        return x * inv[..., None], inv

    def forward(x, w):
        z = norm(x)[0] * w.double()
        y = z.clone()
        y[..., first] = z[..., first] * c[:, None] - z[..., second] * n[:, None]
        y[..., second] = z[..., second] * c[:, None] + z[..., first] * n[:, None]
        return y

    def backward(x, w, dy):
        u, inv = norm(x)
        dy = dy.double()
        g = dy.clone()
        g[..., first] = dy[..., first] * c[:, None] + dy[..., second] * n[:, None]
        g[..., second] = dy[..., second] * c[:, None] - dy[..., first] * n[:, None]
        dw = torch.einsum("nhd,nhd->d", g, u)
        g *= w.double()
        along = torch.einsum("nhd,nhd->nh", g, u) / d
        return (g - u * along[..., None]) * inv[..., None], dw

    if case["op"] == "rope_grad":
        dq, dwq = backward(s["q"], s["q_weight"], s["dq"])
        dk, dwk = backward(s["k"], s["k_weight"], s["dk"])
        return dq, dk, dwq, dwk
    q, k = forward(s["q"], s["q_weight"]), forward(s["k"], s["k_weight"])
    if not case["append"]:
        return q, k
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    slots = s["slots"].tolist()
    keep = [t for t, at in enumerate(slots) if at >= 0]
    page = torch.tensor([slots[t] // case["page"] for t in keep], device=kc.device)
    off = torch.tensor([slots[t] % case["page"] for t in keep], device=kc.device)
    t = torch.tensor(keep, device=kc.device)
    kc[page, :, off], vc[page, :, off] = k[t], s["v"].double()[t]
    return q, kc, vc


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "attend":
        return _exact_rope(case, s)
    H, Hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    G = H // Hk
    new, length = _lengths(case)
    _, end, first, anchor = (torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in _spans(case))
    out = torch.zeros(sum(new), H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), H), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(new, length)):
        if n == 0:
            continue
        pages = s["block_table"][b, : -(-m // page)].long()
        key = torch.arange(m, device="cuda")[None]
        t = slice(at, at + n)
        hidden = ~((key < end[t, None]) & ((key >= first[t, None]) | (key < anchor[t, None])))
        for h in range(Hk):
            K = s["k_cache"][pages, h].double().reshape(-1, d)[:m]
            V = s["v_cache"][pages, h].double().reshape(-1, d)[:m]
            for h2 in range(h * G, (h + 1) * G):
                x = (s["q"][t, h2].double() @ K.T) / math.sqrt(d)
                x[hidden] = -math.inf
                z = torch.logsumexp(x, -1)
                lse[t, h2] = z
                out[t, h2] = torch.exp(x - z[:, None]) @ V
        at += n
    return out, lse
