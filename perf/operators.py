"""Measured cases of the operators between a transformer layer's projections:
the norm and rotation of queries and keys, the writing and reading of a paged
4-bit key/value cache, and the attention over that cache.

``own`` false: the plain form in elementary torch operations, in 32 bits.
``own`` true: the library's calls.  Both work on the same buffers, whose
layout is the cache's public format:

* ``pages`` uint8 ``[n_pages, kv_heads, block]``; a block is K codes, K
  (scale, bias) bf16 pairs ``[page][D/G][2]``, V codes, V pairs.
* codes: per 8 tokens and ``DS = min(D, 128)`` values a slab of words
  ``[SD][r 0..7][i 0..3][u 0..DS/32-1]``; a K word holds token ``r``, values
  ``32u + 8i + 0..7``; a V word holds tokens ``2i`` (low half) and ``2i + 1``,
  values ``32u + r + 8n``, ``n = 0..3``; the lowest nibble comes first.
* slot = page * page_size + offset.
"""

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases

def listed():
    rot = dict(op="rotate", dim=128, rot=128, interleaved=False, norm=True)
    wr = dict(op="append", dim=128, group=64, page=64, kv_heads=8)
    at = dict(op="attend", q=1, heads=32, kv_heads=8, dim=128, group=64, page=64, window=0, sinks=0, lo=1.0)
    return [
        # a decode step of 16 sequences: latency
        dict(rot, name="rotate 16 tokens", tokens=16, heads=32, kv_heads=8),
        # the q and k rows of a packed prompt batch of the routed workload's size, half of each head rotated
        dict(rot, name="rotate 4584 tokens", tokens=4584, heads=40, kv_heads=8, rot=64, interleaved=True),
        # the new rows of a decode step of 64 sequences
        dict(wr, name="append 64 tokens", tokens=64),
        # packed prompts going into the cache
        dict(wr, name="append 8192 tokens", tokens=8192),
        # one prompt's prefix read back out of small pages of small heads
        dict(wr, op="read", name="read 573 tokens", tokens=573, dim=64, group=32, page=16),
        # a long prefix read back
        dict(wr, op="read", name="read 32768 tokens", tokens=32768),
        # one user, one new token, after the 573-token prompt: the smallest call
        dict(at, name="attend 1 x 573", seqs=1, ctx=573),
        # a serving batch of ragged contexts
        dict(at, name="attend 64 x 8192", seqs=64, ctx=8192, lo=0.125),
        # long contexts, five query heads to a key head
        dict(at, name="attend 8 x 131072", seqs=8, ctx=131072, heads=40, lo=0.5),
        # a sliding-window layer with first tokens kept, four drafted tokens a sequence, pages of 16
        dict(at, name="attend 32 x 4 windowed", seqs=32, ctx=32768, q=4, page=16, window=1024, sinks=4, lo=0.05),
        # a chunk of a long prompt after what is cached already
        dict(at, name="prefill 2048 of 8192", seqs=1, ctx=8192, q=2048),
        # several prompts of about 600 tokens at once, large heads, none cached before
        dict(at, name="prefill 8 x 600", seqs=8, ctx=600, q=600, heads=16, kv_heads=4, dim=256, lo=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "read", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "rotate":
        heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
        rot = rng.choice([dim, dim // 2, dim // 4])
        tokens = _log(rng, 1, max(1, 4584 * 48 * 128 // ((heads + kv_heads) * dim)) if (heads + kv_heads) * dim > 6144 else 4584)
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.75)
    if op in ("append", "read"):
        most = 8192 if op == "append" else 32768
        tokens = _log(rng, 1, most * 128 // max(128, dim))
        return dict(op=op, tokens=tokens, dim=dim, group=group, page=page, kv_heads=kv_heads)
    heads = kv_heads * rng.choice([1, 2, 4, 5, 6, 8, 16] if kv_heads <= 4 else [1, 2, 4, 5, 8])
    kind = rng.choice(["one", "one", "few", "chunk"])
    if kind == "chunk":
        seqs = _log(rng, 1, 12)
        q = _log(rng, 9, 2048)
        ctx = q + rng.choice([0, _log(rng, 1, 16384)])
        most = 2048 * 8192 * 32 * 128
        while seqs * q * ctx * heads * dim > most // 2:
            q, ctx = (q + 1) // 2, (ctx + 1) // 2
    else:
        seqs = _log(rng, 1, 128)
        q = 1 if kind == "one" else rng.randint(2, 8)
        ctx = max(q, _log(rng, 1, 131072))
        most = 8 * 131072 * 8 * 128 // 2
        while seqs * ctx * kv_heads * dim > most:
            seqs, ctx = (seqs + 1) // 2, max(q, (ctx + 1) // 2)
    window = _log(rng, 16, 4096) if rng.random() < 0.35 else 0
    return dict(op=op, seqs=seqs, ctx=ctx, q=q, heads=heads, kv_heads=kv_heads, dim=dim, group=group, page=page,
                window=window, sinks=rng.randint(0, 8) if window else 0, lo=rng.choice([1.0, 0.5, 0.1]))


def _lengths(case):
    """Context lengths and query rows of the sequences: spread between lo * the most and the most."""
    ctx, rows = [], []
    for i in range(case["seqs"]):
        f = (0.6180339887 * i) % 1.0
        n = max(1, round(case["ctx"] * (1.0 - (1.0 - case["lo"]) * f)))
        chunk = case["q"] > 8
        r = case["q"] if not chunk else max(1, round(case["q"] * (1.0 - (1.0 - case["lo"]) * f)))
        n = max(n, r)
        ctx.append(n)
        rows.append(r)
    return ctx, rows


def _visible(n, rows, window, sinks):
    """Visible (query, key) pairs of one sequence, and the distinct keys that any of its rows sees."""
    pairs = 0
    for j in range(rows):
        p = n - rows + j
        w = p + 1 if not window else min(p + 1, window)
        pairs += w + (min(sinks, p + 1 - w) if window else 0)
    first = n - rows
    lo = max(0, first - window + 1) if window else 0
    return pairs, n - lo + min(sinks, lo)


def work(case):
    if case["op"] == "rotate":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return dict(bytes=4 * n + 4 * case["tokens"] + 2 * case["rot"] + (4 * case["dim"] if case["norm"] else 0),
                    flops=(7 if case["norm"] else 0) * n + 3 * n * case["rot"] // case["dim"])
    kv = 2 * (case["dim"] // 2 + 4 * case["dim"] // case["group"]) * case["kv_heads"]
    if case["op"] in ("append", "read"):
        t, full = case["tokens"], 2 * case["kv_heads"] * case["dim"]
        if case["op"] == "read":
            return dict(bytes=t * (kv + 2 * full + 4), flops=2 * t * full)
        # new rows in, codes out; then the same rows out of the cache and as bf16
        return dict(bytes=t * (2 * full + kv + 4) + t * (kv + 2 * full + 4), flops=8 * t * full)
    nbytes = flops = 0
    for n, r in zip(*_lengths(case)):
        pairs, keys = _visible(n, r, case["window"], case["sinks"])
        nbytes += keys * kv + 4 * r * case["heads"] * case["dim"] + 4 * (-(-n // case["page"])) + 8
        flops += 4 * case["dim"] * case["heads"] * pairs
    return dict(bytes=nbytes, flops=flops)


# ------------------------------------------------------- the cache's format

def _encode(x, group):
    """bf16 [..., D] -> codes uint8 [..., D], scale and bias bf16 [..., D/G]; binary32 decisions."""
    g = x.float().unflatten(-1, (-1, group)) + 0.0
    mn, mx = g.amin(-1), g.amax(-1)
    s, b = ((mx - mn) / 15.0).bfloat16(), mn.bfloat16()
    q = ((g - b.float()[..., None]) / s.float()[..., None]).round().clamp(0, 15)
    q = torch.where(s[..., None] == 0, torch.zeros_like(q), q)
    return q.to(torch.uint8).flatten(-2), s, b


def _shapes(dim, group, page):
    ds = min(dim, 128)
    codes, pairs = page * dim // 2, page * (dim // group) * 4
    return ds, dim // ds, ds // 32, codes, pairs


def _regions(pages, dim, group, page):
    """Views of the four parts of every block: K bytes [P, H, n8, SD, r, i, u, 4], K pairs bf16 [P, H, page, D/G, 2],
    V bytes [P, H, n8, SD, r, i, u, 2, 2] (the last two: token parity, byte), V pairs."""
    ds, sd, u, codes, pairs = _shapes(dim, group, page)
    k, ks, v, vs = pages.split([codes, pairs, codes, pairs], -1)
    n8 = page // 8
    pair = lambda t: t.view(torch.bfloat16).unflatten(-1, (page, dim // group, 2))  # noqa: E731
    return (k.unflatten(-1, (n8, sd, 8, 4, u, 4)), pair(ks), v.unflatten(-1, (n8, sd, 8, 4, u, 2, 2)), pair(vs))


def _nibbles(b):
    """uint8 [..., n] -> codes uint8 [..., 2n], the low nibble first."""
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _bytes(q):
    return q[..., 0::2] | (q[..., 1::2] << 4)


def _k_rows(q, dim):
    """Codes [..., D] -> the bytes of a token's K rows [..., SD, i, u, 4]."""
    ds, sd, u, _, _ = _shapes(dim, dim, 8)
    q = q.unflatten(-1, (sd, u, 4, 8))
    return _bytes(q.transpose(-3, -2))


def _v_rows(q, dim):
    """Codes [..., D] -> the bytes of a token's V rows [..., SD, r, u, 2]."""
    ds, sd, u, _, _ = _shapes(dim, dim, 8)
    q = q.unflatten(-1, (sd, u, 4, 8))       # sd, u, n, r
    return _bytes(q.movedim(-1, -3))         # sd, r, u, n


def _k_codes(b):
    """The inverse of _k_rows."""
    return _nibbles(b).transpose(-3, -2).flatten(-4)


def _v_codes(b):
    return _nibbles(b).movedim(-3, -1).flatten(-4)


def _values(codes, pairs, group):
    """fp32 s * q + b."""
    g = codes.unflatten(-1, (-1, group)).float()
    return (pairs[..., :1].float() * g + pairs[..., 1:].float()).flatten(-2)


def _write(pages, slots, k, v, group, page):
    dim = k.shape[-1]
    kb, ks, vb, vs = _regions(pages, dim, group, page)
    at, o = slots.long() // page, slots.long() % page
    q, s, b = _encode(k, group)
    kb[at, :, o // 8, :, o % 8] = _k_rows(q, dim)
    ks[at, :, o] = torch.stack((s, b), -1)
    q, s, b = _encode(v, group)
    vb[at, :, o // 8, :, :, o % 8 // 2, :, o % 2] = _v_rows(q, dim)
    vs[at, :, o] = torch.stack((s, b), -1)


def _read(pages, slots, dim, group, page):
    kb, ks, vb, vs = _regions(pages, dim, group, page)
    at, o = slots.long() // page, slots.long() % page
    k = _values(_k_codes(kb[at, :, o // 8, :, o % 8]), ks[at, :, o], group)
    v = _values(_v_codes(vb[at, :, o // 8, :, :, o % 8 // 2, :, o % 2]), vs[at, :, o], group)
    return k, v


# ----------------------------------------------------------------- prepare

def _keys(gen, shape):
    """Keys as a model has them: some channels much larger than the others."""
    k = torch.randn(shape, generator=gen, device=DEV)
    big = torch.rand(shape[-1], generator=gen, device=DEV) < 0.06
    return (k * torch.where(big, 4.0, 0.8)).bfloat16()


def _prepare_rotate(case, gen):
    t, d = case["tokens"], case["dim"]
    # q, k and v of one fused projection's output: rows with a stride
    width = case["heads"] + 2 * case["kv_heads"]
    qkv = torch.randn(t, width, d, generator=gen, device=DEV).mul_(3.0).bfloat16()
    first = torch.randint(0, 100000, (1,), generator=gen, device=DEV)
    pos = (torch.arange(t, device=DEV) + first).int() if t > 64 else torch.randint(
        0, 131072, (t,), generator=gen, device=DEV, dtype=torch.int32)
    j = torch.arange(case["rot"] // 2, device=DEV, dtype=torch.float64)
    state = dict(case=case, q=qkv[:, :case["heads"]], k=qkv[:, case["heads"]:case["heads"] + case["kv_heads"]],
                 positions=pos, inv_freq=(1e6 ** (-2.0 * j / case["rot"])).float(), qw=None, kw=None)
    if case["norm"]:
        state["qw"] = (1 + 0.3 * torch.randn(d, generator=gen, device=DEV)).bfloat16()
        state["kw"] = (1 + 0.3 * torch.randn(d, generator=gen, device=DEV)).bfloat16()
    return state


def _prepare_cache(case, gen):
    """A cache that already held something, new rows and their slots (a sequence's tokens in order in shuffled pages)."""
    t, h, d, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    n_pages = -(-t // page) + 2
    slots = torch.randperm(n_pages, generator=gen, device=DEV)[:, None] * page + torch.arange(page, device=DEV)
    slots = slots.flatten()[page // 3:page // 3 + t].int()
    pages = torch.zeros(n_pages, h, 2 * (page * d // 2 + page * (d // case["group"]) * 4), dtype=torch.uint8, device=DEV)
    state = dict(case=case, pages=pages, slots=slots, k=_keys(gen, (t, h, d)),
                 v=torch.randn(t, h, d, generator=gen, device=DEV).bfloat16())
    if case["op"] == "read":
        _write(pages, slots, state["k"], state["v"], case["group"], page)
    return state


def _prepare_attend(case, gen):
    h, d, page, group = case["kv_heads"], case["dim"], case["page"], case["group"]
    ctx, rows = _lengths(case)
    used = [-(-n // page) for n in ctx]
    total = sum(used)
    n_pages, width = total + 3, max(used)
    order = torch.randperm(n_pages, generator=gen, device=DEV)[:total].int()
    table = torch.full((len(ctx), width), -1, dtype=torch.int32, device=DEV)
    lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    used = torch.tensor(used, device=DEV)
    table[torch.arange(width, device=DEV)[None] < used[:, None]] = order
    # what was never written holds whatever the memory held: here NaN scales
    pages = torch.full((n_pages, h, 2 * (page * d // 2 + page * (d // group) * 4)), 255, dtype=torch.uint8, device=DEV)
    kb, ks, vb, vs = _regions(pages, d, group, page)
    seq = torch.repeat_interleave(torch.arange(len(ctx), device=DEV), used)
    nth = torch.arange(total, device=DEV) - (used.cumsum(0) - used)[seq]
    live = (nth[:, None] * page + torch.arange(page, device=DEV) < lens[seq][:, None])[:, None, :, None, None]
    nan = torch.full((1,), float("nan"), dtype=torch.bfloat16, device=DEV)
    # both are encoded in their pages' order, tokens beside heads
    for codes, pairs, made, x in ((kb, ks, "k", _keys(gen, (total, h, page, d))),
                                  (vb, vs, "v", torch.randn(total, h, page, d, generator=gen, device=DEV).bfloat16())):
        q, s, b = _encode(x, group)
        if made == "k":
            codes[order.long()] = _k_rows(q, d).unflatten(2, (page // 8, 8)).movedim(3, 4)
        else:
            codes[order.long()] = _v_rows(q, d).unflatten(2, (page // 8, 4, 2)).permute(0, 1, 2, 5, 6, 3, 7, 4, 8)
        pairs[order.long()] = torch.where(live, torch.stack((s, b), -1), nan)
        del q, s, b
    t = sum(rows)
    q = torch.randn(t, case["heads"], d, generator=gen, device=DEV).mul_(1.2).bfloat16()
    starts = None if case["q"] == 1 else torch.tensor([0] + rows, dtype=torch.int32, device=DEV).cumsum(0).int()
    return dict(case=case, q=q, pages=pages, table=table, lens=lens, starts=starts, most=max(rows))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    if case["op"] == "rotate":
        return _prepare_rotate(case, gen)
    return _prepare_attend(case, gen) if case["op"] == "attend" else _prepare_cache(case, gen)


# --------------------------------------------------------------- plain form

def _plain_rotate(x, weight, angle, case):
    n = x.float()
    if weight is not None:
        n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + 1e-6) * weight.float()
    rot = case["rot"]
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    if case["interleaved"]:
        a, b = n[..., 0:rot:2], n[..., 1:rot:2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = n[..., :rot // 2], n[..., rot // 2:rot]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((r, n[..., rot:]), -1).bfloat16()


def _plain_attend(st):
    case, q, lens = st["case"], st["q"], st["lens"]
    h, d, page, group = case["kv_heads"], case["dim"], case["page"], case["group"]
    seqs, most, rep = lens.shape[0], st["most"], case["heads"] // case["kv_heads"]
    held = st["pages"][st["table"].clamp(min=0).long()]                      # [S, p, H, block]
    kb, ks, vb, vs = _regions(held.flatten(0, 1), d, group, page)
    k = _values(_k_codes(kb.movedim(3, 4)).flatten(2, 3), ks, group)         # [S p, H, page, D]
    v = _values(_v_codes(vb.permute(0, 1, 2, 5, 7, 3, 4, 6, 8)).flatten(2, 4), vs, group)
    k, v = (x.unflatten(0, (seqs, -1)).transpose(1, 2).flatten(2, 3) for x in (k, v))  # [S, H, L, D]
    starts = st["starts"] if st["starts"] is not None else torch.arange(seqs + 1, device=q.device)
    rows = (starts[1:] - starts[:-1]).long()
    j = torch.arange(most, device=q.device)
    at = (starts[:-1, None].long() + j).clamp(max=q.shape[0] - 1)
    qs = q[at].float().unflatten(2, (h, rep)).permute(0, 2, 3, 1, 4)         # [S, H, rep, most, D]
    score = (qs.flatten(2, 3) @ k.transpose(-1, -2)) / math.sqrt(d)
    t = torch.arange(k.shape[2], device=q.device)
    p = (lens[:, None].long() - rows[:, None] + j)[..., None]                # [S, most, 1]
    sees = (t <= p) & (t < lens[:, None, None])
    if case["window"]:
        sees &= (t > p - case["window"]) | (t < case["sinks"])
    score = score.unflatten(2, (rep, most)).masked_fill(~sees[:, None, None], -math.inf)
    m = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(m == -math.inf, 0.0, m))
    v = torch.where((t < lens[:, None])[:, None, :, None], v, 0.0)
    o = w.flatten(2, 3) @ v
    total = w.sum(-1).flatten(2, 3)[..., None]
    o = torch.where(total > 0, o / total, 0.0).unflatten(2, (rep, most))     # [S, H, rep, most, D]
    row = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(starts.long(), row, right=True) - 1
    return o.permute(0, 3, 1, 2, 4)[seq, row - starts.long()[seq]].flatten(1, 2).bfloat16()


def run(state):
    case = state["case"]
    if case["op"] == "rotate":
        if own:
            import affine_bit_matmul_gb300 as mxq

            return mxq.qk_norm_rope(state["q"], state["k"], state["positions"], state["inv_freq"], state["qw"],
                                    state["kw"], interleaved=case["interleaved"])
        angle = state["positions"].float()[:, None] * state["inv_freq"]
        return tuple(_plain_rotate(x, w, angle, case) for x, w in ((state["q"], state["qw"]), (state["k"], state["kw"])))
    if case["op"] in ("append", "read"):
        pages, slots, dim, group = state["pages"], state["slots"], case["dim"], case["group"]
        if own:
            import affine_bit_matmul_gb300 as mxq

            if case["op"] == "append":
                mxq.kv_append(state["k"], state["v"], pages, slots, group_size=group)
            return mxq.kv_read(pages, slots, dim, group_size=group)
        if case["op"] == "append":
            _write(pages, slots, state["k"], state["v"], group, case["page"])
        return tuple(x.bfloat16() for x in _read(pages, slots, dim, group, case["page"]))
    if own:
        import affine_bit_matmul_gb300 as mxq

        return mxq.kv_attention(state["q"], state["pages"], state["table"], state["lens"], state["starts"],
                                max_q_len=state["most"], group_size=case["group"], window=case["window"],
                                sinks=case["sinks"])
    return _plain_attend(state)


# ------------------------------------------------------------------- exact

def _exact_rotate(x, weight, case, st):
    n = x.double()
    if weight is not None:
        n = n / torch.sqrt(n.pow(2).mean(-1, keepdim=True) + 1e-6) * weight.double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       st["positions"].double()[:, None, None] * st["inv_freq"].double())
    j = torch.arange(case["rot"] // 2, device=DEV)
    i1, i2 = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + case["rot"] // 2)
    z = torch.complex(n[..., i1], n[..., i2]) * turn
    out = n.clone()
    out[..., i1], out[..., i2] = z.real, z.imag
    return out


def _exact_places(case):
    """For (offset in page, value): the byte of its K and of its V code in a block, and their shifts."""
    d, page = case["dim"], case["page"]
    t = torch.arange(page, device=DEV)[:, None]
    x = torch.arange(d, device=DEV)[None]
    ds = min(d, 128)
    u, words = x % ds // 32, ds // 32
    slab = (t // 8 * (d // ds) + x // ds) * 32
    k_word, k_nib = (slab + t % 8 * 4 + x % 32 // 8) * words + u, x % 8
    v_word, v_nib = (slab + x % 8 * 4 + t % 8 // 2) * words + u, t % 2 * 4 + x % 32 // 8
    base = page * d // 2 + page * (d // case["group"]) * 4
    return k_word * 4 + k_nib // 2, k_nib % 2 * 4, base + v_word * 4 + v_nib // 2, v_nib % 2 * 4


def _exact_values(block, case):
    """uint8 [..., block] -> K and V in 64 bits, [..., page, D]."""
    d, page, group = case["dim"], case["page"], case["group"]
    kb, kn, vb, vn = _exact_places(case)
    half = page * d // 2
    out = []
    for where, shift, first in ((kb, kn, half), (vb, vn, block.shape[-1] - page * (d // group) * 4)):
        code = (block[..., where] >> shift.to(torch.uint8)) & 15
        p = block[..., first:first + page * (d // group) * 4].contiguous().view(torch.bfloat16).double()
        p = p.unflatten(-1, (page, d // group, 2)).repeat_interleave(group, -2)
        out.append(p[..., 0] * code.double() + p[..., 1])
    return out


def _exact_stored(x, group):
    """The values a bf16 tensor has once it is held in 4 bits: the format's binary32 decisions, each as one rounding
    of an operation in 64 bits."""
    r = lambda y: y.float().double()  # noqa: E731
    g = x.double().unflatten(-1, (-1, group))
    lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
    s = (r(r(hi - lo) / 15)).bfloat16().double()
    q = torch.clamp(torch.round(r(r(g - lo) / torch.where(s == 0, 1.0, s))), 0, 15) * (s != 0)
    return (s * q + lo).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(st["q"], st["qw"], case, st), _exact_rotate(st["k"], st["kw"], case, st)
    if case["op"] in ("append", "read"):
        return _exact_stored(st["k"], case["group"]), _exact_stored(st["v"], case["group"])
    ctx, rows = _lengths(case)
    rep, out, first = case["heads"] // case["kv_heads"], [], 0
    for i, (n, r) in enumerate(zip(ctx, rows)):
        ids = st["table"][i, :-(-n // case["page"])].long()
        q = st["q"][first:first + r].double().transpose(0, 1)
        first += r
        t = torch.arange(n, device=DEV)
        p = torch.arange(n - r, n, device=DEV)[:, None]
        hide = t > p
        if case["window"]:
            hide |= (p - t >= case["window"]) & (t >= case["sinks"])
        heads = []
        for h in range(case["kv_heads"]):
            k, v = (x.flatten(0, 1)[:n] for x in _exact_values(st["pages"][ids, h], case))
            s = (q[h * rep:(h + 1) * rep] @ k.T) * case["dim"] ** -0.5
            s[:, hide] = -math.inf
            heads.append(torch.softmax(s, -1) @ v)
        out.append(torch.cat(heads).transpose(0, 1))
    return torch.cat(out)
