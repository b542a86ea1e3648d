"""Measured cases of the operators that a decode step of several continuations of
one prompt uses: attention over a cache whose first tokens a group of sequences
shares, the selection of beams, and the reordering of the cache after it.

``own`` false: the plain form in elementary torch operations.  ``own`` true: the
library's calls.  Both work on the same buffers, whose layout is the cache's
public format:

* ``pages`` uint8 ``[(layers,) n_pages, kv_heads, block]``; a block is K codes, K
  (scale, bias) bf16 pairs ``[page][D/G][2]``, V codes, V pairs.
* codes: per 8 tokens and ``DS = min(D, 128)`` values a slab of words
  ``[SD][r 0..7][i 0..3][u 0..DS/32-1]``; a K word holds token ``r``, values
  ``32u + 8i + 0..7``; a V word holds tokens ``2i`` (low half) and ``2i + 1``,
  values ``32u + r + 8n``, ``n = 0..3``; the lowest nibble comes first.
"""

import math

import torch

own = False

DEV = "cuda"
INF = math.inf


# ------------------------------------------------------------------- cases

def listed():
    at = dict(op="attend", prompts=1, q=1, heads=32, kv_heads=8, dim=128, group=64, page=64, lo=1.0, ragged=False)
    sel = dict(op="select", dtype="bf16", done=True, first=False)
    mv = dict(op="reorder", layers=1, kv_heads=8, dim=128, group=64, page=64, ragged=False)
    return [
        # four beams of one user after the 573-token prompt, a few tokens in: the smallest call
        dict(at, name="attend 4 on 573 + 16", beams=4, prefix=573, tokens=16),
        # a serving batch of beams: 16 prompts of 512 to 2048 tokens, 8 beams each
        dict(at, name="attend 16 x 8 on 2048 + 256", prompts=16, beams=8, prefix=2048, tokens=256, lo=0.25),
        # 64 conversations after one instruction text
        dict(at, name="attend 64 on 8192 + 1024", beams=64, prefix=8192, tokens=1024, lo=0.1),
        # many answers sampled about one long document, five query heads to a key head
        dict(at, name="attend 256 on 32768 + 512", beams=256, prefix=32768, tokens=512, heads=40, lo=0.2),
        # four drafted tokens a sequence, three documents with unlike numbers of readers, small heads, pages of 16
        dict(at, name="attend 3 x 6 x 4 on 16384 + 300", prompts=3, beams=6, prefix=16384, tokens=300, q=4, heads=16, dim=64,
             group=32, page=16, lo=0.5, ragged=True),
        # large heads, 20 samples each of 5 prompts
        dict(at, name="attend 5 x 20 on 5000 + 600", prompts=5, beams=20, prefix=5000, tokens=600, heads=16, kv_heads=4, dim=256,
             lo=0.3),
        # a step of four beams of one user
        dict(sel, name="select 1 x 4 of 32768", prompts=1, beams=4, vocab=32768, k=4),
        # rows of an odd length in 32 bits, the first step (one live beam a prompt), twice as many candidates as beams
        dict(sel, name="select 24 x 5 of 50001", prompts=24, beams=5, vocab=50001, k=10, dtype="fp32", first=True),
        # a large batch
        dict(sel, name="select 64 x 8 of 131072", prompts=64, beams=8, vocab=131072, k=8),
        # four beams of one user, one layer's cache: latency
        dict(mv, name="reorder 1 x 4", prompts=1, beams=4, tokens=100),
        # a batch of beams, 16 layers at once
        dict(mv, name="reorder 16 x 8, 16 layers", prompts=16, beams=8, tokens=190, layers=16),
        # more prompts with small pages of small heads, beams that ended earlier than others
        dict(mv, name="reorder 60 x 5, 7 layers", prompts=60, beams=5, tokens=333, layers=7, kv_heads=4, dim=64, group=32, page=16,
             ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "select", "reorder"])
    dim = rng.choice([64, 128, 128, 256])
    shape = dict(dim=dim, group=rng.choice([g for g in (32, 64, 128) if g <= dim]), page=rng.choice([16, 32, 64, 128]),
                 kv_heads=rng.choice([1, 2, 4, 8]))
    if op == "select":
        vocab, beams = _log(rng, 50, 262144), rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
        prompts = _log(rng, 1, max(1, min(256, 64 * 8 * 131072 // (2 * vocab * beams))))
        return dict(op=op, prompts=prompts, beams=beams, vocab=vocab, k=min(rng.choice([beams, beams, 2 * beams]), 64),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), done=rng.random() < 0.7, first=rng.random() < 0.2)
    if op == "reorder":
        beams, tokens = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 32]), _log(rng, 1, 700)
        per = beams * (tokens // shape["page"] + 2) * shape["page"] * shape["kv_heads"] * dim
        prompts = _log(rng, 1, max(1, min(128, 300_000_000 // per)))
        layers = _log(rng, 1, max(1, min(32, 300_000_000 // (per * prompts))))
        return dict(shape, op=op, prompts=prompts, beams=beams, tokens=tokens, layers=layers, ragged=rng.random() < 0.3)
    kv = shape["kv_heads"]
    heads = kv * rng.choice([1, 2, 4, 5, 6, 8, 16] if kv <= 4 else [1, 2, 4, 5, 8])
    prompts = rng.choice([1, 1, _log(rng, 1, 32)])
    beams = _log(rng, 1, 256 if prompts == 1 else 32)
    prefix, tokens = _log(rng, 1, 32768), rng.choice([_log(rng, 1, 2048), _log(rng, 1, 64)])
    q = rng.choice([1, 1, 1, 2, 4, 7])
    tokens = max(tokens, q)
    while prompts * prefix * kv * dim > 100_000_000 or prompts * beams * q * heads * prefix > 300_000_000:
        prefix, beams = (prefix + 1) // 2, (beams + 1) // 2 if beams > 8 else beams
    while prompts * beams * (tokens + 128) * kv * dim > 130_000_000 and tokens > 2 * q:
        tokens = max(q, (tokens + 1) // 2)
    while prompts * beams * (tokens + 128) * kv * dim > 130_000_000:
        prompts, beams = (prompts + 1) // 2, (beams + 1) // 2
    return dict(shape, op=op, prompts=prompts, beams=beams, prefix=prefix, tokens=tokens, q=q, heads=heads,
                lo=rng.choice([1.0, 0.5, 0.1]), ragged=rng.random() < 0.3)


def _spread(most, count, lo, least=1):
    """`count` numbers between lo * most and most."""
    return [max(least, round(most * (1.0 - (1.0 - lo) * ((0.6180339887 * i) % 1.0)))) for i in range(count)]


def _sizes(case):
    """Sequences of each group, prefix lengths, each sequence's own tokens and query rows."""
    beams = _spread(case["beams"], case["prompts"], 0.3 if case["ragged"] else 1.0)
    prefix = _spread(case["prefix"], case["prompts"], case["lo"])
    tokens = _spread(case["tokens"], sum(beams), case["lo"], case["q"])
    rows = [max(1, case["q"] - (i % 2 if case["ragged"] else 0)) for i in range(sum(beams))]
    return beams, prefix, tokens, rows


def _lens(case):
    """Tokens of each sequence in [prompts][beams]."""
    n = _spread(case["tokens"], case["prompts"], 0.3)
    return [[max(0, t - (3 * b if case["ragged"] else 0)) for b in range(case["beams"])] for t in n]


def work(case):
    if case["op"] == "select":
        n = case["prompts"] * case["beams"] * case["vocab"]
        return dict(bytes=n * (2 if case["dtype"] == "bf16" else 4) + 5 * case["prompts"] * (case["beams"] + 3 * case["k"]), flops=4 * n)
    kv = 2 * (case["dim"] // 2 + 4 * case["dim"] // case["group"]) * case["kv_heads"]
    if case["op"] == "reorder":
        # with parents drawn at random (1 - 1/W)^W of the beams go and as many pages are copied, half a page of tokens each
        seqs, b = case["prompts"] * case["beams"], case["beams"]
        columns = case["tokens"] // case["page"] + 2
        moved = seqs * (1 - 1 / b) ** b * min(case["page"] / 2, case["tokens"])
        return dict(bytes=int(2 * moved * kv * case["layers"]) + seqs * (12 * columns + 12), flops=0)
    beams, prefix, tokens, rows = _sizes(case)
    nbytes, flops, first = 0, 0, 0
    for b, p in zip(beams, prefix):
        nbytes += p * kv + 4 * (-(-p // case["page"])) + 8
        for i in range(first, first + b):
            nbytes += tokens[i] * kv + 4 * rows[i] * case["heads"] * case["dim"] + 4 * (-(-tokens[i] // case["page"])) + 8
            flops += 4 * case["dim"] * case["heads"] * rows[i] * (p + tokens[i] - rows[i] // 2)
        first += b
    return dict(bytes=nbytes, flops=flops)


# ------------------------------------------------------- the cache's format

def _half(case):
    """Bytes of the keys, or of the values, of a page of one head: codes, pairs."""
    return case["page"] * case["dim"] // 2, case["page"] * (case["dim"] // case["group"]) * 4


def _encode(x, group):
    """bf16 [..., D] -> codes uint8 [..., D], (scale, bias) bf16 [..., D/G, 2]; binary32 decisions."""
    g = x.float().unflatten(-1, (-1, group)) + 0.0
    mn, mx = g.amin(-1), g.amax(-1)
    s = ((mx - mn) / 15.0).bfloat16()
    q = ((g - mn[..., None]) / s.float()[..., None]).round().clamp(0, 15)
    q = torch.where(s[..., None] == 0, torch.zeros_like(q), q)
    return q.to(torch.uint8).flatten(-2), torch.stack((s, mn.bfloat16()), -1)


def _pages_of(k, v, live, case):
    """bf16 [P, H, page, D] -> blocks uint8 [P, H, block]; pairs of tokens that are not live are NaN."""
    p, h, page, d = k.shape
    ds = min(d, 128)
    nan = torch.full((1,), float("nan"), dtype=torch.bfloat16, device=DEV)
    out = []
    for name, x in (("k", k), ("v", v)):
        q, pairs = _encode(x, case["group"])
        q = q.view(p, h, page // 8, 8, d // ds, ds // 32, 4, 8)          # slab, r, SD, u, i (n), 0..7 (r)
        if name == "k":
            q = q.permute(0, 1, 2, 4, 3, 6, 5, 7)                        # slab, SD, r, i, u, nibble
        else:
            q = q.unflatten(3, (4, 2)).permute(0, 1, 2, 5, 8, 3, 6, 4, 7)  # slab, SD, r, i, u, parity, n
        q = q.reshape(p, h, -1, 2)
        out += [q[..., 0] | (q[..., 1] << 4), torch.where(live[:, None, :, None, None], pairs, nan).reshape(p, h, -1).view(torch.uint8)]
    return torch.cat(out, -1)


def _held(blocks, case):
    """Blocks uint8 [..., H, block] of consecutive pages -> K, V fp32 [..., H, page, D]."""
    d, page, group = case["dim"], case["page"], case["group"]
    ds = min(d, 128)
    codes, pairs = _half(case)
    k, ks, v, vs = blocks.split([codes, pairs, codes, pairs], -1)
    nib = lambda b: torch.stack((b & 15, b >> 4), -1).flatten(-2)  # noqa: E731
    k = nib(k).unflatten(-1, (page // 8, d // ds, 8, 4, ds // 32, 8))    # slab, SD, r, i, u, 0..7
    k = k.movedim(-4, -5).transpose(-3, -2).flatten(-6, -5).flatten(-4)  # token, values
    v = nib(v).unflatten(-1, (page // 8, d // ds, 8, 4, ds // 32, 2, 4))  # slab, SD, r, i, u, parity, n
    v = v.movedim((-4, -2), (-6, -5)).movedim((-2, -1), (-3, -2)).flatten(-7, -5).flatten(-4)
    scaled = lambda q, p: (p.view(torch.bfloat16).unflatten(-1, (page, d // group, 2)).float()[..., None, :],  # noqa: E731
                           q.unflatten(-1, (-1, group)).float())
    out = []
    for q, p in ((k, ks.contiguous()), (v, vs.contiguous())):
        p, q = scaled(q, p)
        out.append((p[..., 0] * q + p[..., 1]).flatten(-2))
    return out


# ----------------------------------------------------------------- prepare

def _table(gen, lens, page, first, order):
    """Page tables of sequences of these lengths out of order[first:]: int32 [S, widest], -1 where there is none."""
    used = torch.tensor([-(-n // page) for n in lens], device=DEV)
    width = max(1, int(used.max()))
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    total = int(used.sum())
    table[torch.arange(width, device=DEV) < used[:, None]] = order[first:first + total]
    return table, total


def _prepare_attend(case, gen):
    h, d, page = case["kv_heads"], case["dim"], case["page"]
    beams, prefix, tokens, rows = _sizes(case)
    lens = prefix + tokens
    count = sum(-(-n // page) for n in lens)
    order = torch.randperm(count + 3, generator=gen, device=DEV)[:count].int()
    prefix_table, at = _table(gen, prefix, page, 0, order)
    table, _ = _table(gen, tokens, page, at, order)
    # keys as a model has them: some channels much larger than the others
    big = torch.where(torch.rand(d, generator=gen, device=DEV) < 0.06, 4.0, 0.8)
    pages = torch.full((count + 3, h, 2 * sum(_half(case))), 255, dtype=torch.uint8, device=DEV)
    left = torch.cat([torch.arange(-(-n // page), device=DEV) * -page + n for n in lens])  # tokens from this page on
    for i in range(0, count, 4096):
        n = min(4096, count - i)
        k = (torch.randn(n, h, page, d, generator=gen, device=DEV) * big).bfloat16()
        v = torch.randn(n, h, page, d, generator=gen, device=DEV).bfloat16()
        live = torch.arange(page, device=DEV) < left[i:i + n, None]
        pages[order[i:i + n].long()] = _pages_of(k, v, live, case)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    q = torch.randn(sum(rows), case["heads"], d, generator=gen, device=DEV).mul_(1.2).bfloat16()
    even = not case["ragged"]
    return dict(case=case, q=q, pages=pages, prefix_table=prefix_table, prefix_lens=ints(prefix), table=table, lens=ints(tokens),
                groups=None if even else ints([0] + beams).cumsum(0).int(), starts=None if case["q"] == 1 else ints([0] + rows).cumsum(0).int(),
                most=max(rows), most_group=max(beams))


def _prepare_select(case, gen):
    n, w, v = case["prompts"], case["beams"], case["vocab"]
    # a few likely words, the same for the beams of a prompt up to noise
    usual = torch.randn(v, generator=gen, device=DEV).mul_(2.0)
    logits = torch.randn(n * w, v, generator=gen, device=DEV).mul_(1.5).add_(usual)
    logits += 2.5 * torch.randn(n, 1, v, generator=gen, device=DEV).expand(n, w, v).reshape(n * w, v)
    logits = logits.bfloat16() if case["dtype"] == "bf16" else logits
    # some words are not allowed
    logits[:, torch.randint(0, v, (max(1, v // 100),), generator=gen, device=DEV)] = -INF
    scores = -torch.rand(n, w, generator=gen, device=DEV).mul_(8.0).add_(12.0)
    if case["first"]:
        scores[:, 1:], scores[:, 0] = -INF, 0.0
    done = None
    if case["done"]:
        done = torch.rand(n, w, generator=gen, device=DEV) < 0.15
        if case["first"]:
            done[:, 0] = False
    return dict(case=case, logits=logits, scores=scores, done=done, end=v // 3)


def _prepare_reorder(case, gen):
    """A cache some steps after its start: pages of each column of a group in any order, full ones shared."""
    n, w, page = case["prompts"], case["beams"], case["page"]
    lens = torch.tensor(_lens(case), device=DEV)
    columns = case["tokens"] // page + 2
    home = torch.randperm(n * w * columns, generator=gen, device=DEV).int().view(n, w, columns)
    turn = torch.rand(n, w, columns, generator=gen, device=DEV).argsort(1)
    table = home.gather(1, turn)
    full = (torch.arange(columns, device=DEV) + 1) * page <= lens[..., None]
    # a full page may be that of any other full one
    other = torch.where(full[:, None], torch.rand(n, w, w, columns, generator=gen, device=DEV), -1.0).argmax(2)
    table = torch.where(full, table.gather(1, other), table)
    pages = torch.randint(0, 256, (case["layers"], n * w * columns, case["kv_heads"], 2 * sum(_half(case))), generator=gen,
                          dtype=torch.uint8, device=DEV)
    return dict(case=case, pages=pages, home=home.flatten(0, 1), table=table.flatten(0, 1), lens=lens.flatten().int(),
                parents=torch.randint(0, w, (n, w), generator=gen, device=DEV, dtype=torch.int32))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    return {"attend": _prepare_attend, "select": _prepare_select, "reorder": _prepare_reorder}[case["op"]](case, gen)


# --------------------------------------------------------------- plain form

def _tokens(pages, table, case):
    """K, V fp32 [S, H, tokens, D] of the sequences of a page table."""
    k, v = _held(pages[table.clamp(min=0).long()], case)                 # [S, p, H, page, D]
    return k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)


def _part(q, k, v, sees, live, case):
    """Of rows q [B, rows, Hq, D] over k, v [B, H, L, D]: largest score, sum, weighted sum, [B, rows, Hq(, D)].
    sees bool [B, rows, L], live bool [B, L]."""
    rep = case["heads"] // case["kv_heads"]
    b, rows = q.shape[:2]
    qs = q.unflatten(2, (-1, rep)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, H, rows rep, D]
    score = (qs @ k.transpose(-1, -2)).div_(math.sqrt(case["dim"])).unflatten(2, (rows, rep))
    score = score.masked_fill_(~sees[:, None, :, None], -INF)
    m = score.amax(-1)
    w = score.sub_(torch.where(m == -INF, 0.0, m)[..., None]).exp_()
    o = w.flatten(2, 3) @ torch.where(live[:, None, :, None], v, 0.0)
    back = lambda x: x.permute(0, 2, 1, 3, *range(4, x.dim())).flatten(2, 3)  # noqa: E731
    return back(m), back(w.sum(-1)), back(o.unflatten(2, (rows, rep)))


def _plain_attend(st):
    case, q = st["case"], st["q"].float()
    seqs, n = st["lens"].shape[0], st["prefix_lens"].shape[0]
    starts = st["starts"] if st["starts"] is not None else torch.arange(seqs + 1, device=DEV)
    groups = st["groups"] if st["groups"] is not None else torch.arange(n + 1, device=DEV) * (seqs // n)
    starts, groups = starts.long(), groups.long()
    row = torch.arange(q.shape[0], device=DEV)

    def rows_of(first, most):
        """Rows of q in [B, most], and where each row of q is there."""
        b = torch.searchsorted(first, row, right=True) - 1
        return (first[:-1, None] + torch.arange(most, device=DEV)).clamp(max=q.shape[0] - 1), (b, row - first[b])

    # the groups' prefixes, for all rows of a group
    k, v = _tokens(st["pages"], st["prefix_table"], case)
    live = torch.arange(k.shape[2], device=DEV) < st["prefix_lens"][:, None]
    at, place = rows_of(starts[groups], st["most"] * st["most_group"])
    m1, l1, o1 = (x[place] for x in _part(q[at], k, v, live[:, None].expand(-1, at.shape[1], -1), live, case))
    # the sequences' own tokens
    k, v = _tokens(st["pages"], st["table"], case)
    t = torch.arange(k.shape[2], device=DEV)
    live = t < st["lens"][:, None]
    at, place = rows_of(starts, st["most"])
    last = (st["lens"] - (starts[1:] - starts[:-1]))[:, None] + torch.arange(st["most"], device=DEV)
    m2, l2, o2 = (x[place] for x in _part(q[at], k, v, live[:, None] & (t <= last[..., None]), live, case))
    m = torch.maximum(m1, m2)
    m = torch.where(m == -INF, 0.0, m)
    f1, f2 = (m1 - m).exp(), (m2 - m).exp()
    total = l1 * f1 + l2 * f2
    out = (o1 * f1[..., None] + o2 * f2[..., None]) / torch.where(total > 0, total, 1.0)[..., None]
    return out.bfloat16()


def _plain_select(st):
    case, scores = st["case"], st["scores"].double()
    n, w, k = case["prompts"], case["beams"], case["k"]
    x = st["logits"].double().view(n, w, -1)
    top = x.amax(-1, keepdim=True)
    cand = x - top - (x - top).exp().sum(-1, keepdim=True).log() + scores[..., None]
    if st["done"] is not None:
        cand = cand.masked_fill_(st["done"][..., None], -INF)
        cand[..., st["end"]] = torch.where(st["done"], scores, cand[..., st["end"]])
    cand = cand.nan_to_num_(nan=-INF, posinf=INF, neginf=-INF).flatten(1)
    kth = cand.topk(k).values[:, -1:]
    more, level = cand > kth, cand == kth
    chosen = more | (level & (level.cumsum(-1, dtype=torch.int32) <= k - more.sum(-1, keepdim=True)))
    at = chosen.nonzero()[:, 1].view(n, k)                               # the lowest first
    best, order = cand.gather(1, at).sort(dim=-1, descending=True, stable=True)
    at = at.gather(1, order)
    parents, tokens = at // case["vocab"], at % case["vocab"]
    out = best.float(), parents.int(), tokens.int()
    return out if st["done"] is None else out + (st["done"].gather(1, parents) | (tokens == st["end"]),)


def _plain_reorder(st):
    case, page = st["case"], st["case"]["page"]
    n, w = st["parents"].shape
    parents = st["parents"].long()
    home, table = (st[x].view(n, w, -1) for x in ("home", "table"))
    lens = st["lens"].view(n, w).gather(1, parents)
    theirs = table.gather(1, parents[..., None].expand_as(table))
    column = torch.arange(table.shape[2], device=DEV)
    full = (column + 1) * page <= lens[..., None]
    lowest = ~((parents[:, :, None] == parents[:, None, :]).tril(-1).any(-1))
    keeps = full | lowest[..., None]
    # the group's pages of each column that nobody keeps, in order, go to those who keep none
    taken = ((theirs[:, :, None] == home[:, None]) & keeps[:, :, None]).any(1)
    free = taken.to(torch.uint8).sort(dim=1, stable=True).indices
    nth = (~keeps).cumsum(1) - 1
    new = torch.where(keeps, theirs, home.gather(1, free.gather(1, nth.clamp(min=0))))
    # the tokens of the page that is being written, in whole slabs of 8
    part = lens % page
    child = (~lowest & (part > 0)).flatten().nonzero()[:, 0]
    at = (lens // page).flatten()[child]
    src, dst = (x.flatten(0, 1)[child, at].long() for x in (theirs, new))
    slabs = (part.flatten()[child] + 7) // 8 * 8
    codes, pairs = _half(case)
    byte = torch.arange(2 * (codes + pairs), device=DEV) % (codes + pairs)
    token = torch.where(byte < codes, byte * 2 // case["dim"], (byte - codes) * case["group"] // (4 * case["dim"]))
    moves = token < slabs[:, None, None]
    pages = st["pages"]
    pages[:, dst] = torch.where(moves, pages[:, src], pages[:, dst])
    return new.flatten(0, 1), lens.flatten(), pages


def run(state):
    case = state["case"]
    if own:
        import affine_bit_matmul_gb300 as mxq

        if case["op"] == "attend":
            return mxq.kv_attention_shared(state["q"], state["pages"], state["prefix_table"], state["prefix_lens"], state["table"],
                                           state["lens"], state["groups"], state["starts"], max_q_len=state["most"],
                                           max_group=state["most_group"], group_size=case["group"])
        if case["op"] == "select":
            return mxq.beam_select(state["logits"], state["scores"], case["k"], done=state["done"], end_token=state["end"])
        return mxq.kv_reorder(state["pages"], state["table"], state["home"], state["lens"], state["parents"], case["dim"],
                              group_size=case["group"]) + (state["pages"],)
    return {"attend": _plain_attend, "select": _plain_select, "reorder": _plain_reorder}[case["op"]](state)


# ------------------------------------------------------------------- exact

def _exact_places(case):
    """For (token of a page, value): the byte of its K and of its V code in a block, and their shifts."""
    d, page = case["dim"], case["page"]
    t, x = torch.arange(page, device=DEV)[:, None], torch.arange(d, device=DEV)[None]
    ds = min(d, 128)
    u, words = x % ds // 32, ds // 32
    slab = (t // 8 * (d // ds) + x // ds) * 32
    k_word, k_nib = (slab + t % 8 * 4 + x % 32 // 8) * words + u, x % 8
    v_word, v_nib = (slab + x % 8 * 4 + t % 8 // 2) * words + u, t % 2 * 4 + x % 32 // 8
    base = sum(_half(case))
    return k_word * 4 + k_nib // 2, k_nib % 2 * 4, base + v_word * 4 + v_nib // 2, v_nib % 2 * 4


def _exact_values(block, case, places):
    """uint8 [..., block] -> K and V in 64 bits, [..., page, D]."""
    kb, kn, vb, vn = places
    codes, pairs = _half(case)
    out = []
    for where, shift, first in ((kb, kn, codes), (vb, vn, 2 * codes + pairs)):
        code = (block[..., where] >> shift.to(torch.uint8)) & 15
        p = block[..., first:first + pairs].contiguous().view(torch.bfloat16).double()
        p = p.unflatten(-1, (case["page"], -1, 2)).repeat_interleave(case["group"], -2)
        out.append(p[..., 0] * code.double() + p[..., 1])
    return out


def _exact_attend(case, st):
    beams, prefix, tokens, rows = _sizes(case)
    rep, places, out, i, first = case["heads"] // case["kv_heads"], _exact_places(case), [], 0, 0

    def values(table, n, head):
        ids = table[:-(-n // case["page"])].long()
        return (x.flatten(0, 1)[:n] for x in _exact_values(st["pages"][ids, head], case, places))

    for g, count in enumerate(beams):
        r0 = first
        heads = []
        for h in range(case["kv_heads"]):
            kp, vp = values(st["prefix_table"][g], prefix[g], h)
            got, r = [], r0
            for s in range(i, i + count):
                k, v = values(st["table"][s], tokens[s], h)
                k, v = torch.cat((kp, k)), torch.cat((vp, v))
                q = st["q"][r:r + rows[s], h * rep:(h + 1) * rep].double()
                score = torch.einsum("rhd,td->rht", q, k) * case["dim"] ** -0.5
                t = torch.arange(k.shape[0], device=DEV)
                hide = t[None] > (k.shape[0] - rows[s] + torch.arange(rows[s], device=DEV))[:, None]
                score = score.masked_fill(hide[:, None], -INF)
                got.append(torch.softmax(score, -1) @ v)
                r += rows[s]
            first = r
            heads.append(torch.cat(got))
        i += count
        out.append(torch.cat(heads, 1))
    return torch.cat(out)


def _exact_select(case, st):
    n, w, v = case["prompts"], case["beams"], case["vocab"]
    best, parents, tokens = [], [], []
    for g in range(n):
        cand = torch.log_softmax(st["logits"][g * w:(g + 1) * w].double(), -1) + st["scores"][g].double()[:, None]
        for b in range(w):
            if st["done"] is not None and st["done"][g, b]:
                cand[b] = -INF
                cand[b, st["end"]] = st["scores"][g, b]
        x, at = torch.sort(cand.nan_to_num(nan=-INF, neginf=-INF).flatten(), descending=True, stable=True)
        best.append(x[:case["k"]])
        parents.append(at[:case["k"]] // v)
        tokens.append(at[:case["k"]] % v)
    best, parents, tokens = torch.stack(best), torch.stack(parents).int(), torch.stack(tokens).int()
    if st["done"] is None:
        return best, parents, tokens
    ended = torch.stack([st["done"][g][parents[g].long()] for g in range(n)])
    return best, parents, tokens, ended | (tokens == st["end"])


def exact(case, seed):
    if case["op"] == "reorder":
        return None  # nothing is computed
    st = prepare(case, seed)
    return _exact_attend(case, st) if case["op"] == "attend" else _exact_select(case, st)
