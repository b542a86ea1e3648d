"""How near the attention of few rows comes to float64: element by element at short lengths,
and in the 2-norm at lengths where one warp adds tens of thousands of tokens."""

import numpy as np
import pytest

from tests.test_gpu_kv_attention import LENS, Case
from tests.test_gpu_kv_cache import SHAPES, i32

pytestmark = pytest.mark.gpu


def value_pairs(cache):
    """Scale and bias of the values, float64 [slots, H, D] each."""
    D, G, page = cache.D, cache.group, cache.page
    first = cache.bytes.shape[-1] // 2 + page * D // 2
    p = cache.bytes[:, :, first:first + page * (D // G) * 4].copy().view(np.uint16)
    p = (p.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    p = p.reshape(cache.n_pages, cache.H, page, D // G, 2).transpose(0, 2, 1, 3, 4).reshape(-1, cache.H, D // G, 2)
    return np.repeat(p[..., 0], G, -1), np.repeat(p[..., 1], G, -1)


def few_rows(q, cache, table, ctx, starts):
    """float64 out [T, Hq, D], and what it may be off by in each element.

    The kernel multiplies codes 0..15 by weights times scales rounded to f16 and adds the
    biases apart, in fp32.  With P the weights, out = sum P s q + sum P b:
    * the output is rounded to bf16, 8 bits: 2^-8 of it at most;
    * P s has 11 bits, each off by 2^-11 of itself at most: 2^-11 C, C = sum P s q; below
      2^-14 of f16 (2^-20 of the largest scale) by half of 2^-24 of it: 2^-31 max(s) for each token,
      times codes of at most 15: n 2^-27 max(s);
    * the instructions add 16 products at a time, towards zero, to what is at most the sum of 512
      tokens: 2^-15 C; the biases' sums and the joined ones, to nearest: 2^-17 (C + sum P |b|);
    * scores of up to 256 products in steps of 16 from zero, likewise, off by
      2^-17 F, F = scale sum |q_d| (s c_d + |b|) at most, and the exponentials of them,
      2^-21 (1 + |S|): weights off by a factor 1 + e, their sum too: 2 e sum P |v|."""
    T, Hq, D = q.shape
    rep, scale = Hq // cache.H, D ** -0.5
    vs, vb = value_pairs(cache)
    out, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    q = q.astype(np.float64)
    for i, n in enumerate(ctx):
        a, b = starts[i], starts[i + 1]
        for row in range(a, b):
            t = np.arange(max(0, n - (b - a) + row - a + 1))
            if not len(t):
                continue
            at = table[i][t // cache.page].astype(np.int64) * cache.page + t % cache.page
            for h in range(Hq):
                k, v, s, bias = cache.k[at, h // rep], cache.v[at, h // rep], vs[at, h // rep], vb[at, h // rep]
                score = scale * (k @ q[row, h])
                # the keys' s c_d + |b| is at most |k| + 2 |b|, and their |b| at most max |k| of the row
                F = scale * ((np.abs(k) + 2 * np.abs(k).max(-1, keepdims=True)) @ np.abs(q[row, h])).max()
                w = np.exp(score - score.max())
                w /= w.sum()
                out[row, h] = w @ v
                C = w @ (v - bias)
                e = 2.0 ** -17 * F + 2.0 ** -21 * (1 + np.abs(score).max())
                tol[row, h] = (2.0 ** -8 * np.abs(out[row, h]) + 2.0 ** -11 * C + 2.0 ** -15 * C +
                               2.0 ** -17 * (C + w @ np.abs(bias)) + 2 * e * (w @ np.abs(v)) +
                               len(t) * 2.0 ** -27 * s.max()) * (1 + 2.0 ** -8) + 1e-30
    return out, tol


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("heads,rows", [(4, 1), (3, 2), (12, 1), (4, 4)])
def test_every_element_of_few_rows(D, G, heads, rows):
    ctx = LENS + [1500]
    c = Case(ctx, [rows] * len(ctx), heads, 1, D, G, 64, seed=3 * D + G + heads + rows)
    o, _, status = c.run()
    assert status == 0
    ref, tol = few_rows(c.q, c.cache, c.table, c.ctx, c.starts)
    err = np.abs(o - ref)
    assert (err <= tol).all(), "worst err/tol %.3g" % (err / tol).max()


# 2-norm of the error over that of the result, of values around zero: the rounding to bf16 1.66e-3;
# weights with 11 bits, 1.9e-4 of themselves on average, on codes that are, times their
# scale, about 2.6 times the values: 5e-4; sums towards zero of at most 512 tokens, of whose products the biases
# then take most away: 3e-4.  Together 1.76e-3.
MOST = 1.9e-3


@pytest.mark.parametrize("seqs,heads,D,G", [
    (8, 40, 128, 64),    # cut finely: a row tile is shared by some five blocks
    (40, 32, 128, 64), (40, 64, 128, 32), (40, 128, 128, 128),  # a block has whole row tiles, of 4, 8 and 16 rows
    (40, 32, 64, 32), (40, 128, 64, 64), (40, 32, 256, 64), (40, 64, 256, 128), (40, 128, 256, 32)])
def test_long_contexts_are_as_good_as_the_output_type(seqs, heads, D, G):
    import torch

    import affine_bit_matmul_gb300 as mxq

    n, H, page = 131072, 8, 64
    gen = torch.Generator(device="cuda").manual_seed(D + G + seqs)
    loud = torch.where(torch.rand(D, generator=gen, device="cuda") < 0.06, 4.0, 0.8)
    k = (torch.randn((n, H, D), generator=gen, device="cuda") * loud).bfloat16()
    v = torch.randn((n, H, D), generator=gen, device="cuda").bfloat16()
    order = torch.randperm(n // page, generator=gen, device="cuda").int()
    t = torch.arange(n, device="cuda")
    pages = torch.zeros((n // page, H, mxq.kv_block_bytes(D, page, G)), dtype=torch.uint8, device="cuda")
    mxq.kv_append(k, v, pages, order[t // page] * page + (t % page).int(), group_size=G)
    # every sequence has these pages; the lengths differ a little
    table = order[None].expand(seqs, -1).contiguous()
    lens = [n - 7 * i for i in range(seqs)]
    q = (torch.randn((seqs, heads, D), generator=gen, device="cuda") * 1.2).bfloat16()
    o = mxq.kv_attention(q, pages, table, i32(lens), group_size=G).double()

    def held(x):  # what the cache makes of the values, in float64
        g = x.float().unflatten(-1, (-1, G)) + 0.0
        b = g.amin(-1, keepdim=True)
        s = ((g.amax(-1, keepdim=True) - b) / 15.0).bfloat16().float()
        c = ((g - b) / s).round().clamp(0, 15)
        return (s.double() * c.double() + b.double()).flatten(-2)

    rep = heads // H
    some = list(range(0, seqs, 3))
    off = norm = 0.0
    for h in range(H):
        kk, vv = held(k[:, h]), held(v[:, h])
        for i in some:
            qq = q[i, h * rep:(h + 1) * rep].double()
            w = torch.softmax((qq @ kk[:lens[i]].T) * D ** -0.5, -1)
            ref = w @ vv[:lens[i]]
            off += float((o[i, h * rep:(h + 1) * rep] - ref).pow(2).sum())
            norm += float(ref.pow(2).sum())
    assert (off / norm) ** 0.5 <= MOST, "%.3e of the norm" % (off / norm) ** 0.5


def test_rows_of_sequences_beside_one_whose_rows_decrease():
    import affine_bit_matmul_gb300 as mxq

    c = Case([100, 60, 30], [3, 2, 4], 4, 2, 128, 64, 16, seed=13)
    c.starts_d[1], c.starts_d[2] = 5, 3   # sequence 0 has 5 rows, 1 has -2, 2 has 6: rows 3 and 4 are of both
    o, _, status = c.run(max_q_len=6)
    assert status == mxq.DEV_BAD_SEQUENCE
    for i, n, a, b, rows in ((0, 100, 0, 5, [0, 1, 2]), (2, 30, 3, 9, [5, 6, 7, 8])):
        table, starts = c.table[i:i + 1], [a, b]
        ref, tol = few_rows(c.q, c.cache, table, [n], starts)
        assert (np.abs(o - ref)[rows] <= tol[rows]).all()
    # a bound that leaves all of them out writes nothing
    o, _, status = c.run(max_q_len=4)
    assert status == mxq.DEV_BAD_SEQUENCE and np.isnan(o).all()


@pytest.mark.parametrize("heads", [129, 160])
def test_more_query_heads_to_a_key_head_than_a_row_tile_holds(heads):
    # single rows, in parts of at most 16 heads; a prompt, in parts of at most 128
    c = Case([90, 33], [1, 1], heads, 1, 64, 64, 32, seed=heads)
    c.check()
    o, _, _ = c.run()
    ref, tol = few_rows(c.q, c.cache, c.table, c.ctx, c.starts)
    assert (np.abs(o - ref) <= tol).all()
    Case([90, 150], [3, 40], heads, 1, 64, 64, 32, seed=heads).check()
