"""Plain 64-bit forms of the key/value cache operators for the tests: the
cache's format by index arithmetic in numpy, the encoder's binary32 decisions,
and attention in float64.  Shares no code with the library."""

from __future__ import annotations

import numpy as np


def bf16(x):
    """float64/float32 array -> the nearest bf16 values (ties to even), as float32."""
    u = np.ascontiguousarray(np.asarray(x, dtype=np.float32)).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16
    return u.astype(np.uint32).view(np.float32).reshape(np.shape(x))


def bf16_bits(x):
    return (np.ascontiguousarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def encode(x, group):
    """bf16 values [..., D] (float32) -> codes uint8 [..., D], scale and bias [..., D/G] (bf16
    values as float32), every decision in binary32."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(x.shape[:-1] + (-1, group)) + np.float32(0)
    mn, mx = g.min(-1), g.max(-1)
    s = bf16((mx - mn) / np.float32(15))
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((g - mn[..., None]) / s[..., None])
    q = np.where(s[..., None] == 0, 0, np.clip(q, 0, 15))
    return q.astype(np.uint8).reshape(x.shape), s, mn


def decode(q, s, b, group):
    """float64 s * q + b."""
    g = q.reshape(q.shape[:-1] + (-1, group)).astype(np.float64)
    return (s.astype(np.float64)[..., None] * g + b.astype(np.float64)[..., None]).reshape(q.shape)


def block_bytes(D, page, group):
    return page * 2 * (D // 2 + 4 * (D // group))


class Cache:
    """A cache on the host: bytes [n_pages, H, block] written row by row with the documented
    places, and the values the rows stand for."""

    def __init__(self, n_pages, H, D, page, group, fill=0):
        self.n_pages, self.H, self.D, self.page, self.group = n_pages, H, D, page, group
        self.bytes = np.full((n_pages, H, block_bytes(D, page, group)), fill, dtype=np.uint8)
        self.k = np.zeros((n_pages * page, H, D))
        self.v = np.zeros((n_pages * page, H, D))
        self.half_range = np.zeros((n_pages * page, H, D))  # 7.5 s of each value of v

    def write(self, slots, k, v):
        """k, v: bf16 values [T, H, D] in float32."""
        D, G, page = self.D, self.group, self.page
        ds = min(D, 128)
        words = ds // 32
        d = np.arange(D)
        for which, x in (("k", k), ("v", v)):
            q, s, b = encode(x, G)
            getattr(self, which)[slots] = decode(q, s, b, G)
            if which == "v":
                self.half_range[slots] = np.repeat(7.5 * s.astype(np.float64), G, axis=-1)
            base = 0 if which == "k" else self.bytes.shape[-1] // 2
            for row, slot in enumerate(slots):
                p, t = slot // page, slot % page
                slab = t // 8 * (D // ds) + d // ds
                e = d % ds
                if which == "k":
                    word = (slab * 32 + (t % 8) * 4 + (e % 32) // 8) * words + e // 32
                    nib = e % 8
                else:
                    word = (slab * 32 + (e % 8) * 4 + (t % 8) // 2) * words + e // 32
                    nib = (t % 2) * 4 + (e % 32) // 8
                at, shift = base + word * 4 + nib // 2, (nib % 2) * 4
                for h in range(self.H):
                    blk = self.bytes[p, h]
                    for sh in (0, 4):
                        m = shift == sh
                        blk[at[m]] = (blk[at[m]] & (0xF0 if sh == 0 else 0x0F)) | (q[row, h][m] << sh)
                    pairs = np.stack([bf16_bits(s[row, h]), bf16_bits(b[row, h])], -1).reshape(-1)
                    off = base + page * D // 2 + t * (D // G) * 4
                    blk[off:off + pairs.size * 2] = pairs.view(np.uint8)


def attention(q, cache, table, ctx, starts, scale, window=0, sinks=0):
    """float64 out [T, Hq, D], lse [T, Hq], and the sums that the error bound needs: A = sum_t P_t
    7.5 s_t (half the range that a code spans), B = sum_t P_t |v_t|, and per row and head E =
    max_t scale sum_d |q_d k_td|."""
    T, Hq, D = q.shape
    rep = Hq // cache.H
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    A, B, E = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    q = q.astype(np.float64)
    for i, n in enumerate(ctx):
        a, b = (starts[i], starts[i + 1])
        t = np.arange(n)
        slots = np.asarray([table[i][x // cache.page] * cache.page + x % cache.page for x in t], dtype=np.int64)
        for row in range(a, b):
            p = n - (b - a) + row - a
            see = t <= p
            if window:
                see &= (t > p - window) | (t < sinks)
            at = slots[see]
            if at.size == 0:
                continue
            for h in range(Hq):
                k, v = cache.k[at, h // rep], cache.v[at, h // rep]
                s = scale * (k @ q[row, h])
                E[row, h] = abs(scale) * (np.abs(k) @ np.abs(q[row, h])).max()
                m = s.max()
                w = np.exp(s - m)
                lse[row, h] = m + np.log(w.sum())
                w /= w.sum()
                out[row, h] = w @ v
                A[row, h] = w @ cache.half_range[at, h // rep]
                B[row, h] = w @ np.abs(v)
    return out, lse, A, B, E


def score_error(E, rounded):
    """How far a score may be off: fp32 sums of up to 256 products, each of a query value and a
    code of up to 31 instead of the value itself (2^-14 E covers 2^-24 (256 + 8) times a few);
    where keys are `rounded`, 11 bits of precision besides (2^-11 E)."""
    return (2.0 ** -14 + (2.0 ** -11 if rounded else 0.0)) * E


def tolerance(ref, A, B, E, rounded):
    """What the kernels' roundings may add up to, element by element.

    One rounding of the output to bf16: 2^-8 |ref|.  Few rows: each weight times its scale is
    rounded to bf16 against codes centred on 7.5: 2^-8 A.  Many rows (`rounded`): weights and
    values have 11 bits of precision: 2 * 2^-11 B.  Scores off by e move the weights by a factor
    exp(+-e) and their sum likewise: 2 e B, and some for the exponentials themselves."""
    e = score_error(E, rounded)[..., None] + 2.0 ** -18
    mine = 2.0 ** -10 * B if rounded else 2.0 ** -8 * A
    return 2.0 ** -8 * np.abs(ref) + mine + 2.0 * e * B + 1e-30


def relative(x, ref):
    """2-norm of the error over the result's: bf16 roundings of the output (2^-8 / sqrt 3 at
    most) and of the weights, whose codes are up to about twice the values they add up to."""
    n = np.linalg.norm(ref)
    return np.linalg.norm(x - ref) / n if n else float(np.abs(x).max(initial=0.0) > 0)


MOST_RELATIVE = 5e-3
