"""Signs in the paged 4-bit key/value cache: groups of negative zeros going in, and
pairs whose scale is negative in what the attention reads."""

import numpy as np
import pytest

from tests import kv_util as ku
from tests.test_gpu_kv_attention import Case
from tests.test_gpu_kv_cache import SHAPES, dev_bf16, i32

pytestmark = pytest.mark.gpu


def zeros_of_both_signs(rng, T, H, D):
    """Rows in whose groups everything is -0, or +0, or both, or at most -0, or at least -0."""
    x = rng.standard_normal((T, H, D // 32, 32))
    kind = rng.integers(0, 6, (T, H, D // 32, 1))
    neg, pos = np.full(x.shape, -0.0), np.zeros(x.shape)
    some = rng.random(x.shape) < 0.3
    x = np.where(kind == 1, neg, x)
    x = np.where(kind == 2, pos, x)
    x = np.where(kind == 3, np.where(some, neg, pos), x)
    x = np.where(kind == 4, np.where(some, neg, -np.abs(x)), x)
    x = np.where(kind == 5, np.where(some, neg, np.abs(x)), x)
    x = ku.bf16(x.reshape(T, H, D))
    x[0, 0] = -0.0  # every group of the first row, and half of the second
    x[1, 0, :D // 2] = -0.0
    return x


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("T", [5, 700])  # below and above the size from which a warp takes 8 tokens
def test_groups_of_negative_zeros_bit_for_bit(D, G, T):
    import torch

    import affine_bit_matmul_gb300 as mxq

    H, page = 2, 32
    rng = np.random.default_rng(D + G + T)
    k, v = zeros_of_both_signs(rng, T, H, D), zeros_of_both_signs(rng, T, H, D)
    assert np.signbit(v[0, 0]).all()
    n_pages = T // page + 2
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    want = ku.Cache(n_pages, H, D, page, G)
    want.write(slots, k, v)
    pages = torch.zeros(want.bytes.shape, dtype=torch.uint8, device="cuda")
    k_d, v_d = dev_bf16(k), dev_bf16(v)
    assert bool((v_d[0, 0].view(torch.int16) == -32768).all())
    mxq.kv_append(k_d, v_d, pages, i32(slots), group_size=G)
    assert np.array_equal(pages.cpu().numpy(), want.bytes)
    # the weights' encoder has the same rule
    rows = torch.cat((k_d, v_d)).float().view(-1, D)
    codes, scales, biases = mxq.quantize(rows, bits=4, group_size=G)
    assert not bool((scales.view(torch.int16) < 0).any()) and not bool((biases.view(torch.int16) == -32768).any())


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("rows", [1, 40])
def test_attention_after_a_token_of_negative_zeros(D, G, rows):
    import torch

    import affine_bit_matmul_gb300 as mxq

    c = Case([300, 90], [rows, rows], 4, 2, D, G, 32, seed=D + G)
    # written anew through the library: the first tokens' values are -0 in some or all groups
    k, v = ku.bf16(c.cache.k), ku.bf16(c.cache.v)
    at = [c.table[i, t // 32] * 32 + t % 32 for i, t in ((0, 0), (0, 70), (1, 3))]
    v[at[0]] = -0.0
    v[at[1], :, :G] = -0.0
    v[at[2], 0] = -0.0
    held = np.flatnonzero((c.cache.v != 0).any((1, 2)))
    fresh = ku.Cache(c.cache.n_pages, 2, D, 32, G, fill=0xFF)
    fresh.write(held, k[held], v[held])
    c.cache = fresh
    c.pages_d = torch.full(fresh.bytes.shape, 0xFF, dtype=torch.uint8, device="cuda")
    mxq.kv_append(dev_bf16(k[held]), dev_bf16(v[held]), c.pages_d, i32(held), group_size=G)
    c.check()


def turned(cache, slots, which):
    """Gives the groups `which` [slots, H, D/G] of the values at `slots` a negative scale: the same
    codes count down from the group's maximum."""
    D, G, page = cache.D, cache.group, cache.page
    half = cache.bytes.shape[-1] // 2
    for row, slot in enumerate(slots):
        p, t = slot // page, slot % page
        for h in range(cache.H):
            first = half + page * D // 2 + t * (D // G) * 4
            pairs = cache.bytes[p, h, first:first + D // G * 4].view(np.uint16).reshape(-1, 2)
            s = (pairs[:, 0].astype(np.uint32) << 16).view(np.float32)
            b = (pairs[:, 1].astype(np.uint32) << 16).view(np.float32)
            top = ku.bf16(b + 15 * s)
            m = which[row, h]
            q = (cache.v[slot, h].reshape(-1, G) - b[:, None].astype(np.float64)) / np.where(s == 0, 1, s)[:, None]
            now = top[:, None] - s[:, None].astype(np.float64) * np.rint(q)
            cache.v[slot, h] = np.where(m[:, None], now, cache.v[slot, h].reshape(-1, G)).reshape(-1)
            pairs[m, 0] ^= 0x8000
            pairs[m, 1] = ku.bf16_bits(top)[m]


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("heads,rows", [(4, 1), (8, 1), (4, 4), (4, 40)])
def test_values_with_negative_scales(D, G, heads, rows):
    import torch

    c = Case([330, 90, 17], [rows, rows, min(rows, 17)], heads, 1, D, G, 32, seed=D + heads + rows)
    rng = np.random.default_rng(G)
    slots = np.flatnonzero((c.cache.v != 0).any((1, 2)))
    turned(c.cache, slots, rng.random((len(slots), 1, D // G)) < 0.1)
    c.pages_d = torch.from_numpy(c.cache.bytes).cuda()
    c.check()
    # and all of them
    c = Case([200, 90], [rows, rows], heads, 1, D, G, 16, seed=D + heads + rows)
    slots = np.flatnonzero((c.cache.v != 0).any((1, 2)))
    turned(c.cache, slots, np.ones((len(slots), 1, D // G), dtype=bool))
    c.pages_d = torch.from_numpy(c.cache.bytes).cuda()
    c.check()
