"""Signs in the paged 4-bit key/value cache: groups of negative zeros going in."""

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
