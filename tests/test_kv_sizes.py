"""Sizes past 32 bits, on the host."""

import pytest


def test_sizes_past_32_bits_are_not_taken_for_their_lowest_bits():
    from affine_bit_matmul_gb300 import build

    build.build()
    import affine_bit_matmul_gb300 as mxq

    assert mxq.kv_block_bytes(128, 64, 64) == 9216
    for bad in ((2 ** 32 + 128, 64, 64), (128, 2 ** 32 + 64, 64), (128, 64, 2 ** 32 + 64), (128 - 2 ** 32, 64, 64)):
        with pytest.raises(ValueError):
            mxq.kv_block_bytes(*bad)
    whole = mxq.kv_attention_workspace_bytes(40, 4, 8, 2, 128, 40)
    assert whole > mxq.kv_attention_workspace_bytes(40, 4, 8, 2, 128, 1)
    assert mxq.kv_attention_workspace_bytes(40, 4, 8, 2, 128, 2 ** 32 + 1) == whole


@pytest.fixture(scope="module")
def L():
    from affine_bit_matmul_gb300 import build

    build.build()
    import affine_bit_matmul_gb300 as mxq

    return mxq.lib()


def attend(L, T, S, heads, kv_heads, D, width, page, most):
    import ctypes

    at = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
    starts = at if most > 1 else None
    need = L.mxq_kv_attention_workspace_bytes(T, S, heads, kv_heads, D, most)
    return L.mxq_kv_attention(at, heads * D, D, at, at, at, starts, at, None, T, S, heads, kv_heads, D, 8, width, page, 64,
                              most, 0.1, 0, 0, at, need, None, None)


@pytest.mark.parametrize("T,S,heads,kv_heads,width,page,most", [
    (1 << 23, 1, 8, 2, 1 << 19, 16, 1 << 23),        # one prompt of 2^23 rows over 2^23 tokens: 2^33 units
    (1 << 30, 1 << 30, 1, 1, 1, 16, 1 << 30),        # more row tiles than 32 bits
    (1 << 26, 1 << 26, 8, 8, 1 << 20, 128, 1),       # 2^19 sequences to a thread, 2^22 units each
    (4, 4, 1 << 12, 1 << 12, 1 << 23, 128, 1),       # 2^37 units in a sequence
])
def test_calls_with_more_units_than_32_bits_count_are_refused(L, T, S, heads, kv_heads, width, page, most):
    assert attend(L, T, S, heads, kv_heads, 64, width, page, most) == 3


@pytest.mark.parametrize("T,S,heads,kv_heads,width,page,most", [
    (1 << 20, 1024, 32, 8, 1 << 13, 128, 1 << 20),   # 2^20 rows in a table for 2^20 tokens a sequence
    (4096, 4096, 64, 8, 1 << 13, 128, 1), (16, 16, 128, 128, 1 << 16, 128, 1), (1 << 20, 1, 32, 8, 1 << 13, 128, 1 << 20),
])
def test_long_calls_reach_the_device_check(L, T, S, heads, kv_heads, width, page, most):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the call would run")
    assert attend(L, T, S, heads, kv_heads, 128, width, page, most) in (4, 5)
