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
