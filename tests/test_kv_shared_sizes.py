"""Workspaces of attention over shared prefixes, and the calls that they allow, on the host."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from affine_bit_matmul_gb300 import build

    build.build()
    import affine_bit_matmul_gb300 as mxq

    return mxq.lib()


def attend(L, T, S, N, heads, kv_heads, D, pages, most, group):
    at = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
    need = L.mxq_kv_attention_shared_workspace_bytes(T, S, N, heads, kv_heads, D, most, group)
    return L.mxq_kv_attention_shared(at, heads * D, D, at, at, at, at, at, at, at, at, None, T, S, N, heads, kv_heads, D, 8, pages,
                                     pages, 64, 64, most, group, 0.1, at, need, None, None)


@pytest.mark.parametrize("T,S,N,most", [(2048 + 255, 256, 1, 2048), (2048 + 255, 256, 32, 2048), (1000 + 127, 128, 16, 1000)])
def test_one_long_sequence_among_short_ones_takes_no_room_for_all_as_long(L, T, S, N, most):
    import torch

    need = L.mxq_kv_attention_shared_workspace_bytes(T, S, N, 32, 8, 128, most, S // N)
    # a place is 16 rows of 130 numbers, one for each row tile of 4 tokens of a key/value head, each sequence's last one
    # and each of 160 x 16 warps; the tensor cores' are of 256 rows, of at most T / 64 + N tiles and 160 blocks
    places = (T // 4 + S) * 8 + 16 * 160, (T // 64 + N) * 8 + 160
    assert need <= (places[0] * 16 + places[1] * 256) * 130 * 4 + (S + N) * 64 + 4096 <= 300 << 20
    # tables of 131072 tokens are no reason to refuse it (these pointers are for machines without a GPU only)
    if not torch.cuda.is_available():
        assert attend(L, T, S, N, 32, 8, 128, 2048, most, S // N) in (4, 5)


def test_calls_that_cannot_be_counted_are_refused(L):
    # 2^22 row tiles of 2^10 tiles of tokens; row tiles of sequences that may overlap
    assert attend(L, 1 << 22, 1 << 22, 1, 4, 1, 64, 1 << 10, 4, 1 << 22) == 3
    assert attend(L, 1 << 24, 1 << 22, 1, 4, 1, 64, 1, 1 << 20, 1) == 3


def test_sizes_past_32_bits_are_not_taken_for_their_lowest_bits(L):
    import affine_bit_matmul_gb300 as mxq

    small = mxq.kv_attention_shared_workspace_bytes(4, 4, 2, 8, 2, 128, 1, 2)
    assert mxq.kv_attention_shared_workspace_bytes(4, 2 ** 32 + 4, 2, 8, 2, 128, 1, 2) > small
    assert mxq.kv_attention_shared_workspace_bytes(2 ** 32 + 4, 4, 2, 8, 2, 128, 2 ** 33, 2) > small
    for bad in ((4, 4, 2 ** 32, 8, 2, 128), (4, 4, 2, 8, 2 ** 32 + 2, 128), (4, 4, 2, 8 - 2 ** 32, 2, 128)):
        assert mxq.kv_attention_shared_workspace_bytes(*bad, 1, 2) == (0 if bad[2] == 2 else mxq.kv_attention_shared_workspace_bytes(
            4, 4, 2 ** 31 - 1, 8, 2, 128, 1, 2))
