"""As many rows as 32 bits count."""

import numpy as np
import pytest

from tests import kv_util as ku
from tests.test_gpu_kv_cache import dev_bf16, i32

pytestmark = pytest.mark.gpu


def test_append_of_as_many_rows_as_there_can_be():
    import torch

    import affine_bit_matmul_gb300 as mxq

    T, D, G, page = 2 ** 31 - 1, 64, 32, 16
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 9 GB")
    row = ku.bf16(np.random.default_rng(1).standard_normal((1, 1, D)))
    k = dev_bf16(row).expand(T, 1, D)           # one row, again and again
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    at = {0: 5, 2 ** 30: 0, T - 9: 17, T - 1: 31}
    slots[list(at)] = i32(list(at.values()))
    pages = torch.zeros((2, 1, ku.block_bytes(D, page, G)), dtype=torch.uint8, device="cuda")
    status = i32([-1])
    mxq.kv_append(k, k, pages, slots, group_size=G, dev_status=status)
    assert int(status.item()) == 0
    want = ku.Cache(2, 1, D, page, G)
    want.write(np.asarray(list(at.values())), np.repeat(row, 4, 0), np.repeat(row, 4, 0))
    assert np.array_equal(pages.cpu().numpy(), want.bytes)
