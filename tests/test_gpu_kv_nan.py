"""Queries that are not numbers, in the attention over the 4-bit cache."""

import numpy as np
import pytest

from tests import kv_util as ku
from tests.test_gpu_kv_attention import Case
from tests.test_gpu_kv_cache import host, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,rows", [(4, 1), (8, 1), (4, 4), (4, 40)])
@pytest.mark.parametrize("width", [0, 400])  # not cut, and cut over many blocks
def test_a_row_that_is_not_a_number_says_so_in_its_log_sum(heads, rows, width):
    import torch

    import affine_bit_matmul_gb300 as mxq

    c = Case([300, 90], [rows, rows], heads, 1, 128, 64, 32, seed=heads + rows, extra_width=width)
    bad = (rows, 1)  # the first row of the second sequence, its second head
    c.q_d[bad] = float("nan")
    o, lse, status = c.run()
    assert status == 0
    assert np.isnan(o[bad]).all() and np.isnan(lse[bad])
    rest = np.ones(lse.shape, dtype=bool)
    rest[bad] = False
    ref, ref_lse, A, B, E = ku.attention(c.q, c.cache, c.table, c.ctx, c.starts, 128 ** -0.5)
    many = bool(c.many().all())
    assert (np.abs(o - ref) <= ku.tolerance(ref, A, B, E, many))[rest].all()
    assert (np.abs(lse - ref_lse) <= ku.score_error(E, many) + 2.0 ** -18 * (1 + np.abs(ref_lse)))[rest].all()
    # a row that sees nothing has no log sum, whatever its query is
    q = torch.full((2, heads, 128), float("nan"), device="cuda").bfloat16()
    lse = torch.zeros((2, heads), device="cuda")
    o = mxq.kv_attention(q, c.pages_d, c.table_d, i32([0, 0]), group_size=64, lse=lse)
    assert not host(o).any() and bool((lse == -float("inf")).all())
