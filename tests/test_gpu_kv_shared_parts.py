"""Attention over shared prefixes where a key/value head's query heads do not divide evenly into the parts that a row
tile takes: the smaller part then has fewer row tiles than the others."""

import numpy as np
import pytest

from tests import test_gpu_kv_shared as shared
from tests.test_gpu_kv_shared import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["as wide as needed", "wide"])
def width(request):
    shared.WIDE = 200000 if request.param == "wide" else 0
    yield request.param
    shared.WIDE = 0


# more than 16 heads are parts of up to 16 for warps on their own, more than 128 parts of up to 128 for the tensor
# cores; 19 and 40 heads in parts of 10 and 14 with one smaller one, 129 in 65 and 64
@pytest.mark.parametrize("heads", [17, 25, 40, 71, 113, 129, 133, 257])
@pytest.mark.parametrize("rows", [2, 4, 16])
def test_several_rows_of_uneven_parts(width, heads, rows):
    # sequences that fill their row of the table, the last one too, with an odd number of pages of 16: a tile of
    # 32 tokens then ends a page after the table
    Case([200, 64], [2, 3], [80, 40, 48, 30, 80], [rows, 1, rows, rows, 2], heads, 1, 128, 64, 16, seed=heads + rows).check()


@pytest.mark.parametrize("D,G", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("heads,rows", [(17, 2), (71, 3), (129, 4), (131, 8)])
def test_uneven_parts_of_two_heads(width, D, G, heads, rows):
    Case([130], [2], [64, 33], [rows, rows], 2 * heads, 2, D, G, 32, seed=D + heads).check()


@pytest.mark.parametrize("seqs", [1, 2, 4, 7])
@pytest.mark.parametrize("heads", [129, 137, 257])
def test_groups_of_single_rows_of_uneven_parts(width, heads, seqs):
    Case([3000], [seqs], [17 + i for i in range(seqs)], [1] * seqs, heads, 1, 64, 64, 64, seed=heads + seqs).check(q_starts=None)


def test_the_same_bits_beside_other_groups(width):
    # pieces of the smaller part are left out anywhere in a run
    c = Case([400, 90, 1500], [3, 1, 4], [20, 70, 5, 64, 33, 90, 11, 48], [4, 1, 3, 2, 4, 4, 2, 1], 129, 1, 128, 64, 16, seed=1)
    o, lse = c.check()
    for _ in range(3):
        again = c.run()
        assert again[2] == 0 and np.array_equal(again[0], o) and np.array_equal(again[1], lse)
