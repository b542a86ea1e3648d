"""Attention over shared prefixes with starts that decrease: what is written is right, the rest as it was."""

import numpy as np
import pytest

from tests import test_gpu_kv_shared as shared
from tests.test_gpu_kv_cache import i32
from tests.test_gpu_kv_shared import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["as wide as needed", "wide"])
def width(request):
    shared.WIDE = 200000 if request.param == "wide" else 0
    yield request.param
    shared.WIDE = 0


def left_or_right(case, starts, max_group):
    """The status is set, and every row is untouched or right for a group that has its sequence."""
    import affine_bit_matmul_gb300 as mxq

    o, lse, st = case.run(q_starts=None, group_starts=i32(starts), max_group=max_group)
    assert st == mxq.DEV_BAD_SEQUENCE
    written = ~np.isnan(o).any((1, 2))
    assert np.isnan(o[~written]).all() and np.isnan(lse[~written]).all() and not np.isnan(lse[written]).any()
    fits = np.zeros(len(o), dtype=bool)
    seqs = len(case.own)
    for g, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        if not 0 <= a <= b <= seqs or b - a > max_group:
            continue
        # all sequences after this group's prefix
        case.groups = np.asarray([0] * (g + 1) + [seqs] * (len(starts) - 1 - g), dtype=np.int32)
        ref, ref_lse, tol, lse_tol = case.exact(128 ** -0.5)
        with np.errstate(invalid="ignore"):
            same = (np.abs(o - ref) <= tol).all((1, 2)) & (np.abs(lse - ref_lse) <= lse_tol).all(1)
        fits[a:b] |= same[a:b]
    assert (written <= fits).all(), "rows %s" % np.flatnonzero(written & ~fits)
    return written


@pytest.mark.parametrize("seqs", [3, 7, 300])
def test_groups_that_overlap(width, seqs):
    # the second and fourth group decrease; the others are all sequences, or those but one
    case = Case([70, 40, 90, 20, 130], [seqs, 0, 0, 0, 0], [20] * seqs, [1] * seqs, 8, 2, 128, 64, 32, seed=seqs)
    left_or_right(case, [0, seqs, 0, seqs, 1, seqs], seqs)


def test_a_group_that_decreases_leaves_the_others(width):
    case = Case([70, 40, 90], [4, 3, 3], [20] * 10, [1] * 10, 8, 2, 128, 64, 32, seed=5)
    assert left_or_right(case, [0, 7, 4, 10], 7)[:4].all()


def test_sequences_that_overlap(width):
    import affine_bit_matmul_gb300 as mxq

    case = Case([70], [9], [60] * 9, [40] + [0] * 8, 8, 2, 128, 64, 32, seed=6)
    # five sequences of 40 rows: more row tiles than 40 rows can have
    o, lse, st = case.run(q_starts=i32([0, 40, 0, 40, 0, 40, 0, 40, 0, 40]), max_q_len=40)
    assert st == mxq.DEV_BAD_SEQUENCE and np.isnan(o).all() and np.isnan(lse).all()
    # one that decreases, with its rows in the next one only
    o, lse, st = case.run(q_starts=i32([0, 30, 20, 40, 40, 40, 40, 40, 40, 40]), max_q_len=40)
    assert st == mxq.DEV_BAD_SEQUENCE


def test_one_long_sequence_among_short_ones(width):
    rows = [1] * 40
    rows[17] = 300
    case = Case([100, 40], [25, 15], [max(r, 5 + i) for i, r in enumerate(rows)], rows, 8, 2, 128, 64, 32, seed=7)
    case.check()


@pytest.mark.parametrize("starts", [[0, 1, 2, 3, 4, 5, 6, 9], [0, 1, 2, 3, 4, 2, 6, 7], [-3, 1, 2, 3, 4, 5, 6, 7], [5, 1, 5, 1, 5, 1, 5, 1],
                                    [0, 2, 4, 7, 7, 7, 7, 7], [0, 1, 1, 3, 3, 5, 6, 7]])
@pytest.mark.parametrize("groups", [[3, 4], [7, 0]])
def test_sequences_beside_malformed_ones(width, groups, starts):
    import affine_bit_matmul_gb300 as mxq

    case = Case([100, 70], groups, [20] * 7, [1] * 7, 4, 1, 128, 64, 16, seed=16)
    o, lse, st = case.run(q_starts=i32(starts), max_q_len=2)
    fine = [0 <= a <= b <= 7 and b - a <= 2 for a, b in zip(starts[:-1], starts[1:])]
    assert st == (0 if all(fine) else mxq.DEV_BAD_SEQUENCE)
    of = {}  # row -> the sequences that have it
    for i in np.flatnonzero(fine):
        for row in range(starts[i], starts[i + 1]):
            of.setdefault(row, []).append(i)
    written = ~np.isnan(o).any((1, 2))
    assert not written[[row for row in range(7) if row not in of]].any()
    # where the starts of a group's first or last sequence are malformed its rows are not known
    edges = np.concatenate([[0], np.cumsum(groups)])
    known = [0 <= starts[a] <= starts[b] <= 7 for a, b in zip(edges[:-1], edges[1:])]
    for row, seqs in of.items():
        if len(seqs) > 1:
            continue
        i = seqs[0]
        case.starts = np.asarray([starts[i]] * (i + 1) + [starts[i + 1]] * (7 - i), dtype=np.int32)
        ref, ref_lse, tol, lse_tol = case.exact(128 ** -0.5)
        right = written[row] and (np.abs(o - ref) <= tol)[row].all() and (np.abs(lse - ref_lse) <= lse_tol)[row].all()
        inside = any(k and a <= i < b and starts[a] <= starts[i] and starts[i + 1] <= starts[b] for k, a, b in zip(known, edges[:-1], edges[1:]))
        assert right if inside else right or not written[row]
