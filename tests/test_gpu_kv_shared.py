"""Attention over shared prefixes against float64, over head shapes, lengths, groups and kinds of
rows; its checks of entries, streams and graphs."""

import numpy as np
import pytest

from tests import kv_util as ku
from tests.test_gpu_kv_cache import SHAPES, dev_bf16, host, i32

pytestmark = pytest.mark.gpu

# The calls choose by the width of the page tables whether a group's prefix is taken for all of its rows at once
# or each sequence goes over it for itself: both have to be right for any lengths.
WIDE = 0


@pytest.fixture(autouse=True, params=["as wide as needed", "wide"])
def table_width(request):
    global WIDE
    WIDE = 200000 if request.param == "wide" else 0
    yield
    WIDE = 0


class Case:
    """Groups of sequences over one cache in shuffled pages; slots that nothing wrote hold NaN scales."""

    def __init__(self, prefix, groups, own, rows, heads, kv_heads, D, G, page, seed=0, q_std=1.2, v_scale=1.0):
        """prefix: tokens of each group's prefix; groups: its number of sequences; own, rows: of each sequence."""
        import torch

        rng = np.random.default_rng(seed)
        lens = list(prefix) + list(own)
        used = [-(-n // page) for n in lens]
        order = rng.permutation(sum(used) + 2)
        self.cache = ku.Cache(len(order), kv_heads, D, page, G, fill=0xFF)
        tables, at = [], 0
        for part in (used[:len(prefix)], used[len(prefix):]):
            wide = 0 if tables else WIDE // page  # of the prefixes' table
            t = np.full((len(part), max(max(part), 1, wide)), -1, dtype=np.int32)
            for i, n in enumerate(part):
                t[i, :n] = order[at:at + n]
                at += n
            tables.append(t)
        self.prefix_table, self.table = tables
        scale = np.where(rng.random(D) < 0.06, 4.0, 0.8)
        for t, part in zip(tables, (prefix, own)):
            for i, n in enumerate(part):
                if n:
                    self.cache.write(self.slots(t[i], n), ku.bf16(rng.standard_normal((n, kv_heads, D)) * scale),
                                     ku.bf16(rng.standard_normal((n, kv_heads, D)) * v_scale))
        self.prefix, self.own, self.rows, self.group = list(prefix), list(own), list(rows), G
        self.groups = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
        self.starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.max_group = max(max(groups), 1)
        self.q = ku.bf16(rng.standard_normal((int(self.starts[-1]), heads, D)) * q_std)
        self.pages_d, self.q_d = torch.from_numpy(self.cache.bytes).cuda(), dev_bf16(self.q)
        self.prefix_table_d, self.table_d = i32(self.prefix_table), i32(self.table)
        self.prefix_d, self.own_d, self.groups_d, self.starts_d = i32(self.prefix), i32(self.own), i32(self.groups), i32(self.starts)

    def slots(self, row, n):
        t = np.arange(n)
        return row[t // self.cache.page].astype(np.int64) * self.cache.page + t % self.cache.page

    def args(self, **kw):
        kw.setdefault("max_q_len", max(self.rows))
        kw.setdefault("max_group", self.max_group)
        kw.setdefault("q_starts", self.starts_d)
        kw.setdefault("group_starts", self.groups_d)
        a = [kw.pop(x, y) for x, y in (("q", self.q_d), ("pages", self.pages_d), ("prefix_table", self.prefix_table_d),
                                       ("prefix_lens", self.prefix_d), ("page_table", self.table_d), ("ctx_lens", self.own_d))]
        return a, dict(kw, group_size=self.group)

    def run(self, **kw):
        import torch

        import affine_bit_matmul_gb300 as mxq

        out = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
        status = i32([-1])
        a, kw = self.args(**kw)
        got = mxq.kv_attention_shared(*a, out=out, lse=lse, dev_status=status, **kw)
        assert got is out
        return host(out).astype(np.float64), lse.cpu().numpy().astype(np.float64), int(status.item())

    def rounded(self, max_group=None):
        """Whether keys and values of the prefixes are rounded to 11 bits (more than 32 rows of a group)."""
        rep = self.q.shape[1] // self.cache.H
        rows = min((max_group or self.max_group) * max(self.rows), len(self.q))
        return rows * -(-rep // -(-rep // 16)) > 32

    def exact(self, scale):
        """float64 out, lse; the tolerance of every element and of every lse."""
        T, Hq, D = self.q.shape
        rep = Hq // self.cache.H
        out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
        tol, lse_tol = np.full((T, Hq, D), 1e-30), np.zeros((T, Hq))
        rounded = self.rounded()
        q = self.q.astype(np.float64)
        for i, n in enumerate(self.own):
            g = int(np.searchsorted(self.groups, i, side="right")) - 1
            pre = self.slots(self.prefix_table[g], self.prefix[g]) if 0 <= g < len(self.prefix) else np.zeros(0, np.int64)
            a, b = self.starts[i], self.starts[i + 1]
            own = self.slots(self.table[i], n)
            for row in range(a, b):
                at = np.concatenate([pre, own[:max(0, n - (b - a) + row - a + 1)]])
                if at.size == 0:
                    continue
                # which of the tokens have rounded keys and values
                cut = np.arange(at.size) < (pre.size if rounded else 0)
                for h in range(self.cache.H):
                    k, v, half = self.cache.k[at, h], self.cache.v[at, h], self.cache.half_range[at, h]
                    hs = slice(h * rep, (h + 1) * rep)
                    s = scale * (q[row, hs] @ k.T)
                    e = abs(scale) * (np.abs(q[row, hs]) @ np.abs(k).T)
                    # scores off by e_t: as in kv_util.score_error, by the part that a token is in
                    e = (e * np.where(cut, 2.0 ** -14 + 2.0 ** -11, 2.0 ** -14)).max(-1) + 2.0 ** -18
                    m = s.max(-1, keepdims=True)
                    w = np.exp(s - m)
                    lse[row, hs] = m[:, 0] + np.log(w.sum(-1))
                    w /= w.sum(-1, keepdims=True)
                    out[row, hs] = w @ v
                    B = w @ np.abs(v)
                    mine = 2.0 ** -8 * ((w * ~cut) @ half) + 2.0 ** -10 * ((w * cut) @ np.abs(v))
                    tol[row, hs] = 2.0 ** -8 * np.abs(out[row, hs]) + mine + 2.0 * e[:, None] * B + 1e-30
                    lse_tol[row, hs] = e + 2.0 ** -18 * (1 + np.abs(lse[row, hs]))
        return out, lse, tol, lse_tol

    def check(self, status=0, scale=None, **kw):
        o, lse, st = self.run(scale=scale, **kw)
        assert st == status
        ref, ref_lse, tol, lse_tol = self.exact(self.q.shape[-1] ** -0.5 if scale is None else scale)
        assert np.isfinite(o).all()
        err = np.abs(o - ref)
        assert (err <= tol).all(), "worst err/tol %.3g at %s" % ((err / tol).max(), np.unravel_index((err / tol).argmax(), err.shape))
        empty = np.isinf(ref_lse)
        assert np.array_equal(np.isinf(lse) & (lse < 0), empty) and not o[empty].any()
        assert (np.abs(lse[~empty] - ref_lse[~empty]) <= lse_tol[~empty]).all()
        assert ku.relative(o, ref) <= ku.MOST_RELATIVE
        return o, lse


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("page,groups,heads,kv_heads", [(16, [2, 3], 4, 1), (64, [9, 5], 8, 2), (128, [40, 30], 8, 2)])
def test_every_shape(D, G, page, groups, heads, kv_heads):
    own = [1 + 7 * i % 90 for i in range(sum(groups))]
    Case([200, 77], groups, own, [1] * sum(groups), heads, kv_heads, D, G, page, seed=D + G).check(q_starts=None)


@pytest.mark.parametrize("seqs", [1, 3, 4, 5, 8, 9, 17, 64, 65, 130])
@pytest.mark.parametrize("prefix", [1, 31, 64, 129, 1000])
def test_one_group(seqs, prefix):
    Case([prefix], [seqs], [1 + i % 20 for i in range(seqs)], [1] * seqs, 8, 2, 128, 64, 32, seed=seqs + prefix).check(
        q_starts=None, group_starts=None)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (5, 1), (16, 1), (17, 1), (40, 2), (71, 1), (130, 1)])
def test_head_groups(heads, kv_heads):
    for groups in ([1, 2], [12, 30]):
        Case([300, 90], groups, [40] * sum(groups), [1] * sum(groups), heads, kv_heads, 128, 64, 32, seed=heads).check(q_starts=None)


@pytest.mark.parametrize("most", [2, 4, 9, 33])
def test_several_rows_a_sequence(most):
    rows = [1 + (3 * i) % most for i in range(14)]
    rows[5] = 0
    own = [max(r, 5 * i) for i, r in enumerate(rows)]
    Case([130, 400, 70], [4, 9, 1], own, rows, 8, 2, 128, 64, 16, seed=most).check(max_q_len=most)


def test_empty_parts():
    # no prefix, no own tokens, neither; groups without sequences; sequences of no group, before and after the groups
    c = Case([0, 90, 0, 64], [3, 2, 0, 2], [5, 0, 64, 0, 7, 0, 1], [1] * 7, 4, 2, 128, 64, 32, seed=3)
    o, lse = c.check(q_starts=None)
    assert np.isinf(lse[1]).all() and not o[1].any()
    c = Case([40, 50], [2, 3], [9, 0, 33, 8, 5, 70, 11], [2, 1, 3, 1, 1, 1, 2], 4, 2, 128, 64, 16, seed=4)
    c.groups = np.asarray([1, 3, 6], dtype=np.int32)
    c.check(group_starts=i32(c.groups))
    # rows at or before the first own token see the prefix only
    c = Case([40], [2], [2, 0], [5, 3], 4, 2, 128, 64, 16, seed=5)
    c.check()


def test_large_and_small_magnitudes():
    for std in (12.0, 1e-3):
        Case([700, 65], [20, 2], [60] * 22, [1] * 22, 8, 2, 128, 64, 64, seed=9, q_std=std).check(q_starts=None, scale=0.02)
    Case([700, 65], [20, 2], [60] * 22, [1] * 22, 8, 2, 128, 64, 64, seed=10, v_scale=1e4).check(q_starts=None)


def test_as_the_same_tokens_without_sharing():
    """The same keys and values in tables of their own for each sequence give the same result up to both calls' roundings."""
    import affine_bit_matmul_gb300 as mxq

    c = Case([256, 128], [5, 20], [40] * 25, [1] * 25, 8, 2, 128, 64, 64, seed=11)
    whole = np.full((25, 5), -1, dtype=np.int32)
    lens = []
    for i in range(25):
        g = 0 if i < 5 else 1
        n = c.prefix[g] // 64
        whole[i, :n] = c.prefix_table[g, :n]
        whole[i, n] = c.table[i, 0]
        lens.append(c.prefix[g] + 40)
    o = host(mxq.kv_attention(c.q_d, c.pages_d, i32(whole), i32(lens))).astype(np.float64)
    assert ku.relative(c.run(q_starts=None)[0], o) <= 2 * ku.MOST_RELATIVE


def test_a_long_batch_with_little_to_share():
    # each sequence for itself over contexts that are cut
    Case([900, 30], [1, 1], [2500, 3000], [1, 1], 8, 8, 128, 64, 64, seed=21).check(q_starts=None)
    Case([900] * 40, [1] * 40, [300] * 40, [2] * 40, 8, 2, 128, 64, 64, seed=22).check()


def test_many_groups_and_long_prefixes_are_cut_anywhere():
    groups = [1 + i % 7 for i in range(70)]
    prefix = [1 + (97 * i) % 700 for i in range(70)]
    own = [(31 * i) % 150 for i in range(sum(groups))]
    Case(prefix, groups, own, [1] * sum(groups), 4, 1, 64, 32, 16, seed=12).check(q_starts=None)
    Case([9000], [33], [1 + i for i in range(33)], [1] * 33, 4, 1, 64, 32, 128, seed=13).check(q_starts=None)


def test_bound_of_the_group_decides_the_kernel_only():
    c = Case([500, 100], [4, 3], [30] * 7, [1] * 7, 8, 2, 128, 64, 64, seed=14)
    few, _ = c.check(q_starts=None, max_group=4)
    many, _, st = c.run(q_starts=None, max_group=7)
    c.max_group = 100
    assert st == 0 and ku.relative(many, c.exact(128 ** -0.5)[0]) <= ku.MOST_RELATIVE
    again, _, _ = c.run(q_starts=None, max_group=4)
    assert np.array_equal(few, again)


def test_strided_queries_and_other_scale():
    import torch

    c = Case([90], [9], [20] * 9, [1] * 9, 8, 2, 64, 32, 32, seed=15)
    wide = torch.full((9, 12, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = c.q_d
    c.check(q=wide[:, 2:10], q_starts=None, scale=0.3)
    flip = torch.empty((8, 9, 64), dtype=torch.bfloat16, device="cuda")
    flip.copy_(c.q_d.transpose(0, 1))
    c.check(q=flip.transpose(0, 1), q_starts=None)


def test_bad_entries_are_reported_and_harmless():
    import affine_bit_matmul_gb300 as mxq

    c = Case([100, 70], [3, 4], [20] * 7, [1] * 7, 4, 1, 128, 64, 16, seed=16)
    good, good_lse, tol, _ = c.exact(128 ** -0.5)

    def same(o, left):
        # (where the tokens are cut, and so how they are added up, goes by all lengths)
        assert (np.abs(o[left] - good[left]) <= tol[left]).all()

    def same_but(changed, **kw):
        o, lse, st = c.run(**{"q_starts": None, **kw})
        same(o, [i for i in range(7) if i not in changed])
        return o, lse, st

    # a page outside the cache: its tokens are invisible
    for far in (-1, len(c.cache.bytes), 2 ** 31 - 1):
        t = c.prefix_table.copy()
        t[0, 3] = far
        o, _, st = same_but([0, 1, 2], prefix_table=i32(t))
        assert st == mxq.DEV_BAD_PAGE and np.isfinite(o).all()
        t = c.table.copy()
        t[5, 1] = far
        o, _, st = same_but([5], page_table=i32(t))
        assert st == mxq.DEV_BAD_PAGE and np.isfinite(o).all()
    # lengths past the tables, or negative: clamped
    o, _, st = same_but([0, 1, 2], prefix_lens=i32([-5, 70]))
    assert st == mxq.DEV_BAD_SEQUENCE and np.isfinite(o).all()
    o, _, st = same_but([3], ctx_lens=i32([20, 20, 20, -1, 20, 20, 20]))
    assert st == mxq.DEV_BAD_SEQUENCE and np.isfinite(o).all()
    # groups out of range, of too many sequences, decreasing
    for groups, lost in (([0, 3, 8], [3, 4, 5, 6]), ([-1, 3, 7], [0, 1, 2]), ([3, 0, 0], list(range(7)))):
        o, _, st = c.run(q_starts=None, group_starts=i32(groups))
        assert st == mxq.DEV_BAD_SEQUENCE
        same(o, [i for i in range(7) if i not in lost])
    o, _, st = same_but([3, 4, 5, 6], max_group=3)
    assert st == mxq.DEV_BAD_SEQUENCE and np.isnan(o[3:]).all()
    # rows out of range or too many: left out
    for starts in ([0, 1, 2, 3, 4, 5, 6, 9], [0, 1, 2, 3, 4, 2, 6, 7], [-3, 1, 2, 3, 4, 5, 6, 7], [5, 1, 5, 1, 5, 1, 5, 1]):
        o, _, st = c.run(q_starts=i32(starts), max_q_len=2)
        assert st & mxq.DEV_BAD_SEQUENCE


def test_same_bits_every_time():
    c = Case([3000], [50], [100 + i for i in range(50)], [1] * 50, 8, 2, 128, 64, 64, seed=17)
    first = c.run(q_starts=None)
    for _ in range(5):
        again = c.run(q_starts=None)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_another_stream_and_graphs_with_their_own_workspaces():
    import torch

    import affine_bit_matmul_gb300 as mxq

    cases = [Case([700], [4], [30] * 4, [1] * 4, 8, 2, 128, 64, 64, seed=18), Case([900], [60], [50] * 60, [1] * 60, 8, 2, 128, 64, 64, seed=19)]
    want = [c.run(q_starts=None)[0] for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for c, w in zip(cases, want):
        a, kw = c.args(q_starts=None)
        got = mxq.kv_attention_shared(*a, stream=side, **kw)
        side.synchronize()
        assert np.array_equal(host(got), w)
    graphs, outs = [], []
    for c in cases:
        a, kw = c.args(q_starts=None)
        kw["out"] = torch.zeros_like(c.q_d)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                mxq.kv_attention_shared(*a, **kw)
        graphs.append(g)
        outs.append(kw["out"])
    for _ in range(3):
        for g, o, w in zip(graphs, outs, want):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(host(o), w)
