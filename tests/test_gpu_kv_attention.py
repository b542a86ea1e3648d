"""Attention over the paged 4-bit cache against float64, over head shapes,
lengths, masks and kinds of rows; its checks, streams and graphs."""

import numpy as np
import pytest

from tests import kv_util as ku
from tests.test_gpu_kv_cache import SHAPES, dev_bf16, host, i32

pytestmark = pytest.mark.gpu


class Case:
    """A cache with sequences in shuffled pages; slots that nothing wrote hold NaN scales."""

    def __init__(self, ctx, rows, heads, kv_heads, D, G, page, seed=0, q_std=1.2, extra_width=0):
        import torch

        rng = np.random.default_rng(seed)
        used = [-(-n // page) for n in ctx]
        n_pages = sum(used) + 2
        order = rng.permutation(n_pages)
        width = max(max(used), 1) + extra_width
        self.table = np.full((len(ctx), width), -1, dtype=np.int32)
        self.cache = ku.Cache(n_pages, kv_heads, D, page, G, fill=0xFF)
        at = 0
        for i, n in enumerate(ctx):
            self.table[i, :used[i]] = order[at:at + used[i]]
            at += used[i]
            if n:
                t = np.arange(n)
                slots = self.table[i, t // page].astype(np.int64) * page + t % page
                scale = np.where(rng.random(D) < 0.06, 4.0, 0.8)
                self.cache.write(slots, ku.bf16(rng.standard_normal((n, kv_heads, D)) * scale),
                                 ku.bf16(rng.standard_normal((n, kv_heads, D))))
        self.ctx, self.rows, self.group = list(ctx), list(rows), G
        self.starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.q = ku.bf16(rng.standard_normal((int(self.starts[-1]), heads, D)) * q_std)
        self.pages_d = torch.from_numpy(self.cache.bytes).cuda()
        self.q_d, self.table_d = dev_bf16(self.q), i32(self.table)
        self.ctx_d, self.starts_d = i32(self.ctx), i32(self.starts)

    def run(self, **kw):
        import torch

        import affine_bit_matmul_gb300 as mxq

        out = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
        status = i32([-1])
        kw.setdefault("max_q_len", max(self.rows))
        kw.setdefault("q_starts", self.starts_d)
        got = mxq.kv_attention(self.q_d, self.pages_d, self.table_d, self.ctx_d, group_size=self.group,
                               out=out, lse=lse, dev_status=status, **kw)
        assert got is out
        return host(out).astype(np.float64), lse.cpu().numpy().astype(np.float64), int(status.item())

    def many(self):
        rep = self.q.shape[1] // self.cache.H
        parts = -(-rep // 16)
        return np.asarray([n * -(-rep // parts) > 16 for n in self.rows])

    def check(self, window=0, sinks=0, scale=None, status=0, **kw):
        o, lse, st = self.run(window=window, sinks=sinks, scale=scale, **kw)
        assert st == status
        scale = self.q.shape[-1] ** -0.5 if scale is None else scale
        ref, ref_lse, A, B, E = ku.attention(self.q, self.cache, self.table, self.ctx, self.starts, scale, window,
                                             sinks)
        assert np.isfinite(o).all()
        # sequences of more than 16 rows of one key/value head are computed with rounded keys
        many = np.repeat(self.many(), self.rows)
        err = np.abs(o - ref)
        tol = np.where(many[:, None, None], ku.tolerance(ref, A, B, E, True), ku.tolerance(ref, A, B, E, False))
        assert (err <= tol).all(), "worst err/tol %.3g at %s" % (
            (err / tol).max(), np.unravel_index((err / tol).argmax(), err.shape))
        empty = np.isinf(ref_lse)
        assert np.array_equal(np.isinf(lse) & (lse < 0), empty) and not o[empty].any()
        assert ku.relative(o, ref) <= ku.MOST_RELATIVE
        # the scores' error, and fp32 logarithms of sums
        off = np.where(many[:, None], ku.score_error(E, True), ku.score_error(E, False))
        ref_lse[empty] = lse[empty] = 0.0
        assert (np.abs(lse - ref_lse) <= off + 2.0 ** -18 * (1 + np.abs(ref_lse))).all()


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 130, 577]


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("page,heads,kv_heads", [(16, 4, 1), (64, 6, 2)])
def test_single_rows_every_shape(D, G, page, heads, kv_heads):
    Case(LENS, [1] * len(LENS), heads, kv_heads, D, G, page, seed=D + G).check(q_starts=None)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (5, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 2), (71, 1)])
@pytest.mark.parametrize("page", [32, 128])
def test_head_groups(heads, kv_heads, page):
    Case([200, 1, 33], [1, 1, 1], heads, kv_heads, 128, 64, page, seed=heads).check(q_starts=None)


@pytest.mark.parametrize("rows", [2, 3, 4, 8])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 1), (64, 4), (100, 70), (5000, 3)])
def test_few_rows_with_window(rows, window, sinks):
    ctx = [rows, rows + 1, 90, 64 + rows, 400]
    Case(ctx, [rows] * 5, 4, 2, 128, 64, 16, seed=rows + window).check(window, sinks)


def test_rows_that_see_nothing():
    # more rows than tokens, no tokens at all, and sequences without rows
    c = Case([0, 3, 0, 70, 5], [2, 5, 0, 0, 5], 4, 2, 128, 64, 16)
    c.check()
    c = Case([0, 20], [1, 1], 4, 2, 128, 64, 16)
    c.check(q_starts=None)
    c = Case([10, 0, 50], [40, 33, 60], 4, 2, 128, 64, 16)
    c.check()


def test_large_and_small_magnitudes():
    # scores far apart: the running maximum moves in every tile
    for std in (12.0, 1e-3):
        Case([700, 65], [1, 1], 8, 2, 128, 64, 64, seed=9, q_std=std).check(q_starts=None, scale=0.02)
    Case([300], [120], 8, 2, 128, 64, 64, seed=9, q_std=12.0).check(scale=0.02)


def test_rising_scores_move_the_maximum():
    # later keys ever more alike the query: each tile's maximum beats the last by far
    for rows in (1, 40):
        c = Case([640], [rows], 2, 1, 64, 64, 64, seed=4)
        t = np.arange(640)
        slots = c.table[0, t // 64].astype(np.int64) * 64 + t % 64
        k = np.sign(c.q[-1, 0])[None, None] * (0.02 * t)[:, None, None] + np.zeros((640, 1, 64))
        c.cache.write(slots, ku.bf16(k), ku.bf16(c.cache.v[slots]))
        import torch

        c.pages_d = torch.from_numpy(c.cache.bytes).cuda()
        # scores up to 13 * 51: keep the bound's assumption on their errors with a scale
        c.check(scale=0.125)


def test_pages_behind_the_window_may_be_gone():
    c = Case([500, 300], [1, 1], 4, 2, 128, 64, 16, seed=11)
    ref = c.run(q_starts=None, window=40, sinks=5)
    # page 0 holds the first tokens; the pages between them and the window are given up
    for i, n in enumerate(c.ctx):
        gone = slice(1, (n - 40) // 16)
        c.table[i, gone] = [-1, 10 ** 9][i]
    c.table_d = i32(c.table)
    got = c.run(q_starts=None, window=40, sinks=5)
    assert got[2] == 0 and ref[2] == 0
    assert np.array_equal(ref[0], got[0]) and np.array_equal(ref[1], got[1])


@pytest.mark.parametrize("rows", [1, 50])
def test_bad_pages_are_reported_and_not_seen(rows):
    import affine_bit_matmul_gb300 as mxq

    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        c = Case([200, 90], [rows, rows], 4, 2, 128, 64, 32, seed=12)
        c.table_d[0, 2] = bad
        o, _, st = c.run(max_q_len=rows)
        assert st == mxq.DEV_BAD_PAGE
        # the same as if tokens 64..95 of sequence 0 were not there
        t = np.arange(200)
        q, n = c.q.astype(np.float64), 200
        slots = np.where((t >= 64) & (t < 96), -1, c.table[0, t // 32].astype(np.int64) * 32 + t % 32)
        for row in (0, rows - 1):
            p = n - rows + row
            at = slots[:p + 1]
            at = at[at >= 0]
            s = (c.cache.k[at, 0] @ q[row, 0]) * 128 ** -0.5
            w = np.exp(s - s.max())
            w /= w.sum()
            ref = w @ c.cache.v[at, 0]
            E = np.asarray(128 ** -0.5 * (np.abs(c.cache.k[at, 0]) @ np.abs(q[row, 0])).max())
            tol = ku.tolerance(ref, w @ c.cache.half_range[at, 0], w @ np.abs(c.cache.v[at, 0]), E, rows > 8)
            assert (np.abs(o[row, 0] - ref) <= tol).all()


def test_bad_lengths_and_rows_are_reported():
    import affine_bit_matmul_gb300 as mxq

    good = Case([100, 60, 30], [3, 2, 4], 4, 2, 128, 64, 16, seed=13)
    want = good.run()[0]
    for kind in ("negative", "long", "decreasing", "outside", "more"):
        c = Case([100, 60, 30], [3, 2, 4], 4, 2, 128, 64, 16, seed=13)
        kw = {}
        if kind == "negative":
            c.ctx_d[1] = -5                       # as length 0: its rows see nothing
        elif kind == "long":
            c.ctx_d[1] = 10 ** 6                  # as the table's whole width; those pages are not there
        elif kind == "decreasing":
            c.starts_d[1], c.starts_d[2] = 5, 3   # sequence 1 has -2 rows; 0 has 5, 2 has 6
        elif kind == "outside":
            c.starts_d[3] = 10
        else:
            kw["max_q_len"] = 3
        o, _, st = c.run(**kw)
        assert st & mxq.DEV_BAD_SEQUENCE
        if kind == "negative":
            assert not o[3:5].any() and np.array_equal(o[:3], want[:3]) and np.array_equal(o[5:], want[5:])
        elif kind == "long":
            assert np.array_equal(o[:3], want[:3]) and np.array_equal(o[5:], want[5:])
        elif kind == "outside" or kind == "more":
            assert np.isnan(o[5:]).all() and np.array_equal(o[:5], want[:5])


def test_rows_between_guards_strides_and_order():
    import torch

    import affine_bit_matmul_gb300 as mxq

    # query rows as a slice of a wider projection, output between guard rows
    c = Case([333, 20, 64], [1, 1, 1], 8, 2, 128, 64, 16, seed=14)
    plain = c.run(q_starts=None)[0]
    wide = torch.randn(3, 12, 128, device="cuda").bfloat16()
    wide[:, 2:10] = c.q_d
    guard = torch.full((5, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    mxq.kv_attention(wide[:, 2:10], c.pages_d, c.table_d, c.ctx_d, group_size=64, out=guard[1:4])
    assert np.array_equal(host(guard[1:4]), plain)
    assert bool((guard[0] == 7).all()) and bool((guard[4] == 7).all())
    # heads outermost
    turned = c.q_d.transpose(0, 1).contiguous().transpose(0, 1)
    got = mxq.kv_attention(turned, c.pages_d, c.table_d, c.ctx_d, group_size=64)
    assert np.array_equal(host(got), plain)
    # a prompt the same way
    c = Case([100], [60], 8, 2, 128, 64, 16, seed=15)
    plain = c.run()[0]
    turned = c.q_d.transpose(0, 1).contiguous().transpose(0, 1)
    got = mxq.kv_attention(turned, c.pages_d, c.table_d, c.ctx_d, c.starts_d, max_q_len=60, group_size=64)
    assert np.array_equal(host(got), plain)


@pytest.mark.parametrize("rows", [1, 6, 300])
def test_same_bits_every_time_and_on_another_stream(rows):
    import torch

    import affine_bit_matmul_gb300 as mxq

    ctx = [2000, 300, 1203]
    c = Case(ctx, [rows] * 3, 8, 2, 128, 64, 64, seed=16)
    first = c.run()[0]
    s = torch.cuda.Stream()
    need = mxq.kv_attention_workspace_bytes(3 * rows, 3, 8, 2, 128, rows)
    for _ in range(3):
        ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
        out = torch.empty(c.q.shape, dtype=torch.bfloat16, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        mxq.kv_attention(c.q_d, c.pages_d, c.table_d, c.ctx_d, c.starts_d, max_q_len=rows, out=out,
                         workspace=ws, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert np.array_equal(host(out), first)


def test_captured_steps_follow_the_lengths():
    # a decode step in a graph: lengths and tables are read when it runs
    import torch

    import affine_bit_matmul_gb300 as mxq

    c = Case([500, 64, 1], [1, 1, 1], 8, 2, 128, 64, 16, seed=17, extra_width=2)
    ws = torch.empty(mxq.kv_attention_workspace_bytes(3, 3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda")

    def step():
        mxq.kv_attention(c.q_d, c.pages_d, c.table_d, c.ctx_d, group_size=64, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for ctx in ([500, 64, 1], [123, 0, 1], [16, 63, 1]):
        c.ctx = ctx
        c.ctx_d.copy_(i32(ctx))
        g.replay()
        ref, _, A, B, E = ku.attention(c.q, c.cache, c.table, ctx, c.starts, 128 ** -0.5)
        assert (np.abs(host(out) - ref) <= ku.tolerance(ref, A, B, E, False)).all()


def test_many_sequences():
    # more sequences than threads in a block
    ctx = [1 + (37 * i) % 90 for i in range(700)]
    Case(ctx, [1] * 700, 2, 1, 64, 64, 16, seed=18).check(q_starts=None)


@pytest.mark.parametrize("rows", [1, 64])
def test_waits_that_give_up_report_and_leave_the_next_call_right(rows):
    import affine_bit_matmul_gb300 as mxq

    c = Case([900, 300], [rows, rows], 8, 2, 128, 64, 64, seed=19)
    mxq.set_wait_budget(1)
    try:
        st = c.run()[2]
    finally:
        mxq.set_wait_budget(0)
    assert st == mxq.DEV_TIMEOUT
    c.check()


def test_no_rows_and_no_sequences():
    import torch

    import affine_bit_matmul_gb300 as mxq

    c = Case([5], [1], 2, 1, 64, 64, 16)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    status = i32([3])
    out = mxq.kv_attention(none, c.pages_d, c.table_d[:0], c.ctx_d[:0], dev_status=status)
    assert out.shape == (0, 2, 64) and int(status.item()) == 0
    out = mxq.kv_attention(none, c.pages_d, c.table_d, c.ctx_d, i32([0, 0]), max_q_len=4)
    assert out.shape == (0, 2, 64)


@pytest.mark.parametrize("heads,page", [(8, 64), (20, 16), (32, 128)])
def test_long_runs_of_tiles(heads, page):
    # enough tiles for every block to go round its ring several times
    import torch

    import affine_bit_matmul_gb300 as mxq

    S, n, H, D, G = 7, 20000, 4, 128, 64
    rng = np.random.default_rng(20)
    used = -(-n // page)
    n_pages = S * used
    table = rng.permutation(n_pages).reshape(S, used).astype(np.int32)
    ctx = np.asarray([n, n - 1, n - 63, n // 2, n, 64, n - 500], dtype=np.int32)
    pages = torch.full((n_pages, H, ku.block_bytes(D, page, G)), 255, dtype=torch.uint8, device="cuda")
    held = []
    for i in range(S):
        k = ku.bf16(rng.standard_normal((ctx[i], H, D), dtype=np.float32))
        v = ku.bf16(rng.standard_normal((ctx[i], H, D), dtype=np.float32))
        t = np.arange(ctx[i])
        mxq.kv_append(dev_bf16(k), dev_bf16(v), pages, i32(table[i, t // page] * page + t % page))
        held.append((k, v))
    q = ku.bf16(rng.standard_normal((S, heads, D)))
    for _ in range(3):
        o = host(mxq.kv_attention(dev_bf16(q), pages, i32(table), i32(ctx)))
        for i in range(S):
            for h in (0, H - 1):
                K, V = ku.encode(held[i][0][:, h], G), ku.encode(held[i][1][:, h], G)
                k, v = ku.decode(*K, G), ku.decode(*V, G)
                a = h * heads // H
                s = (q[i, a].astype(np.float64) @ k.T) * D ** -0.5
                w = np.exp(s - s.max())
                w /= w.sum()
                ref = w @ v
                E = np.asarray(D ** -0.5 * (np.abs(k) @ np.abs(q[i, a])).max())
                A = np.repeat(7.5 * (w @ V[1].astype(np.float64)), G)
                assert (np.abs(o[i, a] - ref) <= ku.tolerance(ref, A, w @ np.abs(v), E, False)).all()


def test_many_row_tiles_in_a_block():
    # more one-tile sequences and heads to a block than its list of them holds
    ctx = [1 + i % 3 for i in range(3000)]
    Case(ctx, [1] * 3000, 8, 8, 64, 64, 16, seed=23).check(q_starts=None)


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("heads,rows", [(4, 1), (8, 1), (4, 4)])
def test_tables_much_wider_than_the_sequences(D, G, heads, rows):
    # as far as the call can know the sequences are long, so it cuts them over many blocks
    import torch

    c = Case([577, rows, 64, 300], [rows] * 4, heads, 1, D, G, 64, seed=D + G + heads + rows)
    wide = torch.full((4, 600), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table_d.shape[1]] = c.table_d
    c.table_d = wide
    c.check()
