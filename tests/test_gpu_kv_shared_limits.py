"""Attention over shared prefixes where it could go wrong: more units than 32 bits count, queries that
are not numbers, scales of either sign, long contexts, waits that give up, and the places in a
graph or among streams where a call may stand."""

import numpy as np
import pytest

from tests import kv_util as ku
from tests import test_gpu_kv_shared as shared
from tests.test_gpu_kv_accuracy import MOST
from tests.test_gpu_kv_cache import SHAPES, host, i32
from tests.test_gpu_kv_shared import Case
from tests.test_gpu_kv_signs import turned

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["as wide as needed", "wide"])
def width(request):
    """Both ways of a call: each sequence for itself, and groups at once."""
    shared.WIDE = 200000 if request.param == "wide" else 0
    yield request.param
    shared.WIDE = 0


@pytest.mark.parametrize("groups,rows,heads", [([2, 3], 1, 4), ([2, 1], 4, 4), ([40, 3], 1, 4), ([9, 60], 1, 8), ([70], 5, 4)])
def test_a_row_that_is_not_a_number_says_so(width, groups, rows, heads):
    import torch

    import affine_bit_matmul_gb300 as mxq

    S = sum(groups)
    c = Case([300, 70][:len(groups)], groups, [40 + i % 9 for i in range(S)], [rows] * S, heads, 1, 128, 64, 32, seed=S + rows)
    bad = (rows, 1)  # the first row of the second sequence, its second head
    c.q_d[bad] = float("nan")
    o, lse, status = c.run()
    assert status == 0 and np.isnan(o[bad]).all() and np.isnan(lse[bad])
    rest = np.ones(lse.shape, dtype=bool)
    rest[bad] = False
    ref, ref_lse, tol, lse_tol = c.exact(128 ** -0.5)
    assert (np.abs(o - ref) <= tol)[rest].all() and (np.abs(lse - ref_lse) <= lse_tol)[rest].all()
    # a row that sees nothing has no log sum, whatever its query is
    q = torch.full_like(c.q_d, float("nan"))
    lse = torch.zeros(c.q.shape[:2], device="cuda")
    a, kw = c.args(q=q, prefix_lens=i32([0] * len(groups)), ctx_lens=i32([0] * S))
    o = mxq.kv_attention_shared(*a, lse=lse, **kw)
    assert not host(o).any() and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("groups,rows", [([2, 3], 1), ([3, 2], 4), ([40, 3], 1)])
def test_values_with_negative_scales(width, D, G, groups, rows):
    import torch

    S = sum(groups)
    for share, page in ((0.1, 32), (1.0, 16)):
        c = Case([330, 90], groups, [rows + 11 * i % 70 for i in range(S)], [rows] * S, 4, 1, D, G, page, seed=D + S)
        rng = np.random.default_rng(G)
        slots = np.flatnonzero((c.cache.v != 0).any((1, 2)))
        turned(c.cache, slots, rng.random((len(slots), 1, D // G)) < share)
        c.pages_d = torch.from_numpy(c.cache.bytes).cuda()
        c.check()


@pytest.mark.parametrize("groups,rows", [([2, 3], 1), ([3, 2], 4), ([40, 60], 1), ([9, 20], 5)])
def test_waits_that_give_up_report_and_leave_the_next_call_right(width, groups, rows):
    import affine_bit_matmul_gb300 as mxq

    S = sum(groups)
    c = Case([900, 300], groups, [200 + i for i in range(S)], [rows] * S, 8, 2, 128, 64, 64, seed=19)
    mxq.set_wait_budget(1)
    try:
        o, _, st = c.run()
    finally:
        mxq.set_wait_budget(0)
    # (warps on their own may find all that they wait for there: then the result is)
    assert st in (0, mxq.DEV_TIMEOUT)
    if st == 0:
        ref, _, tol, _ = c.exact(128 ** -0.5)
        assert (np.abs(o - ref) <= tol).all()
    c.check()


def test_waits_for_more_than_the_caches_hold_give_up():
    """600 MB of prefixes for 4 rows of 8 heads each: warps on their own wait for the memory."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    c = Case([900, 300], [2, 3], [200 + i for i in range(5)], [1] * 5, 8, 2, 128, 64, 64, seed=20)
    pages = torch.zeros((8192, 8, mxq.kv_block_bytes(128, 64, 64)), dtype=torch.uint8, device="cuda")
    prefix = torch.arange(8192, dtype=torch.int32, device="cuda").view(64, 128)
    q, status = torch.ones((128, 16, 128), device="cuda").bfloat16(), i32([0])
    a = (q, pages, prefix, i32([8192] * 64), torch.zeros((128, 1), dtype=torch.int32, device="cuda"), i32([1] * 128))
    mxq.kv_attention_shared(*a, dev_status=status)
    assert int(status.item()) == 0
    mxq.set_wait_budget(1)
    try:
        mxq.kv_attention_shared(*a, dev_status=status)
        torch.cuda.synchronize()
    finally:
        mxq.set_wait_budget(0)
    assert int(status.item()) == mxq.DEV_TIMEOUT
    c.check()
    o = mxq.kv_attention_shared(*a, dev_status=status)
    assert int(status.item()) == 0 and not host(o).any()


def test_more_units_than_32_bits_count():
    """16000 rows of one sequence after a million tokens, for 5 heads: 2.6e9 row tiles times tiles of tokens.

    Every page is the same one, so that a row sees each of its tokens as often as there are pages up to
    its position."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    T, heads, kv_heads, D, G, page, pages = 16000, 80, 5, 64, 64, 128, 8190
    rng = np.random.default_rng(0)
    c = ku.Cache(2, kv_heads, D, page, G)
    for p in (0, 1):
        c.write(np.arange(page) + p * page, ku.bf16(rng.standard_normal((page, kv_heads, D))),
                ku.bf16(rng.standard_normal((page, kv_heads, D))))
    n = pages * page - 37
    q = torch.randn((T, heads, D), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    lse = torch.full((T, heads), float("nan"), device="cuda")
    status = i32([-1])
    o = mxq.kv_attention_shared(q, torch.from_numpy(c.bytes).cuda(), i32([[1]]), i32([page]), torch.zeros((1, pages), dtype=torch.int32, device="cuda"),
                                i32([n]), None, i32([0, T]), max_q_len=T, group_size=G, lse=lse, dev_status=status)
    assert int(status.item()) == 0
    rep, scale = heads // kv_heads, D ** -0.5
    for row in (0, 1, 127, 5000, 10111, T - 1):
        seen = n - T + row + 1
        times = seen // page + (np.arange(page) < seen % page)
        times = np.concatenate([times, np.ones(page)])
        for h in range(kv_heads):
            hs = slice(h * rep, (h + 1) * rep)
            k, v, half = (np.concatenate([x[:page, h], x[page:, h]]) for x in (c.k, c.v, c.half_range))
            qq = q[row, hs].double().cpu().numpy()
            s = scale * (qq @ k.T)
            # as in Case.exact; a lane's sums have up to 2^16 terms, each addition off by half a step at most: 2^-8
            # of the weights' sum and of the values'
            e = scale * (np.abs(qq) @ np.abs(k).T).max(-1) * (2.0 ** -14 + 2.0 ** -11) + 2.0 ** -18 + 2.0 ** -8
            w = times * np.exp(s - s.max(-1, keepdims=True))
            want = s.max(-1) + np.log(w.sum(-1))
            w /= w.sum(-1, keepdims=True)
            ref, B = w @ v, w @ np.abs(v)
            got = host(o[row, hs]).astype(np.float64)
            assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * (w @ half) + 2 * e[:, None] * B).all()
            assert (np.abs(lse[row, hs].double().cpu().numpy() - want) <= e + 2.0 ** -18 * (1 + np.abs(want))).all()


@pytest.mark.parametrize("where", ["prefix", "own", "each"])
@pytest.mark.parametrize("heads,D,G", [(16, 128, 64), (32, 128, 32), (64, 128, 128), (32, 64, 32), (64, 64, 64), (16, 256, 64), (64, 256, 128)])
def test_long_contexts_are_as_good_as_the_output_type(where, heads, D, G):
    """131072 tokens in a group's prefix, as the sequences' own, or half of them each; groups of 1 to 32 rows times
    query heads to a key/value head."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    n, H, page, seqs = 131072, 8, 64, 16
    gen = torch.Generator(device="cuda").manual_seed(D + G + heads)
    loud = torch.where(torch.rand(D, generator=gen, device="cuda") < 0.06, 4.0, 0.8)
    k = (torch.randn((n, H, D), generator=gen, device="cuda") * loud).bfloat16()
    v = torch.randn((n, H, D), generator=gen, device="cuda").bfloat16()
    order = torch.randperm(n // page, generator=gen, device="cuda").int()
    t = torch.arange(n, device="cuda")
    pages = torch.zeros((n // page, H, mxq.kv_block_bytes(D, page, G)), dtype=torch.uint8, device="cuda")
    mxq.kv_append(k, v, pages, order[t // page] * page + (t % page).int(), group_size=G)
    groups = seqs if where == "each" else 8
    cut = {"prefix": n - 64, "own": 64, "each": n // 2}[where]
    prefix = order[None].expand(groups, -1).contiguous()  # wide, whatever its length
    own = torch.roll(order, -(cut // page))[None].expand(seqs, -1).contiguous()
    lens = [n - cut - (i if where == "prefix" else 7 * i) for i in range(seqs)]
    q = (torch.randn((seqs, heads, D), generator=gen, device="cuda") * 1.2).bfloat16()
    o = mxq.kv_attention_shared(q, pages, prefix, i32([cut] * groups), own, i32(lens), group_size=G).double()

    def held(x):  # what the cache makes of the values, in float64
        g = x.float().unflatten(-1, (-1, G)) + 0.0
        b = g.amin(-1, keepdim=True)
        s = ((g.amax(-1, keepdim=True) - b) / 15.0).bfloat16().float()
        c = ((g - b) / s).round().clamp(0, 15)
        return (s.double() * c.double() + b.double()).flatten(-2)

    rep = heads // H
    off = norm = 0.0
    for h in range(H):
        kk, vv = held(k[:, h]), held(v[:, h])
        for i in range(0, seqs, 3):
            seen = cut + lens[i]
            qq = q[i, h * rep:(h + 1) * rep].double()
            w = torch.softmax((qq @ kk[:seen].T) * D ** -0.5, -1)
            ref = w @ vv[:seen]
            off += float((o[i, h * rep:(h + 1) * rep] - ref).pow(2).sum())
            norm += float(ref.pow(2).sum())
    assert (off / norm) ** 0.5 <= MOST, "%.3e of the norm" % (off / norm) ** 0.5


@pytest.mark.parametrize("groups", [[4, 3], [40, 30]])
def test_behind_other_work_of_streams_and_graphs(width, groups):
    """A call right behind copies, fills and work of another stream, eagerly and captured."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    S = sum(groups)
    c = Case([500, 100], groups, [30] * S, [1] * S, 8, 2, 128, 64, 64, seed=23)
    want = c.run(q_starts=None)[0]
    # what the call reads is written right before it, on this and on another stream
    side = torch.cuda.Stream()
    status = i32([7])
    held = {x: torch.zeros_like(y) for x, y in (("q", c.q_d), ("prefix_table", c.prefix_table_d), ("prefix_lens", c.prefix_d),
                                               ("ctx_lens", c.own_d), ("page_table", c.table_d))}
    source = dict(q=c.q_d, prefix_table=c.prefix_table_d, prefix_lens=c.prefix_d, ctx_lens=c.own_d, page_table=c.table_d)
    a, kw = c.args(q_starts=None, **held)
    out = torch.zeros_like(c.q_d)

    def both():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for x in ("prefix_table", "page_table", "q"):
                held[x].copy_(source[x])
        for x in ("prefix_lens", "ctx_lens"):
            held[x].copy_(source[x])
        main.wait_stream(side)
        mxq.kv_attention_shared(*a, out=out, dev_status=status, **kw)

    def clear():
        for x in held.values():
            x.zero_()
        out.zero_()
        status.fill_(7)

    clear()
    both()
    assert np.array_equal(host(out), want) and int(status.item()) == 0
    clear()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
        for x in held.values():
            x.zero_()  # and after it
    for _ in range(3):
        clear()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out), want) and int(status.item()) == 0


@pytest.mark.parametrize("groups", [[4, 3], [40, 30]])
def test_two_calls_at_once(width, groups):
    """Two streams, a workspace each."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    S = sum(groups)
    cases = [Case([700, 100], groups, [30 + i % 50 for i in range(S)], [1] * S, 8, 2, 128, 64, 64, seed=s) for s in (24, 25)]
    want = [c.run(q_starts=None)[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.zeros_like(c.q_d) for _ in range(8)] for c in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for c, s, o in zip(cases, streams, outs):
            a, kw = c.args(q_starts=None)
            mxq.kv_attention_shared(*a, out=o[i], stream=s, **kw)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(np.array_equal(host(x), w) for x in o)


def test_tensor_cores_between_matrix_products():
    """Kernels that hold tensor memory before and behind the call."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    c = Case([500, 300], [60, 70], [30] * 130, [1] * 130, 8, 2, 64, 64, 64, seed=26)
    want = c.run(q_starts=None)[0]
    w = torch.randn((1024, 512), device="cuda")
    codes, scales, biases = mxq.quantize(w, bits=4, group_size=64)
    x = torch.randn((300, 512), device="cuda").bfloat16()
    y = mxq.qmm(x, codes, scales, biases, 4)
    torch.cuda.synchronize()
    a, kw = c.args(q_starts=None)
    for _ in range(20):
        y1 = mxq.qmm(x, codes, scales, biases, 4)
        o = mxq.kv_attention_shared(*a, **kw)
        y2 = mxq.qmm(x, codes, scales, biases, 4)
        assert np.array_equal(host(o), want) and torch.equal(y1, y) and torch.equal(y2, y)
