"""Selection of beams and the cache's reordering: results in the place of the arguments, behind other work of
streams and graphs, two calls at once, and logits at the end of what their type holds."""

import numpy as np
import pytest

from tests.test_gpu_beam_select import bf16, check, dev, logits
from tests.test_gpu_kv_cache import i32
from tests.test_gpu_kv_reorder import Case, plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,W", [(1, 4), (7, 8), (3, 64), (40, 5), (200, 8)])
def test_results_in_the_place_of_the_arguments(N, W):
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(N + W)
    x = dev(logits(rng, N, W, 700).reshape(N * W, 700), torch.bfloat16)
    scores, done = dev((-10 * rng.random((N, W))).astype(np.float32)), dev(rng.random((N, W)) < 0.4)
    want = mxq.beam_select(x, scores, done=done, end_token=3)
    got = mxq.beam_select(x, scores, done=done, end_token=3, scores_out=scores, done_out=done)
    assert got[0] is scores and got[3] is done and all(torch.equal(a, b) for a, b in zip(got, want))
    # level candidates, which are found one after the other
    flat, scores = torch.zeros((N * W, 3000), device="cuda"), torch.zeros((N, W), device="cuda")
    done = dev(rng.random((N, W)) < 0.4)
    want = mxq.beam_select(flat, scores, done=done, end_token=3)
    got = mxq.beam_select(flat, scores, done=done, end_token=3, scores_out=scores, done_out=done)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("N", [2, 90])
def test_behind_other_work_of_streams_and_graphs(N):
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(N)
    W, V = 4, 3001
    x, scores = dev(logits(rng, N, W, V).reshape(N * W, V), torch.bfloat16), dev((-rng.random((N, W))).astype(np.float32))
    done = dev(rng.random((N, W)) < 0.3)
    want = mxq.beam_select(x, scores, done=done)
    a, b, d = torch.zeros_like(x), torch.zeros_like(scores), torch.zeros_like(done)
    side = torch.cuda.Stream()

    def both():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            a.copy_(x)
        b.copy_(scores)
        d.copy_(done)
        main.wait_stream(side)
        return mxq.beam_select(a, b, done=d)

    assert all(torch.equal(p, q) for p, q in zip(both(), want))
    for t in (a, b, d):
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both()
        for t in (a, b, d):
            t.zero_()
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    # steps one after the other, each on the scores of the one before, as a stream of dependent kernels
    ref, s, e = [], scores, done
    for i in range(6):
        s, _, _, e = mxq.beam_select(x, s, done=e)
        torch.cuda.synchronize()
        ref.append((s, e))
    s, e = scores.clone(), done.clone()
    steps = []
    for i in range(6):
        mxq.beam_select(x, s, done=e, scores_out=s, done_out=e)
        steps.append((s.clone(), e.clone()))
    assert all(torch.equal(p[0], q[0]) and torch.equal(p[1], q[1]) for p, q in zip(ref, steps))


@pytest.mark.parametrize("N", [2, 90])
def test_two_calls_at_once(N):
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(N)
    data = [(dev(logits(rng, N, 4, 9000).reshape(N * 4, 9000), torch.bfloat16), dev((-rng.random((N, 4))).astype(np.float32))) for _ in range(2)]
    want = [mxq.beam_select(*d) for d in data]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    got = [[mxq.beam_select(*d, stream=s) for d, s in zip(data, streams)] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(p, q) for g, w in zip(pair, want) for p, q in zip(g, w))


def test_logits_near_the_end_of_their_type():
    rng = np.random.default_rng(9)
    for fp32 in (False, True):
        x = logits(rng, 2, 3, 500, fp32)
        x[0, 0, 7] = 2.0 ** 127   # alone on its row: all others have no weight beside it
        x[0, 1, ::3] = -3e38
        x[1, 2] = -2.0 ** 127
        x[1, 2, 5:9] = 2.0 ** 127
        check(x if fp32 else bf16(x), -10 * rng.random((2, 3)), 4, fp32=fp32)
        # rows on which nothing is allowed, by the lowest number of the type or by a very low one
        lowest = -3.4028234663852886e38 if fp32 else -3.3895313892515355e38
        x = logits(rng, 4, 3, 5000, fp32)
        x[0, 1] = x[1] = lowest
        x[2, 0, 17:] = lowest
        x[2, 1] = -1e30
        x[3, 0] = 1e9 + 64 * rng.integers(0, 3, 5000)
        x[3, 1] = 3e37
        for k in (3, 40):
            check(x if fp32 else bf16(x), -10 * rng.random((4, 3)), k, fp32=fp32)


def test_reordering_behind_other_work_of_streams_and_graphs():
    import torch

    import affine_bit_matmul_gb300 as mxq

    c = Case(3, 5, 4, 64, 64, 16, seed=6, lens=[20] * 15)
    parents = c.parents()
    first = torch.from_numpy(c.pages).cuda()
    source = [i32(c.table), i32(c.lens), i32(parents)]
    home = i32(c.home)
    ref = c.pages.copy()
    want = plain(ref, c.table, c.home, c.lens, parents, 64, 64, 16)
    for in_place in (False, True):
        pages = torch.zeros_like(first)
        held = [torch.zeros_like(t) for t in source]
        side = torch.cuda.Stream()

        def both():
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                pages.copy_(first)
                held[0].copy_(source[0])
            held[1].copy_(source[1])
            held[2].copy_(source[2])
            main.wait_stream(side)
            out = dict(table_out=held[0], lens_out=held[1]) if in_place else {}
            return mxq.kv_reorder(pages, held[0], home, held[1], held[2], 64, **out)

        g = torch.cuda.CUDAGraph()
        both()
        with torch.cuda.graph(g):
            t, n = both()
        for _ in range(3):
            pages.zero_()
            t.zero_()
            g.replay()
            assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(n.cpu().numpy(), want[1])
            assert np.array_equal(pages.cpu().numpy(), ref)
