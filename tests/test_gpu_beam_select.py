"""Selection of beams against float64 and a stable sort: sizes, alignments, level logits, beams
that have ended or are not in use; streams and graphs."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def best_of(x, scores, k, done=None, end=0):
    """x float64 [N, W, V] -> scores, parents, tokens, done; equal ones in the order of w V + v."""
    N, W, V = x.shape
    with np.errstate(all="ignore"):
        m = x.max(-1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        cand = x - m - np.log(np.exp(x - m).sum(-1, keepdims=True)) + scores.astype(np.float64)[..., None]
    cand[~np.isfinite(scores)] = -np.inf
    if done is not None:
        cand[done] = -np.inf
        cand[..., end] = np.where(done & np.isfinite(scores), scores, cand[..., end])
    cand = np.where(np.isnan(cand), -np.inf, cand).reshape(N, W * V)
    at = np.argsort(-cand, axis=1, kind="stable")[:, :k]
    parents, tokens = at // V, at % V
    ended = np.take_along_axis(done, parents, 1) | (tokens == end) if done is not None else None
    return np.take_along_axis(cand, at, 1), parents, tokens, ended


def bf16(x):
    import torch

    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().float().numpy()


def dev(x, dtype=None):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def check(x, scores, k, done=None, end=0, fp32=False, stride=None, **kw):
    """x: float32 [N, W, V], bf16 values where not fp32."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    N, W, V = x.shape
    d = dev(x.reshape(N * W, V).astype(np.float32), torch.float32 if fp32 else torch.bfloat16)
    if stride:
        wide = torch.full((N * W, stride), 99.0, dtype=d.dtype, device="cuda")
        wide[:, :V] = d
        d = wide[:, :V]
    got = mxq.beam_select(d, dev(scores.astype(np.float32)), k, done=None if done is None else dev(done), end_token=end, **kw)
    want = best_of(x.astype(np.float64), scores.astype(np.float32), k, done, end)
    s, parents, tokens = (t.cpu().numpy() for t in got[:3])
    assert np.array_equal(parents, want[1]) and np.array_equal(tokens, want[2])
    # one rounding to fp32, and sums of exponentials within 2^-18 (46 additions and an exponential of 2 units)
    ref, dead = want[0], np.isinf(want[0])
    assert np.array_equal(np.isinf(s) & (s < 0), dead)
    assert (np.abs(s - np.where(dead, 0, ref))[~dead] <= (2.0 ** -24 * np.abs(ref) + 2.0 ** -18)[~dead]).all()
    if done is not None:
        assert np.array_equal(got[3].cpu().numpy(), want[3])
    return got


def logits(rng, N, W, V, fp32=False, spread=2.0):
    x = rng.standard_normal((N, W, V)) * spread + 3 * rng.standard_normal((N, 1, V))
    return x.astype(np.float32) if fp32 else bf16(x)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 255, 2047, 2048, 2049, 4096, 16383, 16384, 50001, 131072])
def test_lengths_of_rows(V, fp32):
    rng = np.random.default_rng(V)
    for N, W, k in ((1, 4, min(4, 4 * V)), (3, 5, min(10, 5 * V))):
        check(logits(rng, N, W, V, fp32), -10 * rng.random((N, W)), k, fp32=fp32)


@pytest.mark.parametrize("N,W,k", [(1, 1, 1), (2, 1, 5), (7, 2, 2), (3, 8, 16), (2, 17, 9), (2, 32, 64), (1, 64, 64), (200, 4, 8), (90, 8, 11), (40, 3, 41)])
def test_beams(N, W, k):
    rng = np.random.default_rng(N * W + k)
    check(logits(rng, N, W, 1000), -10 * rng.random((N, W)), k)


def test_all_chunk_sizes():
    rng = np.random.default_rng(5)
    for N in (1, 20, 40, 80, 160):  # parts of two steps to whole rows, one and two blocks an SM
        for fp32 in (False, True):
            check(logits(rng, N, 4, 33001, fp32), -10 * rng.random((N, 4)), 6, fp32=fp32)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("shift", range(8))
def test_alignments(shift, fp32):
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(shift)
    V = 5003
    x = logits(rng, 2, 3, V, fp32)
    scores = -10 * rng.random((2, 3))
    flat = torch.full((6 * V + 64,), 1e9, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    view = flat[shift:shift + 6 * V].view(6, V)
    view.copy_(dev(x.reshape(6, V)))
    got = mxq.beam_select(view, dev(scores.astype(np.float32)), 5)
    want = best_of(x.astype(np.float64), scores.astype(np.float32), 5)
    assert np.array_equal(got[1].cpu().numpy(), want[1]) and np.array_equal(got[2].cpu().numpy(), want[2])
    # rows with a distance
    check(x, scores, 5, fp32=fp32, stride=V + shift)


def test_level_logits_go_to_the_lowest_token():
    rng = np.random.default_rng(1)
    scores = -10 * rng.random((2, 3))
    for x in (np.zeros((2, 3, 40000)), np.full((2, 3, 700), -5.0), np.where(rng.random((2, 3, 20000)) < 0.5, 1.0, 0.0),
              np.where(rng.random((2, 3, 3000)) < 0.1, 0.0, -0.0)):
        check(x.astype(np.float32), scores, 7)
        check(x.astype(np.float32), scores, 64, fp32=True)


def test_equal_beams_go_to_the_lowest_beam():
    rng = np.random.default_rng(2)
    for V in (1000, 33001):
        x = np.repeat(logits(rng, 3, 1, V), 4, axis=1)
        check(x, np.full((3, 4), -1.5), 8)
        check(x, np.full((3, 4), -1.5), 8, fp32=True, stride=V + 1)


def test_tokens_that_are_not_allowed_and_numbers_that_are_none():
    rng = np.random.default_rng(3)
    x = logits(rng, 6, 3, 900)
    x[0, :, 5:] = -np.inf          # fewer tokens than k
    x[1] = -np.inf                 # none at all
    x[2, 1] = -np.inf              # one beam without
    x[3, 0, 17] = np.nan
    x[3, 1, 800] = np.inf
    x[4, :, 3:] = -np.inf
    x[4, 1] = np.nan
    scores = -10 * rng.random((6, 3))
    scores[5] = [-np.inf, -2.0, np.nan]
    for k in (3, 16, 40):
        check(x, scores, k)
        check(x, scores, k, fp32=True)


def test_first_step_and_ended_beams():
    rng = np.random.default_rng(4)
    x = logits(rng, 5, 4, 3001)
    scores = np.full((5, 4), -np.inf)
    scores[:, 0] = 0.0
    check(x, scores, 8)
    done = rng.random((5, 4)) < 0.5
    done[0] = True
    done[1] = False
    scores = -10 * rng.random((5, 4))
    for end in (0, 2, 3000):
        for k in (4, 8, 30):
            check(x, scores, k, done=done, end=end)
    # more results than there are tokens, among ended beams and beams not in use
    scores[2, 1] = scores[0, 2] = -np.inf
    check(x[:, :, :6], scores, 24, done=done, end=3)
    check(x[:, :, :1], scores, 4, done=done, end=0)


def test_ended_rows_are_not_read():
    x = np.full((1, 2, 500), np.nan, dtype=np.float32)
    x[0, 1] = np.arange(500) * 0.01
    check(bf16(x), np.asarray([[-1.0, -2.0]]), 2, done=np.asarray([[True, False]]), end=7)


def test_large_magnitudes():
    rng = np.random.default_rng(6)
    check(logits(rng, 2, 4, 5000, True, 500.0), -1000 * rng.random((2, 4)), 8, fp32=True)
    check(logits(rng, 2, 4, 5000, True, 1e-4), -1e-3 * rng.random((2, 4)), 8, fp32=True)


def test_shapes_of_arguments_and_outputs():
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(7)
    x = logits(rng, 3, 4, 600)
    scores = dev((-10 * rng.random((3, 4))).astype(np.float32))
    flat = dev(x.reshape(12, 600), torch.bfloat16)
    a = mxq.beam_select(flat, scores)
    b = mxq.beam_select(flat.view(3, 4, 600), scores, 4)
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and a[0].shape == (3, 4)
    outs = [torch.empty_like(t) for t in a]
    c = mxq.beam_select(flat, scores, scores_out=outs[0], parents_out=outs[1], tokens_out=outs[2])
    assert all(p is q for p, q in zip(c, outs)) and all(torch.equal(p, q) for p, q in zip(a, c))
    # every third row of a wider tensor
    wide = flat.view(3, 4, 600).repeat_interleave(3, 1)[:, ::3]
    assert all(torch.equal(p, q) for p, q in zip(a, mxq.beam_select(wide, scores)))
    one = mxq.beam_select(flat[:1].expand(12, 600), scores)  # one row for all beams
    ref = mxq.beam_select(flat[:1].repeat(12, 1), scores)
    assert all(torch.equal(p, q) for p, q in zip(one, ref))
    for bad in (lambda: mxq.beam_select(flat, scores, 65), lambda: mxq.beam_select(flat, scores, 0),
                lambda: mxq.beam_select(flat, scores.view(4, 3)[:, :2]), lambda: mxq.beam_select(flat, scores, done=torch.zeros(3, 4, dtype=torch.bool, device="cuda"), end_token=600),
                lambda: mxq.beam_select(flat.t(), scores), lambda: mxq.beam_select(flat.view(3, 4, 600).transpose(0, 1), scores),
                lambda: mxq.beam_select(flat.view(4, 3, 600), scores), lambda: mxq.beam_select(flat, scores, done_out=outs[0])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mxq.beam_select(flat.half(), scores), lambda: mxq.beam_select(flat, scores.double()),
                lambda: mxq.beam_select(flat, scores, done=torch.zeros(3, 4, dtype=torch.int32, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(mxq.MxqError):
        mxq.beam_select(flat, scores, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert mxq.beam_select(flat[:0], scores[:0])[0].shape == (0, 4)


def test_streams_and_graphs():
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(8)
    data = [(dev(logits(rng, 2, 4, 5000).reshape(8, 5000), torch.bfloat16), dev((-rng.random((2, 4))).astype(np.float32))) for _ in range(2)]
    want = [mxq.beam_select(*d) for d in data]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mxq.beam_select(*data[0], stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))
    graphs = []
    for d in data:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(2):
                out = mxq.beam_select(*d)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), w in zip(graphs, want):
            for t in out:
                t.zero_()
            g.replay()
            assert all(torch.equal(p, q) for p, q in zip(out, w))
