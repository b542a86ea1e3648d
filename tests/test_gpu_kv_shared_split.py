"""Attention over shared prefixes on the tensor cores: how the SMs are shared between its two kernels goes by the lengths
of the call, whatever its workspace holds."""

import numpy as np
import pytest

from tests import test_gpu_kv_shared as shared
from tests.test_gpu_kv_cache import host, i32
from tests.test_gpu_kv_shared import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def wide():
    shared.WIDE = 200000
    yield
    shared.WIDE = 0


def workspace(case):
    import affine_bit_matmul_gb300 as mxq

    return mxq.kv_attention_shared_workspace_bytes(len(case.q), len(case.own), len(case.prefix), case.q.shape[1], case.cache.H,
                                                   case.q.shape[2], max(case.rows), case.max_group)


def test_any_workspace():
    import torch

    case = Case([3000, 200], [30, 40], [90] * 70, [1] * 70, 8, 2, 128, 64, 64, seed=31)
    want, _ = case.check()
    need = workspace(case)
    gen = torch.Generator(device="cuda").manual_seed(0)
    for fill in (0, 1, 0x7F, 0xFF, None, "of the last call"):
        if fill is None:
            ws = torch.randint(0, 256, (need,), generator=gen, dtype=torch.uint8, device="cuda")
        elif fill != "of the last call":
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        o, _, st = case.run(workspace=ws)
        assert st == 0 and np.array_equal(o, want)
        # the word by which one kernel tells the other of its share does not outlast the call: a replay of a graph
        # would find it before its own
        assert int(ws[8:16].view(torch.int64).item()) == 0


def test_replays_with_other_lengths_in_one_workspace():
    """From nearly all of the GPU for the prefixes to nearly none, and no prefixes or no own tokens at all; two graphs that
    share a workspace in turn."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    lens = [([3000, 2900], 1), ([40, 1], 700), ([0, 0], 500), ([2000, 1000], 0), ([1500, 0], 300)]
    case = Case([3000, 3000], [40, 30], [700] * 70, [1] * 70, 8, 2, 128, 64, 64, seed=32)
    prefix, own = i32([3000, 3000]), i32([700] * 70)
    ws = torch.full((workspace(case),), 0xFF, dtype=torch.uint8, device="cuda")
    status = i32([0])
    graphs, outs = [], []
    for _ in range(2):
        a, kw = case.args(prefix_lens=prefix, ctx_lens=own, workspace=ws, dev_status=status)
        out = torch.zeros_like(case.q_d)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(2):
                mxq.kv_attention_shared(*a, out=out, **kw)
        graphs.append(g)
        outs.append(out)
    want = []
    for p, n in lens:
        case.prefix, case.own = p, [n] * 70
        want.append(case.check(prefix_lens=i32(p), ctx_lens=i32([n] * 70))[0])
    for turn in range(3):
        for (p, n), w in zip(lens, want):
            prefix.copy_(i32(p))
            own.fill_(n)
            for g, out in zip(graphs, outs):
                out.fill_(float("nan"))
                g.replay()
                torch.cuda.synchronize()
                assert np.array_equal(host(out), w) and int(status.item()) == 0
