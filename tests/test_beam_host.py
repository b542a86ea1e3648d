"""Host side of the operators for several continuations of a prompt: refusals before anything
touches a device, and sizes (no GPU needed)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from affine_bit_matmul_gb300 import build

    build.build()
    import affine_bit_matmul_gb300 as mxq

    return mxq.lib()


FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced
OTHER = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10008)
ODD2 = ctypes.c_void_p(0x10002)
ODD1 = ctypes.c_void_p(0x10001)


def attend(L, q=FAKE, pages=FAKE, ptable=FAKE, plens=FAKE, groups=FAKE, table=FAKE, lens=FAKE, starts=FAKE, out=FAKE, lse=None,
           T=6, S=4, N=2, Hq=8, Hkv=2, D=128, n=8, pwidth=4, width=4, page=16, G=64, most=3, group=4, scale=0.1, ws=FAKE,
           wsb=1 << 28, st=None, qrs=1024):
    return L.mxq_kv_attention_shared(q, qrs, 128, pages, ptable, plens, groups, table, lens, starts, out, lse, T, S, N, Hq, Hkv, D, n,
                                     pwidth, width, page, G, most, group, scale, ws, wsb, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(S=-1), 1), (dict(N=0), 1), (dict(N=-1), 1), (dict(Hq=7), 1), (dict(Hkv=0), 1), (dict(D=80), 1), (dict(n=0), 1),
    (dict(width=0), 1), (dict(pwidth=0), 1), (dict(page=20), 1), (dict(G=48), 1), (dict(G=128, D=64), 1), (dict(most=0), 1),
    (dict(group=0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=0.0), 1), (dict(scale=-0.1), 1),
    (dict(starts=None), 1), (dict(groups=None, N=3), 1), (dict(groups=None, group=1), 1), (dict(q=None), 1), (dict(ptable=None), 1),
    (dict(plens=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(pages=None), 1), (dict(qrs=4), 1),
    (dict(width=1 << 30, page=128), 3), (dict(pwidth=1 << 30, page=128), 3), (dict(q=ODD), 2), (dict(pages=ODD), 2), (dict(out=ODD), 2),
    (dict(lse=ODD2), 2), (dict(lens=ODD2), 2), (dict(plens=ODD2), 2), (dict(groups=ODD2), 2), (dict(ptable=ODD2), 2), (dict(st=ODD2), 2),
    (dict(ws=ODD), 2), (dict(ws=None), 6), (dict(wsb=64), 6),
    # more units than 32 bits count
    (dict(T=1 << 20, S=1 << 20, width=1 << 20, group=8, wsb=1 << 62), 3), (dict(Hq=8 << 16, wsb=1 << 62), 3), (dict(T=1 << 22, S=1 << 22, N=1 << 20, pwidth=1 << 20, wsb=1 << 62), 3)])
def test_shared_attention_argument_checks(L, kw, code):
    assert attend(L, **kw) == code


def select(L, x=FAKE, scores=FAKE, done=None, so=FAKE, po=FAKE, to=FAKE, do=None, N=2, W=4, V=1000, K=4, end=0, stride=1000, fp32=0,
           ws=FAKE, wsb=1 << 28):
    return L.mxq_beam_select(x, stride, fp32, scores, done, so, po, to, do, N, W, V, K, end, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), 1), (dict(W=0), 1), (dict(W=65), 1), (dict(V=0), 1), (dict(V=-3), 1), (dict(K=0), 1), (dict(K=65), 1),
    (dict(W=2, V=3, K=7, stride=3), 1), (dict(stride=-1), 1), (dict(done=FAKE, end=-1), 1), (dict(done=FAKE, end=1000), 1),
    (dict(do=FAKE, end=1000), 1), (dict(x=None), 1), (dict(scores=None), 1), (dict(so=None), 1), (dict(po=None), 1), (dict(to=None), 1),
    (dict(x=ODD1), 2), (dict(x=ODD2, fp32=1), 2), (dict(scores=ODD2), 2), (dict(so=ODD2), 2), (dict(po=ODD2), 2), (dict(to=ODD2), 2),
    (dict(ws=ODD), 2), (dict(W=64, V=1 << 25), 3), (dict(ws=None), 6), (dict(wsb=64), 6),
    # results in the place of scores, or ends, of another number of beams
    (dict(K=2), 1), (dict(K=2, so=OTHER, done=FAKE, do=FAKE), 1)])
def test_select_argument_checks(L, kw, code):
    assert select(L, **kw) == code


def reorder(L, pages=FAKE, table=FAKE, home=OTHER, lens=FAKE, parents=OTHER, to=FAKE, lo=FAKE, S=8, W=4, layers=2, n=32, H=2, D=128,
            width=4, page=16, G=64, ws=FAKE, wsb=1 << 20, st=None):
    return L.mxq_kv_reorder(pages, table, home, lens, parents, to, lo, S, W, layers, n, H, D, width, page, G, ws, wsb, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-4), 1), (dict(S=7), 1), (dict(W=0), 1), (dict(W=65, S=65), 1), (dict(layers=0), 1), (dict(n=0), 1), (dict(H=0), 1),
    (dict(D=96), 1), (dict(width=0), 1), (dict(page=48), 1), (dict(G=16), 1), (dict(pages=None), 1), (dict(table=None), 1),
    (dict(home=None), 1), (dict(lens=None), 1), (dict(parents=None), 1), (dict(to=None), 1), (dict(lo=None), 1), (dict(to=OTHER), 1),
    (dict(lo=OTHER), 1), (dict(pages=ODD), 2), (dict(table=ODD2), 2), (dict(home=ODD2), 2), (dict(st=ODD2), 2), (dict(ws=ODD), 2),
    (dict(width=1 << 30, page=128), 3), (dict(ws=None), 6), (dict(wsb=64), 6)])
def test_reorder_argument_checks(L, kw, code):
    assert reorder(L, **kw) == code


def test_valid_calls_reach_the_device_check(L):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    for rc in (attend(L), attend(L, groups=None), attend(L, starts=None, T=4, most=1), attend(L, T=0), select(L), select(L, N=0),
               select(L, done=FAKE, do=FAKE, x=ODD2), select(L, fp32=1, stride=0), reorder(L), reorder(L, S=0)):
        assert rc in (4, 5)


def test_sizes(L):
    w = L.mxq_kv_attention_shared_workspace_bytes
    assert w(8, 8, 2, 8, 3, 128, 1, 4) == 0 and w(8, 8, 0, 8, 2, 128, 1, 4) == 0 and w(8, 8, 2, 8, 2, 128, 1, 0) == 0
    # a place for each warp's piece
    assert 0 < w(8, 8, 2, 8, 2, 128, 1, 4) < 1 << 25
    # bounds above what there is are as good as that
    assert w(8, 8, 2, 8, 2, 128, 1, 8) == w(8, 8, 2, 8, 2, 128, 1, 10 ** 6)
    # a thousand sequences of 32 heads: less than four times their output in 32 bits, a tile for each processor and each warp
    assert w(1000, 1000, 10, 32, 8, 128, 1, 100) < 4 * 1000 * 32 * 130 * 4 + 160 * (256 + 16 * 16) * 130 * 4
    s = L.mxq_beam_select_workspace_bytes
    assert s(2, 65, 10, 4, 0) == 0 and s(2, 4, 0, 4, 0) == 0 and s(0, 4, 10, 4, 0) >= 0
    assert 0 < s(64, 8, 131072, 8, 0) < 1 << 20
    assert L.mxq_kv_reorder_workspace_bytes(-1) == 0 and L.mxq_kv_reorder_workspace_bytes(100) >= 1600


def test_python_refusals():
    import torch

    import affine_bit_matmul_gb300 as mxq

    cpu = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    ints = torch.zeros(2, 4, dtype=torch.int32)
    for call in (lambda: mxq.kv_attention_shared(cpu, torch.zeros(1, 4, 9216, dtype=torch.uint8), ints, ints[0], ints, ints[0]),
                 lambda: mxq.beam_select(torch.zeros(8, 10), torch.zeros(2, 4)),
                 lambda: mxq.kv_reorder(torch.zeros(1, 4, 9216, dtype=torch.uint8), ints, ints, ints[0], ints, 128)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        mxq.beam_select([[1.0]], None)
