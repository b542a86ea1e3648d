"""Host side of the key/value cache operators: refusals before anything
touches a device, sizes, and the rotation's frequencies (no GPU needed)."""

import ctypes
import math

import numpy as np
import pytest

from tests import kv_util as ku


@pytest.fixture(scope="module")
def L():
    from affine_bit_matmul_gb300 import build

    build.build()
    import affine_bit_matmul_gb300 as mxq

    return mxq.lib()


FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)
ODD2 = ctypes.c_void_p(0x10002)


def rope(L, q=FAKE, k=FAKE, pos=FAKE, f=FAKE, qw=FAKE, kw=FAKE, qo=FAKE, ko=FAKE, T=4, Hq=2, Hk=1, D=128, rot=128,
         qrs=256, qhs=128, krs=128, khs=128):
    return L.mxq_qk_norm_rope(q, qrs, qhs, k, krs, khs, pos, f, qw, kw, qo, 256, 128, ko, 128, 128, T, Hq, Hk, D, rot,
                              0, 1e-6, 0.0, 1.0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(Hq=0, Hk=0), 1), (dict(Hq=-1), 1), (dict(D=0), 1), (dict(D=12), 1), (dict(D=264), 1),
    (dict(rot=8), 1), (dict(rot=144), 1), (dict(rot=-16), 1), (dict(rot=0, qw=None, kw=None), 1),
    (dict(pos=None), 1), (dict(f=None), 1), (dict(q=None), 1), (dict(ko=None), 1), (dict(qrs=4), 1),
    (dict(khs=-8), 1), (dict(q=ODD), 2), (dict(ko=ODD), 2), (dict(qw=ODD), 2), (dict(pos=ODD2), 2), (dict(f=ODD2), 2),
])
def test_rope_argument_checks(L, kw, code):
    assert rope(L, **kw) == code


def append(L, k=FAKE, v=FAKE, pages=FAKE, slots=FAKE, T=4, H=2, D=128, n=8, page=16, G=64, st=None, krs=256, vhs=128):
    return L.mxq_kv_append(k, krs, 128, v, 256, vhs, pages, slots, T, H, D, n, page, G, st, None)


def read(L, pages=FAKE, slots=FAKE, k=FAKE, v=FAKE, T=4, H=2, D=128, n=8, page=16, G=64, st=None):
    return L.mxq_kv_read(pages, slots, k, v, T, H, D, n, page, G, st, None)


SHAPE_FAULTS = [(dict(T=-1), 1), (dict(H=0), 1), (dict(D=96), 1), (dict(D=512), 1), (dict(n=0), 1), (dict(page=48), 1),
                (dict(page=8), 1), (dict(page=256), 1), (dict(G=16), 1), (dict(G=128, D=64), 1), (dict(G=256, D=256), 1)]


@pytest.mark.parametrize("kw,code", SHAPE_FAULTS + [
    (dict(k=None), 1), (dict(slots=None), 1), (dict(krs=12), 1), (dict(vhs=-8), 1), (dict(v=ODD), 2),
    (dict(pages=ODD), 2), (dict(slots=ODD2), 2), (dict(st=ODD2), 2)])
def test_append_argument_checks(L, kw, code):
    assert append(L, **kw) == code


@pytest.mark.parametrize("kw,code", SHAPE_FAULTS + [
    (dict(k=None), 1), (dict(pages=None), 1), (dict(v=ODD), 2), (dict(pages=ODD), 2), (dict(st=ODD2), 2)])
def test_read_argument_checks(L, kw, code):
    assert read(L, **kw) == code


def attend(L, q=FAKE, pages=FAKE, table=FAKE, lens=FAKE, starts=FAKE, out=FAKE, lse=None, T=4, S=2, Hq=8, Hkv=2, D=128,
           n=8, width=4, page=16, G=64, most=3, scale=0.1, window=0, sinks=0, ws=FAKE, wsb=1 << 28, st=None, qrs=1024):
    return L.mxq_kv_attention(q, qrs, 128, pages, table, lens, starts, out, lse, T, S, Hq, Hkv, D, n, width, page, G, most,
                              scale, window, sinks, ws, wsb, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(S=-1), 1), (dict(Hq=7), 1), (dict(Hkv=0), 1), (dict(D=80), 1), (dict(n=0), 1),
    (dict(width=0), 1), (dict(page=20), 1), (dict(G=48), 1), (dict(most=0), 1), (dict(window=-1), 1), (dict(sinks=-1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=0.0), 1), (dict(scale=-0.1), 1), (dict(starts=None), 1),
    (dict(starts=None, T=2, S=2), 1), (dict(q=None), 1), (dict(table=None), 1), (dict(out=None), 1), (dict(qrs=4), 1),
    (dict(width=1 << 30, page=128), 3), (dict(q=ODD), 2), (dict(pages=ODD), 2), (dict(out=ODD), 2), (dict(lse=ODD2), 2),
    (dict(lens=ODD2), 2), (dict(st=ODD2), 2), (dict(ws=ODD), 2), (dict(ws=None), 6), (dict(wsb=64), 6),
])
def test_attention_argument_checks(L, kw, code):
    assert attend(L, **kw) == code


def test_valid_calls_reach_the_device_check(L):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    for rc in (rope(L), rope(L, rot=0), append(L), read(L), attend(L), attend(L, starts=None, T=2, S=2, most=1)):
        assert rc in (4, 5)


def test_sizes(L):
    assert L.mxq_kv_block_bytes(128, 64, 64) == ku.block_bytes(128, 64, 64) == 9216
    for D, G, page in ((64, 32, 16), (256, 128, 128)):
        assert L.mxq_kv_block_bytes(D, page, G) == ku.block_bytes(D, page, G)
    assert L.mxq_kv_block_bytes(128, 24, 64) == 0 and L.mxq_kv_block_bytes(96, 16, 32) == 0
    assert L.mxq_kv_attention_workspace_bytes(4, 4, 8, 3, 128, 1) == 0
    assert L.mxq_kv_attention_workspace_bytes(4, 4, 8, 2, 128, 0) == 0
    assert 0 < L.mxq_kv_attention_workspace_bytes(4, 4, 8, 2, 128, 1)
    # long prompts take no more than the partial results of one block per SM and a list
    assert L.mxq_kv_attention_workspace_bytes(10 ** 6, 4, 64, 1, 256, 10 ** 6) < 1 << 28
    # a bound above the rows there are is as good as their number
    assert (L.mxq_kv_attention_workspace_bytes(40, 4, 8, 2, 128, 10 ** 6) ==
            L.mxq_kv_attention_workspace_bytes(40, 4, 8, 2, 128, 40))


def test_python_refusals():
    import torch

    import affine_bit_matmul_gb300 as mxq

    cpu = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    for call in (lambda: mxq.qk_norm_rope(cpu, cpu, q_weight=cpu[0, 0]),
                 lambda: mxq.kv_append(cpu, cpu, torch.zeros(1, 4, 9216, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)),
                 lambda: mxq.kv_read(torch.zeros(1, 4, 9216, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32), 128),
                 lambda: mxq.kv_attention(cpu, None, None, None)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        mxq.qk_norm_rope([1.0], None)
    with pytest.raises(ValueError):
        mxq.kv_block_bytes(100, 64)


def test_rope_frequencies():
    import affine_bit_matmul_gb300 as mxq

    f, scale = mxq.rope_inv_freq(64)
    want = 10000.0 ** (-np.arange(32) / 32.0)
    assert scale == 1.0 and np.array_equal(f.numpy(), want.astype(np.float32))
    lin, _ = mxq.rope_inv_freq(64, scaling="linear", factor=4.0)
    assert np.array_equal(lin.numpy(), (want / 4).astype(np.float32))
    base, _ = mxq.rope_inv_freq(64, scaling="base", factor=4.0)
    assert base[0] == 1.0 and abs(float(base[-1]) * 4 / want[-1] - 1) < 1e-6
    # bands: turns in 8192 tokens below 1: slowed by 8; above 4: kept; between: in turns
    band, one = mxq.rope_inv_freq(128, 5e5, "bands", 8.0, 8192)
    full = 5e5 ** (-np.arange(64) / 64.0)
    turns = 8192 * full / (2 * math.pi)
    keep = np.clip((turns - 1) / 3, 0, 1)
    assert one == 1.0 and np.allclose(band.numpy(), full * (keep + (1 - keep) / 8), rtol=1e-6)
    assert (keep == 0).any() and (keep == 1).any() and ((keep > 0) & (keep < 1)).any()
    # yarn: the pair that makes 32 turns in 4096 tokens and those before it are kept, the one that
    # makes one turn and those after it are slowed
    yarn, m = mxq.rope_inv_freq(128, 10000.0, "yarn", 16.0, 4096)
    full = 10000.0 ** (-np.arange(64) / 64.0)
    ratio = yarn.numpy() / full
    turns = 4096 * full / (2 * math.pi)
    assert abs(m - (0.1 * math.log(16) + 1)) < 1e-12
    assert np.allclose(ratio[turns > 40], 1) and np.allclose(ratio[turns < 0.8], 1 / 16)
    assert (np.diff(ratio) <= 1e-6).all()
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, scaling="x"), dict(rot_dim=8, factor=0.5),
                dict(rot_dim=8, scaling="bands", factor=2.0), dict(rot_dim=8, scaling="bands", factor=2.0, original_len=9, low=2, high=1)):
        with pytest.raises(ValueError):
            mxq.rope_inv_freq(**bad)
