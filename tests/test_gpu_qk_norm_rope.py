"""The norm of query and key heads with the rotary position against float64."""

import numpy as np
import pytest

from tests import kv_util as ku
from tests.test_gpu_kv_cache import dev_bf16, host, i32

pytestmark = pytest.mark.gpu


def reference(x, w, positions, inv_freq, interleaved, eps, offset, rope_scale):
    n = x.astype(np.float64)
    if w is not None:
        n = n / np.sqrt((n * n).mean(-1, keepdims=True) + eps) * (w.astype(np.float64) + offset)
    size = np.abs(n)
    if inv_freq is not None:
        half = len(inv_freq)
        j = np.arange(half)
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        angle = positions.astype(np.float64)[:, None, None] * inv_freq.astype(np.float64)
        c, s = np.cos(angle) * rope_scale, np.sin(angle) * rope_scale
        out, size = n.copy(), size.copy()
        out[..., a], out[..., b] = n[..., a] * c - n[..., b] * s, n[..., b] * c + n[..., a] * s
        both = (np.abs(n[..., a]) + np.abs(n[..., b])) * abs(rope_scale)
        size[..., a], size[..., b] = both, both
        n = out
    return n, size


def check(got, ref, size):
    # one rounding to bf16 of the result, fp32 arithmetic (sums of up to 256 squares in a tree,
    # sines and cosines to a few units of 2^-24 of one) on terms of at most `size`
    err = np.abs(host(got).astype(np.float64) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * size + 1e-38).all()


def freq(rot, theta=10000.0):
    return (theta ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32)


@pytest.mark.parametrize("D,rot", [(8, 0), (16, 16), (64, 64), (80, 32), (96, 96), (128, 128), (128, 64), (128, 16),
                                   (192, 176), (256, 256), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (3, 5, 1), (70, 7, 3)])
def test_shapes(D, rot, interleaved, T, Hq, Hk):
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(D + rot + T)
    q, k = ku.bf16(rng.standard_normal((T, Hq, D)) * 3), ku.bf16(rng.standard_normal((T, Hk, D)) * 0.1)
    qw, kw = ku.bf16(1 + 0.3 * rng.standard_normal(D)), ku.bf16(0.3 * rng.standard_normal(D))
    pos = rng.integers(-5, 4000, T).astype(np.int32)
    f = freq(rot) if rot else None
    f_d = torch.from_numpy(f).cuda() if rot else None
    for wq, wk, offset in ((qw, kw, 0.0), (None, kw, 1.0), (qw, None, 0.25)) + (((None, None, 0.0),) if rot else ()):
        qo, ko = mxq.qk_norm_rope(dev_bf16(q), dev_bf16(k), i32(pos), f_d, None if wq is None else dev_bf16(wq),
                                  None if wk is None else dev_bf16(wk), eps=1e-5, weight_offset=offset,
                                  interleaved=interleaved, rope_scale=1.25)
        check(qo, *reference(q, wq, pos, f, interleaved, 1e-5, offset, 1.25))
        check(ko, *reference(k, wk, pos, f, interleaved, 1e-5, offset, 1.25))


@pytest.mark.parametrize("theta", [10000.0, 5e6])
def test_far_positions(theta):
    # the angle's error does not grow with the position
    import torch

    import affine_bit_matmul_gb300 as mxq

    pos = np.asarray([0, 1, 4095, 4096, 131071, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, -1, -(2 ** 31)], dtype=np.int32)
    rng = np.random.default_rng(1)
    q = ku.bf16(rng.standard_normal((len(pos), 2, 128)))
    f = freq(128, theta)
    qo, ko = mxq.qk_norm_rope(dev_bf16(q), None, i32(pos), torch.from_numpy(f).cuda())
    assert ko is None
    check(qo, *reference(q, None, pos, f, False, 0.0, 0.0, 1.0))


def test_many_tokens_slices_and_in_place():
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(2)
    T, Hq, Hk, D = 5000, 6, 2, 128
    qkv = ku.bf16(rng.standard_normal((T, Hq + 2 * Hk, D)))
    w = ku.bf16(1 + 0.2 * rng.standard_normal(D))
    pos = (np.arange(T) + 77).astype(np.int32)
    f = freq(D)
    d = dev_bf16(qkv)
    q, k = d[:, :Hq], d[:, Hq:Hq + Hk]
    args = (i32(pos), torch.from_numpy(f).cuda(), dev_bf16(w), dev_bf16(w))
    qo, ko = mxq.qk_norm_rope(q, k, *args)
    check(qo, *reference(qkv[:, :Hq], w, pos, f, False, 1e-6, 0.0, 1.0))
    check(ko, *reference(qkv[:, Hq:Hq + Hk], w, pos, f, False, 1e-6, 0.0, 1.0))
    mxq.qk_norm_rope(q, k, *args, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert np.array_equal(host(d[:, Hq + Hk:]), qkv[:, Hq + Hk:])


def test_zero_rows_of_values_and_no_tokens():
    import torch

    import affine_bit_matmul_gb300 as mxq

    z = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    qo, _ = mxq.qk_norm_rope(z, None, q_weight=w)
    assert not host(qo).any()
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    qo, ko = mxq.qk_norm_rope(none, none, q_weight=w, k_weight=w)
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 2, 64)


def test_memory_for_a_call_on_another_stream():
    """What a call on a stream allocates is not what was just freed on the current one, which
    may still be at work there."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    q = torch.randn((1024, 8, 128), device="cuda").bfloat16()
    w = torch.ones(128, device="cuda").bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    freed = torch.empty_like(q)
    at = freed.data_ptr()
    del freed
    got, _ = mxq.qk_norm_rope(q, None, q_weight=w, stream=s)
    torch.cuda.synchronize()
    assert got.data_ptr() != at
    assert torch.equal(got, mxq.qk_norm_rope(q, None, q_weight=w)[0])
