"""The paged 4-bit key/value cache on the GPU: rows written and read back, bit
for bit against the format by index arithmetic."""

import numpy as np
import pytest

from tests import kv_util as ku

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


def dev_bf16(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().bfloat16()


def i32(x):
    import torch

    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def host(t):
    return t.float().cpu().numpy()


def rows(rng, *shape):
    """Rows with channels of different size, a flat group, signed zeros and large values."""
    x = rng.standard_normal(shape) * np.where(rng.random(shape[-1]) < 0.1, 8.0, 1.0)
    x = ku.bf16(x)
    x[0, 0, :32] = 0.75
    x[-1, -1, 32:64] = np.where(np.arange(32) % 2, 0.0, -0.0)
    x[0, -1] = x[0, -1] * np.float32(2.0 ** 90)
    x[-1, 0] = x[-1, 0] * np.float32(2.0 ** -100)
    return x


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("page,T,H", [(16, 1, 1), (16, 37, 3), (32, 33, 2), (64, 65, 1), (128, 131, 2)])
def test_append_and_read_bit_for_bit(D, G, page, T, H):
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(D + G + page + T)
    n_pages = T // page + 3
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    k, v = rows(rng, T, H, D), rows(rng, T, H, D)
    want = ku.Cache(n_pages, H, D, page, G, fill=0xA5)
    want.write(slots, k, v)
    pages = torch.full(want.bytes.shape, 0xA5, dtype=torch.uint8, device="cuda")
    status = i32([-1])
    mxq.kv_append(dev_bf16(k), dev_bf16(v), pages, i32(slots), group_size=G, dev_status=status)
    assert int(status.item()) == 0
    assert np.array_equal(pages.cpu().numpy(), want.bytes)
    ko, vo = mxq.kv_read(pages, i32(slots), D, group_size=G, dev_status=status)
    assert int(status.item()) == 0
    assert np.array_equal(host(ko), ku.bf16(want.k[slots])) and np.array_equal(host(vo), ku.bf16(want.v[slots]))


@pytest.mark.parametrize("T", [5, 700])  # below and above the size from which a warp takes 8 tokens
def test_codes_halfway_next_to_halfway_and_of_every_size(T):
    """Quotients that are halfway between two codes, one unit of the difference's last place from
    it, and values from the smallest to the largest exponents: the codes are those of the
    formula's subtraction and division in binary32."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    H, D, G, page = 2, 128, 32, 16
    rng = np.random.default_rng(T)
    x = rng.integers(0, 31, (2, T, H, D // G, G)).astype(np.float64) / 2  # codes and the halves between
    x[..., 0], x[..., 1] = 0, 15
    scale = rng.choice([1.0, 1.25, 1.5, 1.75], (2, T, H, D // G, 1)) * 2.0 ** rng.integers(-20, 20, (2, T, H, D // G, 1))
    x = x * scale
    low = rng.integers(0, 16, (2, T, H, D // G, 1)) / 2 * scale  # bias -low; tiny values differ from it by low and a bit
    tiny = rng.random(x.shape) < 0.3
    x = np.where(tiny, rng.choice([-1.0, 1.0], x.shape) * 2.0 ** rng.integers(-26, -16, x.shape) * scale, x - low)
    x[..., 0], x[..., 1] = -low[..., 0], 15 * scale[..., 0] - low[..., 0]
    wide = rng.random((2, T, H)) < 0.3
    far = rng.choice([-1.0, 1.0], x.shape) * (1 + rng.random(x.shape)) * 2.0 ** rng.integers(-140, 126, x.shape)
    spread = 2.0 ** rng.integers(-150, 1, (2, T, H, 1, 1))  # some groups all small
    x = np.where(wide[..., None, None], far * np.where(far < 1, spread, 1), x)
    small = rng.random((2, T, H)) < 0.1
    x = np.where(small[..., None, None], rng.integers(-9, 9, x.shape) * 2.0 ** -133.0, x)  # the type's last places
    k, v = (ku.bf16(a.reshape(T, H, D)) for a in x)
    n_pages = T // page + 2
    slots = np.arange(7, 7 + T).astype(np.int32)
    want = ku.Cache(n_pages, H, D, page, G)
    want.write(slots, k, v)
    pages = torch.zeros(want.bytes.shape, dtype=torch.uint8, device="cuda")
    mxq.kv_append(dev_bf16(k), dev_bf16(v), pages, i32(slots), group_size=G)
    assert np.array_equal(pages.cpu().numpy(), want.bytes)


def test_strided_rows_padding_and_bad_slots():
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(5)
    T, H, D, G, page, n_pages = 21, 2, 128, 64, 16, 4
    wide = ku.bf16(rng.standard_normal((T, 4 * H, D)))
    wide_d = dev_bf16(wide)
    k, v = wide_d[:, H:2 * H], wide_d[:, 2 * H:3 * H]
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    slots[3], slots[8], slots[20] = -1, n_pages * page, 2 ** 31 - 1
    good = (slots >= 0) & (slots < n_pages * page)
    want = ku.Cache(n_pages, H, D, page, G)
    want.write(slots[good], wide[good, H:2 * H], wide[good, 2 * H:3 * H])
    pages = torch.zeros(want.bytes.shape, dtype=torch.uint8, device="cuda")
    status = i32([0])
    mxq.kv_append(k, v, pages, i32(slots), group_size=G, dev_status=status)
    assert int(status.item()) == mxq.DEV_BAD_SLOT
    assert np.array_equal(pages.cpu().numpy(), want.bytes)
    ko, vo = mxq.kv_read(pages, i32(slots), D, group_size=G, dev_status=status)
    assert int(status.item()) == mxq.DEV_BAD_SLOT
    assert not host(ko)[~good].any() and not host(vo)[~good].any()
    assert np.array_equal(host(ko)[good], ku.bf16(want.k[slots[good]]))
    # padding alone is no fault
    mxq.kv_append(k[:1], v[:1], pages, i32([-7]), group_size=G, dev_status=status)
    assert int(status.item()) == 0 and np.array_equal(pages.cpu().numpy(), want.bytes)


def test_one_key_for_all_heads_by_a_zero_stride():
    import torch

    import affine_bit_matmul_gb300 as mxq

    rng = np.random.default_rng(6)
    k = ku.bf16(rng.standard_normal((5, 1, 64)))
    pages = torch.zeros(1, 3, ku.block_bytes(64, 16, 32), dtype=torch.uint8, device="cuda")
    kd = dev_bf16(k).expand(5, 3, 64)
    mxq.kv_append(kd, kd, pages, i32(np.arange(5)), group_size=32)
    want = ku.Cache(1, 3, 64, 16, 32)
    want.write(np.arange(5), np.repeat(k, 3, 1), np.repeat(k, 3, 1))
    assert np.array_equal(pages.cpu().numpy(), want.bytes)


def test_no_rows():
    import torch

    import affine_bit_matmul_gb300 as mxq

    pages = torch.zeros(1, 1, ku.block_bytes(128, 16, 64), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    status = i32([9])
    mxq.kv_append(none, none, pages, i32([]), dev_status=status)
    assert int(status.item()) == 0
    ko, vo = mxq.kv_read(pages, i32([]), 128)
    assert ko.shape == (0, 1, 128) and vo.shape == (0, 1, 128)


def test_pages_past_four_gigabytes():
    import torch

    import affine_bit_matmul_gb300 as mxq

    H, D, G, page = 8, 128, 64, 64
    block = ku.block_bytes(D, page, G)
    n_pages = (9 << 29) // (H * block) + 2          # 4.5 GiB
    pages = torch.zeros(n_pages, H, block, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(7)
    k, v = ku.bf16(rng.standard_normal((70, H, D))), ku.bf16(rng.standard_normal((70, H, D)))
    slots = (n_pages - 2) * page + np.arange(70)
    mxq.kv_append(dev_bf16(k), dev_bf16(v), pages, i32(slots), group_size=G)
    want = ku.Cache(2, H, D, page, G)
    want.write(np.arange(70), k, v)
    assert np.array_equal(pages[-2:].cpu().numpy(), want.bytes)
    assert int(pages[:-2].max()) == 0
    ko, vo = mxq.kv_read(pages, i32(slots), D, group_size=G)
    assert np.array_equal(host(ko), ku.bf16(want.k[:70])) and np.array_equal(host(vo), ku.bf16(want.v[:70]))
    # and attention over them: one sequence in the last two pages
    q = ku.bf16(rng.standard_normal((1, H, D)))
    table = np.asarray([[n_pages - 2, n_pages - 1]], dtype=np.int32)
    o = mxq.kv_attention(dev_bf16(q), pages, i32(table), i32([70]), group_size=G)
    ref, _, A, B, E = ku.attention(q, want, [[0, 1]], [70], [0, 1], D ** -0.5)
    assert (np.abs(host(o) - ref) <= ku.tolerance(ref, A, B, E, False)).all()


def layer_calls(mxq, stream, given=False):
    """All four operators on slices of one projection's output; what they return."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(5)
    rows = torch.randn((37, 12, 128), generator=gen, device="cuda").bfloat16()
    q, k, v = rows[:, :8], rows[:, 8:10], rows[:, 10:]
    w = torch.rand(128, generator=gen, device="cuda").bfloat16()
    freq, scale = mxq.rope_inv_freq(64, device="cuda")
    pos, slots = i32(np.arange(37)), i32(np.r_[np.arange(32, 64), np.arange(5)])
    pages = torch.zeros((2, 2, mxq.kv_block_bytes(128, 32, 32)), dtype=torch.uint8, device="cuda")
    empty = dict(device="cuda", dtype=torch.bfloat16)
    out = [torch.empty((37, h, 128), **empty) for h in (8, 2, 2, 2, 8)] if given else [None] * 5
    lse = torch.empty((37, 8), device="cuda") if given else None
    status = i32([7]) if given else None
    qr, kr = mxq.qk_norm_rope(q, k, pos, freq, w, w, weight_offset=1.0, interleaved=True, rope_scale=scale,
                              q_out=out[0], k_out=out[1], stream=stream)
    assert mxq.kv_append(kr, v, pages, slots, group_size=32, dev_status=status, stream=stream) is pages
    k4, v4 = mxq.kv_read(pages, slots, 128, group_size=32, k_out=out[2], v_out=out[3], stream=stream)
    o = mxq.kv_attention(qr, pages, i32([[1, 0]]), i32([37]), i32([0, 37]), 37, group_size=32, window=20, sinks=2,
                         out=out[4], lse=lse, dev_status=status, stream=stream)
    torch.cuda.synchronize()
    if given:
        assert qr is out[0] and kr is out[1] and k4 is out[2] and v4 is out[3] and o is out[4]
        assert int(status.item()) == 0 and bool(lse.isfinite().all())
    return qr, kr, pages, k4, v4, o


def test_the_same_on_a_given_stream_and_with_given_outputs():
    import torch

    import affine_bit_matmul_gb300 as mxq

    first = layer_calls(mxq, None)
    for got in (layer_calls(mxq, None, True), layer_calls(mxq, torch.cuda.current_stream()),
                layer_calls(mxq, torch.cuda.current_stream(), True)):
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_refusals_of_tensors_on_the_device():
    import torch

    import affine_bit_matmul_gb300 as mxq

    q = torch.zeros((4, 8, 128), device="cuda").bfloat16()
    k = torch.zeros((4, 2, 128), device="cuda").bfloat16()
    pages = torch.full((2, 2, mxq.kv_block_bytes(128, 16, 64)), 3, dtype=torch.uint8, device="cuda")
    slots, table, lens = i32([0, 1, 2, 3]), i32([[0], [1], [0], [1]]), i32([1, 1, 1, 1])
    pos, freq = i32([0, 1, 2, 3]), mxq.rope_inv_freq(128, device="cuda")[0]
    one = torch.zeros((4, 1, 128), device="cuda").bfloat16()
    calls = [
        (ValueError, lambda: mxq.qk_norm_rope(q, k[:3], pos, freq)),
        (ValueError, lambda: mxq.qk_norm_rope(q, k, pos[:3], freq)),
        (ValueError, lambda: mxq.qk_norm_rope(q, k, pos.cpu(), freq)),
        (ValueError, lambda: mxq.qk_norm_rope(q, None, pos, freq, k_out=k)),
        (ValueError, lambda: mxq.qk_norm_rope(q, k, pos, freq, q_out=one.expand(4, 8, 128))),
        (TypeError, lambda: mxq.qk_norm_rope(q, k, pos.long(), freq)),
        (TypeError, lambda: mxq.qk_norm_rope(q.float(), k, pos, freq)),
        (ValueError, lambda: mxq.kv_append(k, q, pages, slots)),
        (ValueError, lambda: mxq.kv_append(k, k, pages, slots[:3])),
        (ValueError, lambda: mxq.kv_append(q, q, pages, slots)),
        (ValueError, lambda: mxq.kv_append(k, k, pages, slots, group_size=16)),
        (ValueError, lambda: mxq.kv_append(k.transpose(1, 2).contiguous().transpose(1, 2), k, pages, slots)),
        (TypeError, lambda: mxq.kv_append(k, k, pages.int(), slots)),
        (ValueError, lambda: mxq.kv_read(pages, slots, 96)),
        (ValueError, lambda: mxq.kv_read(pages, slots, 128, k_out=q)),
        (TypeError, lambda: mxq.kv_read(pages, slots.float(), 128)),
        (ValueError, lambda: mxq.kv_attention(q[:3], pages, table, lens)),
        (ValueError, lambda: mxq.kv_attention(q[:, :7], pages, table, lens)),
        (ValueError, lambda: mxq.kv_attention(q, pages, table[0], lens)),
        (ValueError, lambda: mxq.kv_attention(q, pages, table, lens, max_q_len=0)),
        (ValueError, lambda: mxq.kv_attention(q, pages, table, lens, lse=torch.zeros(4, 7, device="cuda"))),
        (TypeError, lambda: mxq.kv_attention(q, pages, table, lens, out=q.float())),
        (RuntimeError, lambda: mxq.kv_attention(q, pages, table, lens, scale=float("nan"))),
        (RuntimeError, lambda: mxq.kv_attention(q, pages, table, lens, window=-1)),
        (RuntimeError, lambda: mxq.kv_attention(q, pages, table, lens,
                                                workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))),
    ]
    for error, f in calls:
        with pytest.raises(error):
            f()
    torch.cuda.synchronize()
    assert bool((pages == 3).all())
