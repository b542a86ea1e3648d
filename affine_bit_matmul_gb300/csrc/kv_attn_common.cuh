// Shared by the two attention kernels over the 4-bit cache: what a row tile sees,
// descriptors of its pieces, and small helpers.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_format.cuh"
#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "tc_common.cuh"

namespace mxq {
namespace {

enum : int { kBegins = 1, kEnds = 2 };  // a run's piece holds a row tile's first, last unit

// Descriptor of a run's first or last piece of a row tile (workspace).
struct Seg {
    int row0, toks, head0, heads;
    int flags;  // kBegins, kEnds; -1: none
    int pad[3];
};

// What a row tile of a sequence sees.
struct Span {
    int row0, toks, p0;  // rows of q, tokens, position of the first
    int tiles;           // tiles of tokens (at least 1 when it has rows)
    int head_tiles;      // the first of them, from token 0 on (sinks) ...
    int tail;            // ... and the tile where the rest begins
    int bad;             // the sequence's arguments are out of range
};

template <int TILE>
__device__ __forceinline__ Span span_of(const KvAttnParams& p, int s, int plane) {
    Span r;
    r.bad = 0;
    r.tiles = 0;
    r.head_tiles = 0;
    r.tail = 0;
    int a = s, b = s + 1;
    if (p.q_starts) {
        a = __ldg(p.q_starts + s);
        b = __ldg(p.q_starts + s + 1);
    }
    int len = __ldg(p.ctx_lens + s);
    const int most = p.max_pages * p.page_size;
    if (a < 0 || b > p.T || a > b || b - a > p.max_q || len < 0 || len > most) {
        r.bad = 1;
        if (a < 0 || b > p.T || a > b || b - a > p.max_q) b = a;  // none of its rows
        len = min(max(len, 0), most);
    }
    int n = b - a;
    if (n < p.min_rows || n > p.max_rows) n = 0;  // the other kernel's sequence
    const int j0 = plane * p.tile_toks;
    r.row0 = a + j0;
    r.toks = min(p.tile_toks, n - j0);
    r.p0 = len - n + j0;
    if (r.toks <= 0) return r;
    const int hi = r.p0 + r.toks - 1;           // position of the last row
    const int end = hi < 0 ? 0 : hi / TILE + 1;
    int lo = 0;
    if (p.window) lo = max(0, r.p0 - p.window + 1) / TILE;
    int first = min((min(p.sinks, hi + 1) + TILE - 1) / TILE, end);
    if (first < 0) first = 0;
    if (first >= lo) first = lo = 0;
    lo = min(lo, end);
    r.head_tiles = first;
    r.tail = lo;
    r.tiles = max(1, first + end - lo);
    return r;
}

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Larger of two numbers in each half word.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 2^(e - 127) for a biased exponent 1 <= e <= 254.
__device__ __forceinline__ float pow2_of(int e) { return __uint_as_float((uint32_t)e << 23); }

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Log sum exp of a row: m its largest score times log2 e, l its sum.  -inf for a row that
// sees nothing; not a number where its scores are none.
__device__ __forceinline__ float log_sum_of(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t (&w)[W]) {
    if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {  // slabs of 128 values are 512 bytes apart
            const uint4 v = *reinterpret_cast<const uint4*>(at + 512 * i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
}

template <int NG>
__device__ __forceinline__ void load_pairs(const uint8_t* at, uint32_t (&w)[NG]) {
    if constexpr (NG == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(at);
    } else if constexpr (NG == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < NG / 4; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(at + 16 * i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
}

// Lets a kernel use `bytes` of dynamic shared memory, once per device.
template <typename K>
cudaError_t allow_shared(K* kernel, int bytes, std::atomic<uint64_t>& asked) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (asked.load(std::memory_order_acquire) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess) asked.fetch_or(bit, std::memory_order_release);
    return err;
}

}  // namespace
}  // namespace mxq
