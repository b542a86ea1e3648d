// Writing new key and value rows into the pages of a 4-bit cache, and reading
// rows back.
//
// Encoding, per (token, head, group of G values), as mxq_quantize does at 4
// bits: s = bf16(RN(RN(max - min) / 15)), b = bf16(min), q = clamp(rint(RN(RN(x
// - b) / s)), 0, 15), 0 where s == 0; binary32 decisions with IEEE-rounded
// subtraction and division, -0 read as +0.  A read gives bf16(s q + b), one
// rounding.
//
// D / 8 lanes hold one row (token, head, K or V), 8 values each: a group's
// extremes take log2(G / 8) shuffles.  A lane's K codes are one word of the
// page.  A V word mixes two tokens and values 8 apart, so four neighbouring
// lanes exchange their words and each writes two half words.
// HBM-bound at prompt sizes (4 bytes read per value pair, about 1.1 written),
// latency-bound for the rows of a decode step.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_format.cuh"
#include "mxq_device.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kRowThreads = 256;

// Slot -> page and token; false for a row that is skipped.  An entry at or
// past the last slot is reported, a negative one is padding.
__device__ __forceinline__ bool slot_place(const KvRowsParams& p, int t, long long* page, int* tok) {
    const int slot = __ldg(p.slots + t);
    if (slot < 0) return false;
    *page = slot / p.page_size;
    *tok = slot % p.page_size;
    return *page < p.n_pages;
}

__device__ __forceinline__ void report_slot(const KvRowsParams& p, int t) {
    if (p.status && __ldg(p.slots + t) / p.page_size >= p.n_pages)
        atomicOr(p.status, MXQ_DEV_BAD_SLOT);
}

__device__ __forceinline__ float bf16_round(float x) {
    return __bfloat162float(__float2bfloat16_rn(x));
}

template <int D, int G>
__global__ void __launch_bounds__(kRowThreads) kv_append_kernel(const KvRowsParams p) {
    constexpr int kLanes = D / 8;                 // 8, 16 or 32
    constexpr int kRows = kRowThreads / kLanes;   // rows per CTA
    const int lane = threadIdx.x % kLanes;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kLanes;
    const long long rows = 2LL * p.T * p.H;       // (token, head, K or V)
    if (row - threadIdx.x / kLanes + (threadIdx.x & ~31) / kLanes >= rows) return;  // whole warps
    const bool in = row < rows;
    const long long rr = in ? row : rows - 1;
    const int is_v = (int)(rr & 1);
    const int h = (int)((rr >> 1) % p.H);
    const int t = (int)((rr >> 1) / p.H);
    long long page;
    int tok;
    const bool mine = slot_place(p, t, &page, &tok) && in;
    if (!mine && in && lane == 0) report_slot(p, t);

    float x[8] = {};
    if (mine) {
        const __nv_bfloat16* src = is_v ? p.v + (long long)t * p.v_row_stride + (long long)h * p.v_head_stride
                                        : p.k + (long long)t * p.k_row_stride + (long long)h * p.k_head_stride;
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + lane * 8));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    float mn = __int_as_float(0x7f800000), mx = -__int_as_float(0x7f800000);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = __fadd_rn(x[i], 0.f);  // -0 -> +0
        mn = fminf(mn, f);
        mx = fmaxf(mx, f);
    }
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    }
    const float s = bf16_round(__fdiv_rn(__fsub_rn(mx, mn), 15.f));
    const float b = mn;  // a bf16 value already
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float r = 0.f;
        if (s != 0.f) r = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], b), s)), 0.f), 15.f);
        word |= (uint32_t)r << (4 * i);
    }
    // the words of the four lanes whose values are 8, 16 and 24 apart
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __shfl_sync(0xFFFFFFFFu, word, (threadIdx.x & 28) + i);
    if (!mine) return;
    uint8_t* block = p.pages + (page * p.H + h) * (long long)kv_block_bytes(D, G, p.page_size);
    if (is_v) block += kv_block_bytes(D, G, p.page_size) / 2;
    if ((lane & (G / 8 - 1)) == 0) {
        const uint32_t pair = (__float_as_uint(s) >> 16) | (__float_as_uint(b) & 0xFFFF0000u);
        *reinterpret_cast<uint32_t*>(block + kv_code_bytes(D, p.page_size) +
                                     (tok * (D / G) + lane * 8 / G) * 4) = pair;
    }
    if (!is_v) {
        *reinterpret_cast<uint32_t*>(block + kv_k_word(D, tok, lane * 8)) = word;
    } else {
        const int n = lane & 3;  // this lane's values are 32 u + 8 n + 0..7
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * n + e;
            uint32_t half = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) half |= ((w[i] >> (4 * r)) & 15u) << (4 * i);
            *reinterpret_cast<uint16_t*>(block + kv_v_half(D, tok, (lane >> 2) * 32, r)) =
                (uint16_t)half;
        }
    }
}

template <int D, int G>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const KvRowsParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kRows = kRowThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kLanes;
    const long long rows = 2LL * p.T * p.H;
    if (row - threadIdx.x / kLanes + (threadIdx.x & ~31) / kLanes >= rows) return;  // whole warps
    const bool in = row < rows;
    const long long rr = in ? row : rows - 1;
    const int is_v = (int)(rr & 1);
    const int h = (int)((rr >> 1) % p.H);
    const int t = (int)((rr >> 1) / p.H);
    long long page;
    int tok;
    const bool held = slot_place(p, t, &page, &tok);
    if (!held && in && lane == 0) report_slot(p, t);
    uint32_t word = 0, pair = 0;
    if (held) {
        const uint8_t* block =
            p.pages + (page * p.H + h) * (long long)kv_block_bytes(D, G, p.page_size);
        if (is_v) block += kv_block_bytes(D, G, p.page_size) / 2;
        pair = *reinterpret_cast<const uint32_t*>(block + kv_code_bytes(D, p.page_size) +
                                                  (tok * (D / G) + lane * 8 / G) * 4);
        if (!is_v) {
            word = *reinterpret_cast<const uint32_t*>(block + kv_k_word(D, tok, lane * 8));
        } else {
            // half words r = 2 n and 2 n + 1: values 32 u + r + 8 (0..3)
            const int n = lane & 3;
            const uint32_t a = *reinterpret_cast<const uint16_t*>(
                block + kv_v_half(D, tok, (lane >> 2) * 32, 2 * n));
            const uint32_t c = *reinterpret_cast<const uint16_t*>(
                block + kv_v_half(D, tok, (lane >> 2) * 32, 2 * n + 1));
            word = a | (c << 16);
        }
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __shfl_sync(0xFFFFFFFFu, word, (threadIdx.x & 28) + i);
    if (!in) return;
    if (is_v) {
        const int n = lane & 3;
        uint32_t mine = 0;  // value 8 n + r: nibble n of half word r
#pragma unroll
        for (int r = 0; r < 8; ++r)
            mine |= ((w[r >> 1] >> ((r & 1) * 16 + 4 * n)) & 15u) << (4 * r);
        word = mine;
    }
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (held) {
        const float s = __uint_as_float(pair << 16), b = __uint_as_float(pair & 0xFFFF0000u);
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = fmaf(s, (float)((word >> (8 * i)) & 15u), b);
            const float hi = fmaf(s, (float)((word >> (8 * i + 4)) & 15u), b);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[i]) : "f"(hi), "f"(lo));
        }
        o = make_uint4(out[0], out[1], out[2], out[3]);
    }
    __nv_bfloat16* dst = (is_v ? p.v_out : p.k_out) + ((long long)t * p.H + h) * D + lane * 8;
    *reinterpret_cast<uint4*>(dst) = o;
}

}  // namespace

template <typename F>
static cudaError_t by_shape(int D, int G, F&& f) {
#define MXQ_KV_SHAPE(d, g) \
    if (D == d && G == g) return f(std::integral_constant<int, d>(), std::integral_constant<int, g>());
    MXQ_KV_SHAPE(64, 32)
    MXQ_KV_SHAPE(64, 64)
    MXQ_KV_SHAPE(128, 32)
    MXQ_KV_SHAPE(128, 64)
    MXQ_KV_SHAPE(128, 128)
    MXQ_KV_SHAPE(256, 32)
    MXQ_KV_SHAPE(256, 64)
    MXQ_KV_SHAPE(256, 128)
#undef MXQ_KV_SHAPE
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_append(const KvRowsParams& p, int D, int G, cudaStream_t stream) {
    return by_shape(D, G, [&](auto d, auto g) {
        const long long per = kRowThreads / (d / 8);
        const long long grid = (2LL * p.T * p.H + per - 1) / per;
        kv_append_kernel<d, g><<<(unsigned)grid, kRowThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_kv_read(const KvRowsParams& p, int D, int G, cudaStream_t stream) {
    return by_shape(D, G, [&](auto d, auto g) {
        const long long per = kRowThreads / (d / 8);
        const long long grid = (2LL * p.T * p.H + per - 1) / per;
        kv_read_kernel<d, g><<<(unsigned)grid, kRowThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace mxq
