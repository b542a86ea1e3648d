// Writing new key and value rows into the pages of a 4-bit cache, and reading
// rows back.
//
// Encoding, per (token, head, group of G values), as mxq_quantize does at 4
// bits: s = bf16(RN(RN(max - min) / 15)), b = bf16(min), q = clamp(rint(RN(RN(x
// - b) / s)), 0, 15), 0 where s == 0; binary32 decisions with IEEE-rounded
// subtraction and division, -0 read as +0.  A read gives bf16(s q + b), one
// rounding.
//
// D / 8 lanes hold one row (token, head, K or V), 8 values each, and a warp takes
// several tokens of one head: all its loads are issued before anything is done with
// them.  A group's minimum and negated maximum sit in one register, two bf16
// numbers, so log2(G / 8) shuffles give both.
//
// A lane's K codes are one word of the page.  A V word mixes two tokens and values 8
// apart: four neighbouring lanes exchange the bytes of their words (two shuffles)
// and each writes two half words.
//
// Both touch every byte once.  Reading is bound by the memory: 32768 tokens of 8 heads
// of 128 values in 36 us, 4.7 TB/s.  Writing is bound by the instructions that make the
// codes, some 200 for 256 values: 8192 such tokens in 16.7 us, 2.6 TB/s.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_format.cuh"
#include "mxq_device.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kRowThreads = 256;
// Tokens of a warp, when there are kManyWarps such warps for an SM.  With fewer a warp
// takes as many as fill its lanes once: 64 tokens of 8 heads of 128 values are written in
// 1.9 us (3.3 with 8 tokens a warp), 32768 read in 36 (56 with 2).
constexpr int kManyRows = 8;
constexpr int kManyWarps = 8;

// The rows of one warp: tokens t0 .. t0 + ROWS - 1 of one head, keys or values.
struct Rows {
    uint32_t t0;
    int h, is_v;
};

// False for a warp without rows.
template <int ROWS>
__device__ __forceinline__ bool warp_rows(const KvRowsParams& p, Rows* r) {
    const long long w = (long long)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
    const uint32_t groups = ((uint32_t)p.T + ROWS - 1u) / ROWS;
    if (w >= 2LL * groups * p.H) return false;
    const uint32_t rest = (uint32_t)(w >> 1), g = rest / (uint32_t)p.H;
    r->t0 = g * ROWS;
    r->h = (int)(rest - g * (uint32_t)p.H);
    r->is_v = (int)(w & 1);
    return true;
}

// Slot -> page and token; false for a row that is skipped.  An entry at or
// past the last slot is reported, a negative one is padding.
__device__ __forceinline__ bool slot_place(const KvRowsParams& p, int slot, bool reports, long long* page,
                                           int* tok) {
    *page = slot >> p.page_shift;
    *tok = slot & (p.page_size - 1);
    if (slot < 0) return false;
    if (*page < p.n_pages) return true;
    if (reports && p.status) atomicOr(p.status, MXQ_DEV_BAD_SLOT);
    return false;
}

__device__ __forceinline__ float bf16_round(float x) {
    return __bfloat162float(__float2bfloat16_rn(x));
}

__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Between lane n's word with the codes of values 8 n + 0..7 and its two half words
// r = 2 n (low) and 2 n + 1, nibble m of half word r being value 8 m + r.  Each step
// undoes itself, so the way back is the steps in the other order.
__device__ __forceinline__ uint32_t across_lanes(uint32_t w) {  // lane n: byte n of lanes 0..3
    const bool odd = threadIdx.x & 1, up = threadIdx.x & 2;
    w = __byte_perm(w, __shfl_xor_sync(0xFFFFFFFFu, w, 1), odd ? 0x3715 : 0x6240);
    return __byte_perm(w, __shfl_xor_sync(0xFFFFFFFFu, w, 2), up ? 0x3276 : 0x5410);
}

__device__ __forceinline__ uint32_t swap_nibbles(uint32_t w) {  // nibbles 0 1 2 3 -> 0 2 1 3 of both halves
    return (w & 0xF00FF00Fu) | (w & 0x00F000F0u) << 4 | (w & 0x0F000F00u) >> 4;
}

__device__ __forceinline__ uint32_t halves_of(uint32_t w) {
    return __byte_perm(swap_nibbles(across_lanes(w)), 0u, 0x3120);
}

__device__ __forceinline__ uint32_t word_of(uint32_t halves) {
    return across_lanes(swap_nibbles(__byte_perm(halves, 0u, 0x3120)));
}

__device__ __forceinline__ float value_of(uint32_t pair, int odd) {
    return __uint_as_float(odd ? pair & 0xFFFF0000u : pair << 16);
}

__device__ __forceinline__ uint32_t divided_code(float x, float s, float b) {
    return (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x, b), s)), 0.f), 15.f);
}

// Two fp32 numbers in one register pair: one instruction for both.
typedef unsigned long long Two;

__device__ __forceinline__ Two two_of(float a, float b) {
    Two d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ void parts_of(Two x, float* a, float* b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(x));
}

__device__ __forceinline__ Two add2(Two a, Two b) {
    Two d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// NaN if one of them is
__device__ __forceinline__ float abs_max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
    return d;
}

// Of two values, d = x - b and the codes that belong to d * r, r close to 1 / s: code +
// 0x4B400000 as the bits of floats.  *rem is d - code * s, exact: d has 24 bits, the
// product 12, and the difference is at most about s / 2.
__device__ __forceinline__ Two near_codes(uint32_t x, Two minus_b, Two r, Two minus_s, Two* rem) {
    const float whole = 12582912.f;  // 1.5 * 2^23: a sum with it is rounded to an integer
    const Two d = add2(two_of(value_of(x, 0), value_of(x, 1)), minus_b);
    const Two t = fma2(d, r, two_of(whole, whole));
    *rem = fma2(add2(t, two_of(-whole, -whole)), minus_s, d);
    return t;
}

// Codes of 8 values: rint(RN(d / s)) without the divisions.  The nearest integer to
// d * r is the nearest to d / s too where the remainder is below s / 2; where it is
// s / 2 exactly, which happens in every other warp because d and s have few bits, the
// even one of the two is taken.  Where it is so close to s / 2 that RN(d / s) might
// be halfway although d / s is not, or s leaves no room for r or is no number, the
// values are divided after all.
__device__ __forceinline__ uint32_t codes_of(const uint4& v, float s, float b) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    const bool plain = s > 0x1p-100f && s < 0x1p100f;
    const float half = 0.5f * s, sure = half * (1.f - 0x1p-16f);
    uint32_t word = 0;
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    const Two minus_b = two_of(-b, -b), minus_s = two_of(-s, -s), r2 = two_of(r, r);
    float most = 0.f;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        Two rem;
        float lo, hi, t_lo, t_hi;
        parts_of(near_codes(x[i], minus_b, r2, minus_s, &rem), &t_lo, &t_hi);
        parts_of(rem, &lo, &hi);
        most = abs_max3(most, lo, hi);
        word = (word * 16u + __float_as_uint(t_hi)) * 16u + __float_as_uint(t_lo);
    }
    if (!plain || !(most < sure)) {
        bool divides = !plain;
        word = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            Two rem2;
            float rem[2], t[2];
            parts_of(near_codes(x[i], minus_b, r2, minus_s, &rem2), &t[0], &t[1]);
            parts_of(rem2, &rem[0], &rem[1]);
#pragma unroll
            for (int e = 1; e >= 0; --e) {
                uint32_t code = __float_as_uint(t[e]);
                const bool tie = fabsf(rem[e]) == half;
                divides |= !(fabsf(rem[e]) < sure) && !tie;
                if (tie && (code & 1u)) code += rem[e] > 0.f ? 1u : ~0u;
                word = word * 16u + code;
            }
        }
        if (divides) {
            word = 0x3F400000u;
            if (s != 0.f) {
                word = 0;
                uint32_t y[4] = {v.w, v.z, v.y, v.x};
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    word = word << 8 | divided_code(value_of(y[0], 1), s, b) << 4 |
                           divided_code(value_of(y[0], 0), s, b);
                    y[0] = y[1], y[1] = y[2], y[2] = y[3];
                }
                word += 0x3F400000u;
            }
        }
    }
    return word - 0x3F400000u;  // 0x4B400000 * (1 + 16 + ... + 16^7)
}

template <int D, int G, int ROWS>
__global__ void __launch_bounds__(kRowThreads) kv_append_kernel(const KvRowsParams p) {
    constexpr int kLanes = D / 8, kSide = 32 / kLanes, kSteps = ROWS / kSide;
    const int lane = threadIdx.x % kLanes, side = (threadIdx.x & 31) / kLanes;
    Rows w;
    if (!warp_rows<ROWS>(p, &w)) return;
    const __nv_bfloat16* src =
        (w.is_v ? p.v + w.h * p.v_head_stride : p.k + w.h * p.k_head_stride) + lane * 8;
    const long long stride = w.is_v ? p.v_row_stride : p.k_row_stride;
    uint4 x[kSteps];
    int slot[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const uint32_t t = min(w.t0 + i * kSide + side, (uint32_t)p.T - 1u);
        x[i] = __ldg(reinterpret_cast<const uint4*>(src + t * stride));
        slot[i] = __ldg(p.slots + t);
    }
    const int bytes = kv_block_bytes(D, G, p.page_size);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        uint32_t mn = bf16x2_min(bf16x2_min(x[i].x, x[i].y), bf16x2_min(x[i].z, x[i].w));
        uint32_t mx = bf16x2_max(bf16x2_max(x[i].x, x[i].y), bf16x2_max(x[i].z, x[i].w));
        mx ^= 0x80008000u;
        uint32_t ends = bf16x2_min(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
        ends = bf16x2_min(ends, 0x7F807F80u);  // no NaN
#pragma unroll
        for (int o = 1; o < G / 8; o <<= 1)
            ends = bf16x2_min(ends, __shfl_xor_sync(0xFFFFFFFFu, ends, o));
        // -0 -> +0 at both ends: a range of -0 would be stored as a scale of -0
        const float b = __fadd_rn(value_of(ends, 0), 0.f);
        const float range = __fsub_rn(__fadd_rn(-value_of(ends, 1), 0.f), b);
        const float s = bf16_round(__fdiv_rn(range, 15.f));
        const uint32_t word = codes_of(x[i], s, b);
        const uint32_t halves = w.is_v ? halves_of(word) : 0u;
        const uint32_t t = w.t0 + i * kSide + side;
        long long page;
        int tok;
        if (t >= (uint32_t)p.T || !slot_place(p, slot[i], lane == 0 && w.h == 0 && !w.is_v, &page, &tok)) continue;
        uint8_t* block = p.pages + (page * p.H + w.h) * (long long)bytes + (w.is_v ? bytes / 2 : 0);
        if ((lane & (G / 8 - 1)) == 0)
            *reinterpret_cast<uint32_t*>(block + kv_code_bytes(D, p.page_size) +
                                         (tok * (D / G) + lane * 8 / G) * 4) =
                (__float_as_uint(s) >> 16) | (__float_as_uint(b) & 0xFFFF0000u);
        if (!w.is_v) {
            *reinterpret_cast<uint32_t*>(block + kv_k_word(D, tok, lane * 8)) = word;
        } else {
            const int r = 2 * (lane & 3), v0 = (lane >> 2) * 32;
            *reinterpret_cast<uint16_t*>(block + kv_v_half(D, tok, v0, r)) = (uint16_t)halves;
            *reinterpret_cast<uint16_t*>(block + kv_v_half(D, tok, v0, r + 1)) = (uint16_t)(halves >> 16);
        }
    }
}

template <int D, int G, int ROWS>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const KvRowsParams p) {
    constexpr int kLanes = D / 8, kSide = 32 / kLanes, kSteps = ROWS / kSide;
    const int lane = threadIdx.x % kLanes, side = (threadIdx.x & 31) / kLanes;
    Rows w;
    if (!warp_rows<ROWS>(p, &w)) return;
    const int bytes = kv_block_bytes(D, G, p.page_size);
    int slot[kSteps];
    uint32_t code[kSteps], pair[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) slot[i] = __ldg(p.slots + min(w.t0 + i * kSide + side, (uint32_t)p.T - 1u));
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        long long page;
        int tok;
        code[i] = pair[i] = 0;  // a row that is skipped reads as zeros
        if (!slot_place(p, slot[i], lane == 0 && w.h == 0 && !w.is_v, &page, &tok)) continue;
        const uint8_t* block = p.pages + (page * p.H + w.h) * (long long)bytes + (w.is_v ? bytes / 2 : 0);
        pair[i] = *reinterpret_cast<const uint32_t*>(block + kv_code_bytes(D, p.page_size) +
                                                     (tok * (D / G) + lane * 8 / G) * 4);
        if (!w.is_v) {
            code[i] = *reinterpret_cast<const uint32_t*>(block + kv_k_word(D, tok, lane * 8));
        } else {
            const int r = 2 * (lane & 3), v0 = (lane >> 2) * 32;
            const uint32_t lo = *reinterpret_cast<const uint16_t*>(block + kv_v_half(D, tok, v0, r));
            const uint32_t hi = *reinterpret_cast<const uint16_t*>(block + kv_v_half(D, tok, v0, r + 1));
            code[i] = lo | hi << 16;
        }
    }
    __nv_bfloat16* dst = (w.is_v ? p.v_out : p.k_out) + w.h * D + lane * 8;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const uint32_t word = w.is_v ? word_of(code[i]) : code[i];
        const uint32_t t = w.t0 + i * kSide + side;
        if (t >= (uint32_t)p.T) continue;
        const float s = value_of(pair[i], 0), b = value_of(pair[i], 1);
        const uint32_t even = word & 0x0F0F0F0Fu, odd = (word >> 4) & 0x0F0F0F0Fu;
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // 2^23 + code, less 2^23
            const float lo = __uint_as_float(__byte_perm(even, 0x4B000000u, 0x7550 + j)) - 8388608.f;
            const float hi = __uint_as_float(__byte_perm(odd, 0x4B000000u, 0x7550 + j)) - 8388608.f;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[j]) : "f"(fmaf(s, hi, b)), "f"(fmaf(s, lo, b)));
        }
        *reinterpret_cast<uint4*>(dst + (long long)t * p.H * D) = make_uint4(out[0], out[1], out[2], out[3]);
    }
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

// A warp takes 8 tokens of a head when there are enough warps of that size, else as
// many as fill its lanes.
static bool many_rows(const KvRowsParams& p, int sms) {
    return (long long)p.T * p.H * 2 / kManyRows >= kManyWarps * (long long)sms;
}

static unsigned row_blocks(const KvRowsParams& p, int rows) {
    const long long warps = 2LL * (((long long)p.T + rows - 1) / rows) * p.H;
    return (unsigned)((warps + kRowThreads / 32 - 1) / (kRowThreads / 32));
}

cudaError_t launch_kv_append(const KvRowsParams& p, int D, int G, int sms, cudaStream_t stream) {
    return by_shape(D, G, [&](auto d, auto g) {
        constexpr int few = 256 / d;
        if (many_rows(p, sms))
            kv_append_kernel<d, g, kManyRows><<<row_blocks(p, kManyRows), kRowThreads, 0, stream>>>(p);
        else
            kv_append_kernel<d, g, few><<<row_blocks(p, few), kRowThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_kv_read(const KvRowsParams& p, int D, int G, int sms, cudaStream_t stream) {
    return by_shape(D, G, [&](auto d, auto g) {
        constexpr int few = 256 / d;
        if (many_rows(p, sms))
            kv_read_kernel<d, g, kManyRows><<<row_blocks(p, kManyRows), kRowThreads, 0, stream>>>(p);
        else
            kv_read_kernel<d, g, few><<<row_blocks(p, few), kRowThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace mxq
