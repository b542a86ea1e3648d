// RMS norm of query and key heads and the rotary position, in one pass.
//
//   n = x * rsqrt(mean(x^2) + eps) * (w + offset)    (n = x without a weight)
//   a_j = position * inv_freq[j],  c = rope_scale cos a_j, s = rope_scale sin a_j
//   (n1, n2) -> (n1 c - n2 s, n2 c + n1 s)
// over the pairs (j, j + R/2) (half layout) or (2 j, 2 j + 1) (interleaved) of
// the first R values of each head; the others keep n.  Everything between the
// bf16 input and the one rounding to bf16 at the end is in fp32.
//
// The angle grows with the position, so position * inv_freq rounded to fp32
// would be wrong by up to 2^-24 of thousands of radians.  It is reduced to a
// fraction of a turn first: the position is split into two exactly held parts,
// each product is kept as a rounded value and its error (one fma), and the
// product with 1 / 2 pi likewise; what is left is below one turn and goes to
// sincospif. 
//
// D / 8 lanes (rounded up to a power of two) hold a head, 8 values each, so that a
// lane has both sides of its pairs: in the half layout 4 values from j on and 4 from
// j + R/2 on, in the interleaved one 8 in a row; either way lane l turns by the
// angles 4 l .. 4 l + 3.  The angles are the same for every head of a token: a warp
// takes one token and several heads and computes each angle once.
// HBM-bound at large sizes, every value being read and written once: 4584 tokens of
// 48 heads of 128 values in 19.5 us (5.8 TB/s) interleaved, 26.0 (4.3 TB/s) in the half
// layout.  Both execute 12 M warp instructions there, and neither fills the issue slots
// (61% and 49% of the cycles) or the memory: the half layout's twice as many loads and stores
// of 8 bytes take 78 registers, so an SM holds 18 warps instead of 27 to wait with.  A
// decode step's rows (16 tokens) take 2.9 us, a launch and three dependent loads.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mxq_device.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kRopeThreads = 256;
// Warps an SM is given before a warp takes more than one round of heads: 512 tokens of 48
// heads take 5.0 us with 16, 6.0 with 32; the largest calls do not care.
constexpr int kWarps = 16;

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Fraction of a turn, in [-0.5, 0.5], of the angle m * f radians; m exact.
__device__ __forceinline__ float turn_of(float m, float f) {
    const float h = 0.15915494f;                    // 1 / (2 pi), rounded to fp32 ...
    const float hl = 6.4206383e-9f;                 // ... and the rest
    const float p = m * f, e = fmaf(m, f, -p);      // m f = p + e exactly
    const float t = p * h;
    const float tl = fmaf(p, h, -t) + fmaf(p, hl, e * h);
    const float r = (t - rintf(t)) + tl;
    return r - rintf(r);
}

__device__ __forceinline__ void cos_sin(int pos, float f, float scale, float* c, float* s) {
    const int lo = pos & 0xFFF;
    float turn = turn_of((float)lo, f) + turn_of((float)(pos - lo), f);
    turn -= rintf(turn);
    sincospif(2.f * turn, s, c);
    *c *= scale;
    *s *= scale;
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

__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// The 8 values of a lane in pairs: half layout, the two sides' values 0..3 as (0, 1),
// (2, 3) each; interleaved, the first and the second of the pairs likewise.  So
// the rotation works on n[0] with n[2] and on n[1] with n[3].
template <bool INTERLEAVED>
__device__ __forceinline__ void pairs_of(const uint4& v, Two (&n)[4]) {
    float f[8];
    unpack8(v, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        constexpr int g = INTERLEAVED ? 2 : 1;
        const int at = INTERLEAVED ? (j & 1) * 4 + (j >> 1) : j * 2;
        n[j] = two_of(f[at], f[at + g]);
    }
}

template <bool INTERLEAVED>
__device__ __forceinline__ uint4 packed(const Two (&n)[4]) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        constexpr int g = INTERLEAVED ? 2 : 1;
        const int at = INTERLEAVED ? (j & 1) * 4 + (j >> 1) : j * 2;
        parts_of(n[j], &f[at], &f[at + g]);
    }
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

template <bool INTERLEAVED>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* row, int at0, int at1) {
    if (INTERLEAVED) return *reinterpret_cast<const uint4*>(row + at0);
    const uint2 a = *reinterpret_cast<const uint2*>(row + at0);
    const uint2 b = *reinterpret_cast<const uint2*>(row + at1);
    return make_uint4(a.x, a.y, b.x, b.y);
}

// LANES: lanes that hold one head (a power of two, at least D / 8).  A round is 32 /
// LANES query or key heads; a warp takes `most` of a token's rounds.
template <int LANES, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const NormRopeParams p, int most,
                                                                    int parts) {
    constexpr int kSide = 32 / LANES;
    // Rounds that are being loaded.  4584 tokens of 48 heads of 128 values: interleaved
    // 20.6, 19.5, 26.6 us with 2, 3, 4; half layout, whose loads are of 8 bytes, 29.6,
    // 27.8, 26.0.  8192 tokens of 20 heads of 256: half layout 33.5, 37.9, 37.0.
    constexpr int kBatch = INTERLEAVED ? 3 : LANES == 32 ? 2 : 4;
    constexpr int kOwn = kSide >= 4 ? 1 : 4 / kSide;  // angles a lane computes
    const int lane = threadIdx.x % LANES, side = (threadIdx.x & 31) / LANES;
    const long long warp = (long long)blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32;
    const int t = (int)(warp / parts);
    if (t >= p.T) return;  // whole warps
    const int first = (int)(warp % parts) * most, last = first + most;
    const int q_rounds = (p.Hq + kSide - 1) / kSide, k_rounds = (p.Hk + kSide - 1) / kSide;
    const bool live = lane * 8 < p.D, turns = lane * 8 < p.rot;
    // this lane's two runs of 4 values
    int at0 = lane * 8, at1 = at0 + 4;
    if (!INTERLEAVED && turns) at0 = lane * 4, at1 = at0 + p.rot / 2;
    const float inv_d = 1.f / (float)p.D;
    Two c[2], s[2], minus_s[2];
    bool angles = p.rot == 0;

#pragma unroll 1
    for (int of_k = 0; of_k < 2; ++of_k) {
        const NormRopeSide& d = of_k ? p.k : p.q;
        const int before = of_k ? q_rounds : 0, n_rounds = of_k ? k_rounds : q_rounds;
        const int r0 = max(first - before, 0), r1 = min(last - before, n_rounds);
        if (r0 >= r1) continue;
        int left = (of_k ? p.Hk : p.Hq) - r0 * kSide - side;  // heads from this lane's on
        const __nv_bfloat16* src =
            d.x + (long long)t * d.row_stride + (long long)(r0 * kSide + side) * d.head_stride;
        __nv_bfloat16* dst = d.out + (long long)t * d.out_row_stride +
                             (long long)(r0 * kSide + side) * d.out_head_stride;
        const long long src_step = kSide * d.head_stride, dst_step = kSide * d.out_head_stride;
        uint4 x[kBatch];
        int ahead = left;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (live && ahead > 0 && r0 + i < r1) x[i] = load8<INTERLEAVED>(src, at0, at1);
            src += src_step;
            ahead -= kSide;
        }
        if (!angles) {
            angles = true;
            float oc[kOwn], os[kOwn], c4[4], s4[4];
            const int pos = __ldg(p.positions + t);
#pragma unroll
            for (int e = 0; e < kOwn; ++e) {
                const int j = lane * 4 + (side * kOwn + e) % 4;
                oc[e] = 1.f, os[e] = 0.f;
                if (turns) cos_sin(pos, __ldg(p.inv_freq + j), p.rope_scale, &oc[e], &os[e]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c4[i] = __shfl_sync(0xFFFFFFFFu, oc[i % kOwn], i / kOwn * LANES + lane);
                s4[i] = __shfl_sync(0xFFFFFFFFu, os[i % kOwn], i / kOwn * LANES + lane);
            }
            c[0] = two_of(c4[0], c4[1]), c[1] = two_of(c4[2], c4[3]);
            s[0] = two_of(s4[0], s4[1]), s[1] = two_of(s4[2], s4[3]);
            minus_s[0] = two_of(-s4[0], -s4[1]), minus_s[1] = two_of(-s4[2], -s4[3]);
        }
        Two w[4];
        if (d.weight && live) {
            pairs_of<INTERLEAVED>(load8<INTERLEAVED>(d.weight, at0, at1), w);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = fma2(w[j], two_of(1.f, 1.f), two_of(p.weight_offset, p.weight_offset));
        }
        for (int round = r0; round < r1; round += kBatch) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (round + i >= r1) break;  // whole warps
                Two n[4];
                pairs_of<INTERLEAVED>(x[i], n);
                // the round after the ones that are being loaded
                if (live && ahead > 0 && round + i + kBatch < r1) x[i] = load8<INTERLEAVED>(src, at0, at1);
                src += src_step;
                ahead -= kSide;
                if (d.weight) {
                    Two sum = mul2(n[0], n[0]);
#pragma unroll
                    for (int j = 1; j < 4; ++j) sum = fma2(n[j], n[j], sum);
                    float ss, other;
                    parts_of(sum, &ss, &other);
                    ss += other;
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                    const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
                    for (int j = 0; j < 4; ++j) n[j] = mul2(mul2(n[j], two_of(r, r)), w[j]);
                }
                if (turns) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const Two a = n[j], b = n[j + 2];
                        n[j] = fma2(a, c[j], mul2(b, minus_s[j]));
                        n[j + 2] = fma2(b, c[j], mul2(a, s[j]));
                    }
                }
                if (live && left > 0) {
                    const uint4 o = packed<INTERLEAVED>(n);
                    if (INTERLEAVED) {
                        *reinterpret_cast<uint4*>(dst + at0) = o;
                    } else {
                        *reinterpret_cast<uint2*>(dst + at0) = make_uint2(o.x, o.y);
                        *reinterpret_cast<uint2*>(dst + at1) = make_uint2(o.z, o.w);
                    }
                }
                dst += dst_step;
                left -= kSide;
            }
        }
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeParams& p, int sms, cudaStream_t stream) {
    const int units = p.D / 8;
    const int lanes = units <= 2 ? 2 : units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32;
    // a warp takes all heads of a token, or a part of them while that leaves less
    // than kWarps warps to an SM
    const int side = 32 / lanes, all = (p.Hq + side - 1) / side + (p.Hk + side - 1) / side;
    const long long even = (long long)p.T * all / (kWarps * (long long)sms);
    const int least = (int)(even < 1 ? 1 : even < all ? even : all);
    const int parts = (all + least - 1) / least, most = (all + parts - 1) / parts;
    const long long warps = (long long)p.T * parts;
    const unsigned grid = (unsigned)((warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32));
#define MXQ_ROPE(L)                                                                    \
    case L:                                                                            \
        if (p.interleaved)                                                             \
            qk_norm_rope_kernel<L, true><<<grid, kRopeThreads, 0, stream>>>(p, most, parts);        \
        else                                                                           \
            qk_norm_rope_kernel<L, false><<<grid, kRopeThreads, 0, stream>>>(p, most, parts);       \
        break;
    switch (lanes) {
        MXQ_ROPE(2)
        MXQ_ROPE(4)
        MXQ_ROPE(8)
        MXQ_ROPE(16)
        MXQ_ROPE(32)
    }
#undef MXQ_ROPE
    return cudaGetLastError();
}

}  // namespace mxq
