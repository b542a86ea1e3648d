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
// sincospif.  The angles are the same for every head of a token: a CTA takes
// one token (or several, when there are many) and computes them once into
// shared memory.
//
// HBM-bound: every value is read and written once, 16 bytes a lane; D / 8 lanes
// (rounded up to a power of two) hold a head.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mxq_device.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxRot = 256;

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

// LANES: lanes that hold one head (a power of two, at least D / 8).
template <int LANES, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const NormRopeParams p) {
    __shared__ float2 cs[kMaxRot / 2];
    constexpr int kSlots = kRopeThreads / LANES;
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const int heads = p.Hq + p.Hk;
    const int half = p.rot / 2;
    const bool live = lane * 8 < p.D;
    const float inv_d = 1.f / (float)p.D;

    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        if (half) {
            __syncthreads();  // the previous token's angles are no longer read
            const int pos = __ldg(p.positions + t);
            for (int j = threadIdx.x; j < half; j += kRopeThreads)
                cos_sin(pos, __ldg(p.inv_freq + j), p.rope_scale, &cs[j].x, &cs[j].y);
            __syncthreads();
        }
        // every warp runs the same rounds: the shuffles below take whole warps
        for (int h0 = blockIdx.y * kSlots; h0 < heads; h0 += gridDim.y * kSlots) {
            const int h = h0 + slot;
            const bool mine = live && h < heads;
            const bool is_q = h < p.Hq;
            const NormRopeSide& d = is_q ? p.q : p.k;
            const int hh = is_q ? h : h - p.Hq;
            float n[8] = {};
            if (mine) {
                const uint4 v = *reinterpret_cast<const uint4*>(
                    d.x + (long long)t * d.row_stride + (long long)hh * d.head_stride + lane * 8);
                unpack8(v, n);
            }
            if (d.weight) {  // uniform over a head's lanes; a warp may hold q and k heads
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(n[i], n[i], ss);
                const uint32_t group =
                    LANES == 32 ? 0xFFFFFFFFu
                                : ((1u << (LANES & 31)) - 1u) << ((threadIdx.x & 31) / LANES * LANES);
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
                const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
                if (mine) {
                    float w[8];
                    unpack8(__ldg(reinterpret_cast<const uint4*>(d.weight + lane * 8)), w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) n[i] = n[i] * r * (w[i] + p.weight_offset);
                }
            }
            if (half) {
                if (INTERLEAVED) {
                    if (lane * 8 < p.rot) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 a = cs[lane * 4 + i];
                            const float x = n[2 * i], y = n[2 * i + 1];
                            n[2 * i] = fmaf(x, a.x, -y * a.y);
                            n[2 * i + 1] = fmaf(y, a.x, x * a.y);
                        }
                    }
                } else {
                    // lane u of the first half and lane u + R / 16 hold a pair's two sides
                    const int span = p.rot / 16;
                    const bool first = lane < span, turns = lane < 2 * span;
                    const int other = turns ? (first ? lane + span : lane - span) : lane;
                    const int j = (first ? lane : other) * 8;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float y = __shfl_sync(0xFFFFFFFFu, n[i], other, LANES);
                        if (turns) {
                            const float2 a = cs[j + i];
                            n[i] = first ? fmaf(n[i], a.x, -y * a.y) : fmaf(n[i], a.x, y * a.y);
                        }
                    }
                }
            }
            if (mine) {
                uint4 o;
                o.x = pack2(n[0], n[1]);
                o.y = pack2(n[2], n[3]);
                o.z = pack2(n[4], n[5]);
                o.w = pack2(n[6], n[7]);
                *reinterpret_cast<uint4*>(d.out + (long long)t * d.out_row_stride +
                                          (long long)hh * d.out_head_stride + lane * 8) = o;
            }
        }
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeParams& p, int sms, cudaStream_t stream) {
    const int units = p.D / 8;
    const int lanes = units <= 2 ? 2 : units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32;
    const int slots = kRopeThreads / lanes;
    const int rounds = (p.Hq + p.Hk + slots - 1) / slots;
    // few tokens: a CTA takes one round of heads, so that all of a call's
    // loads are in flight at once; many tokens: one CTA takes all heads of a
    // token and the angles are computed once
    const bool few = (long long)p.T * rounds <= 4LL * sms;
    const long long most = 16LL * sms;
    const dim3 grid((unsigned)(p.T < most ? p.T : most), few ? (unsigned)rounds : 1u);
#define MXQ_ROPE(L)                                                                    \
    case L:                                                                            \
        if (p.interleaved)                                                             \
            qk_norm_rope_kernel<L, true><<<grid, kRopeThreads, 0, stream>>>(p);        \
        else                                                                           \
            qk_norm_rope_kernel<L, false><<<grid, kRopeThreads, 0, stream>>>(p);       \
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
