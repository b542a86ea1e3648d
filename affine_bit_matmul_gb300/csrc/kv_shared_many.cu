// The groups' rows over their prefixes on the tensor cores, and the joining of both parts of
// an attention call over shared prefixes.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_many.cuh"

namespace mxq {
namespace {

template <int D, int G>
cudaError_t launch(KvSharedParams& p, cudaStream_t stream) {
    using SH = Shape<D, G>;
    static std::atomic<uint64_t> asked{0};  // devices on which the kernel may take its memory
    cudaError_t err = allow_shared(kv_prefill_kernel<D, G, KvSharedParams>, SH::kSmem, asked);
    if (err != cudaSuccess) return err;
    p.tile_tokens = kTile;
    p.end_units = kEndUnits;
    kv_prefill_kernel<D, G, KvSharedParams><<<(unsigned)p.ctas, kThreads, SH::kSmem, stream>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- joining

// Pieces of a row of one part.
struct Pieces1 {
    long long at;  // floats before the first one's (largest score, sum) of this row
    long long sums;  // ... and before its weighted sum
    int n;
};

__device__ __forceinline__ Pieces1 pieces_of(const KvSharedParams& p, const Item& it, int item, int row,
                                             int head, int D) {
    Pieces1 r;
    r.n = 0;
    r.at = r.sums = 0;
    const long long each = __ldcg(p.totals);
    if (it.planes == 0 || each == 0) return r;
    const int rep = p.Hq / p.Hkv, h = head / rep, part = head % rep / p.part_heads;
    const int hh = head % rep % p.part_heads, heads = min(p.part_heads, rep - part * p.part_heads);
    const int vheads = p.Hkv * p.head_parts, vh = h * p.head_parts + part;
    const int tiles = (it.len + p.tile_tokens - 1) / p.tile_tokens;
    const int2 before = __ldcg(p.before + item);
    const int n = vh * it.planes + row / p.tile_toks;
    const long long u = (long long)before.x * vheads + (long long)n * (tiles + p.end_units);
    const int c0 = (int)(u / each), c1 = (int)((u + tiles - 1) / each);
    const long long stride = (long long)p.tile_rows * (D + 2);
    const int in = row % p.tile_toks * heads + hh;
    r.n = c1 - c0 + 1;
    r.at = ((long long)before.y * vheads + n + c0) * stride + 2 * in;
    r.sums = r.at - 2 * in + 2 * p.tile_rows + (long long)in * D;
    return r;
}

// One warp joins a row of one query head, 32 pieces at a time: lane i takes the weight of piece
// i, then all lanes add the pieces' sums in order.
template <int D>
__global__ void __launch_bounds__(256) kv_shared_join_kernel(const KvSharedParams a, const KvSharedParams b) {
    pdl_wait();
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31, s = blockIdx.x;
    const int head = blockIdx.y * 8 + threadIdx.x / 32;
    if (head >= b.Hq) return;
    const Item own = item_of(b, s);
    if (own.rows == 0) return;
    // its group
    int g = -1;
    if (a.groups) {
        int lo = 0, hi = a.groups_n - 1;  // the last group that starts at or before s
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (__ldg(a.groups + mid) <= s) lo = mid;
            else hi = mid - 1;
        }
        if (__ldg(a.groups + lo) <= s && s < __ldg(a.groups + lo + 1)) g = lo;
    } else {
        g = s / (a.S / a.groups_n);
    }
    Item pre{};
    if (g >= 0) {
        pre = item_of(a, g);
        if (own.row0 < pre.row0 || own.row0 + own.rows > pre.row0 + pre.rows) {
            if (lane == 0) flag_status(a.status, MXQ_DEV_BAD_SEQUENCE);
            return;
        }
    }
    for (int j = 0; j < own.rows; ++j) {
        float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.f;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const KvSharedParams& p = part ? b : a;
            const Pieces1 x = part ? pieces_of(b, own, s, j, head, D)
                                   : pieces_of(a, pre, g, own.row0 + j - pre.row0, head, D);
            const long long stride = (long long)p.tile_rows * (D + 2);
            for (int k0 = 0; k0 < x.n; k0 += 32) {
                float2 ml = make_float2(-INFINITY, 0.f);
                if (k0 + lane < x.n)
                    ml = __ldcg(reinterpret_cast<const float2*>(p.partial + x.at + (k0 + lane) * stride));
                float top = ml.x;
#pragma unroll
                for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
                const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
                const float f = exp2_approx(m - ref), w = exp2_approx(ml.x - ref);
                float sum = ml.y * w;
#pragma unroll
                for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
                m = mn;
                l = fmaf(l, f, sum);
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] *= f;
                const int n = min(32, x.n - k0);
#pragma unroll 4
                for (int k = 0; k < n; ++k) {
                    const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
                    const float* y = p.partial + x.sums + (k0 + k) * stride + lane * V;
                    float v[V];
                    if constexpr (V == 2) {
                        *reinterpret_cast<float2*>(v) = __ldcg(reinterpret_cast<const float2*>(y));
                    } else {
#pragma unroll
                        for (int i = 0; i < V; i += 4)
                            *reinterpret_cast<float4*>(v + i) = __ldcg(reinterpret_cast<const float4*>(y + i));
                    }
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = fmaf(v[i], wk, o[i]);
                }
            }
        }
        const long long to = (long long)(own.row0 + j) * b.Hq + head;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = cvt_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
        __nv_bfloat16* out = b.out + to * D + lane * V;
        if constexpr (V == 2) *reinterpret_cast<uint32_t*>(out) = w[0];
        else if constexpr (V == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
        if (b.lse && lane == 0) b.lse[to] = log_sum_of(m, l);
    }
}

}  // namespace

cudaError_t launch_kv_shared_many(KvSharedParams& p, int D, int G, cudaStream_t stream) {
#define MXQ_KV_SHARED(d, g) \
    if (D == d && G == g) return launch<d, g>(p, stream);
    MXQ_KV_SHARED(64, 32)
    MXQ_KV_SHARED(64, 64)
    MXQ_KV_SHARED(128, 32)
    MXQ_KV_SHARED(128, 64)
    MXQ_KV_SHARED(128, 128)
    MXQ_KV_SHARED(256, 32)
    MXQ_KV_SHARED(256, 64)
    MXQ_KV_SHARED(256, 128)
#undef MXQ_KV_SHARED
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_shared_join(const KvSharedParams& prefix, const KvSharedParams& own, int D,
                                  cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)own.S, (unsigned)(own.Hq + 7) / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return D == 64    ? cudaLaunchKernelEx(&cfg, kv_shared_join_kernel<64>, prefix, own)
           : D == 128 ? cudaLaunchKernelEx(&cfg, kv_shared_join_kernel<128>, prefix, own)
                      : cudaLaunchKernelEx(&cfg, kv_shared_join_kernel<256>, prefix, own);
}

}  // namespace mxq
