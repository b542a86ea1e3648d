// The groups' rows over their prefixes on the tensor cores, and the joining of both parts of
// an attention call over shared prefixes.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_many.cuh"

namespace mxq {
namespace {

template <int D, int G>
cudaError_t launch(const KvSharedParams& prefix, const KvSharedParams& own, cudaStream_t stream) {
    using SH = Shape<D, G>;
    static std::atomic<uint64_t> asked{0};  // devices on which the kernel may take its memory
    constexpr auto kernel = kv_prefill_kernel<D, G, KvSharedParams, KvSharedParams>;
    const cudaError_t err = allow_shared(kernel, SH::kSmem, asked);
    if (err != cudaSuccess) return err;
    // its blocks are placed while what comes before finishes
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)prefix.sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = SH::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, prefix, own);
}

// ---------------------------------------------------------------- joining

// Pieces of a row of one part.
struct RowPieces {
    long long at;    // floats before the first one's (largest score, sum) of this row
    long long sums;  // ... and before its weighted sum
    int n;
    int twice;       // 1: two for each place, the second of them 128 rows later
};

__device__ __forceinline__ RowPieces pieces_of(const KvSharedParams& p, const Before& b, long long run, int row,
                                               int head, int D) {
    RowPieces r;
    r.n = r.twice = 0;
    r.at = r.sums = 0;
    if (b.item_planes == 0 || run == 0) return r;
    const int rep = p.Hq / p.Hkv, h = head / rep, part = head % rep / p.part_heads;
    const int hh = head % rep % p.part_heads, heads = min(p.part_heads, rep - part * p.part_heads);
    const int vheads = p.Hkv * p.head_parts, vh = h * p.head_parts + part;
    const int tiles = (b.len + (1 << p.tile_shift) - 1) >> p.tile_shift;
    const int flat = row * heads + hh, plane = flat / p.tile_rows, in = flat - plane * p.tile_rows;
    const int n = vh * b.item_planes + plane;
    const long long u = (long long)b.units * vheads + (long long)n * (tiles + p.end_units);
    // (most often they fit 32 bits, and the divisions are short)
    const bool large = (u + tiles) >> 32 != 0;
    const int c0 = large ? (int)(u / run) : (int)((unsigned)u / (unsigned)run);
    const int c1 = large ? (int)((u + tiles - 1) / run) : (int)((unsigned)(u + tiles - 1) / (unsigned)run);
    const long long stride = (long long)p.tile_rows * (D + 2);
    r.twice = p.on_tensor_cores && p.tile_rows == 256 && b.rows * heads - plane * 256 <= 128;
    r.n = (c1 - c0 + 1) << r.twice;
    r.at = ((long long)b.planes * vheads + n + c0) * stride + 2 * in;
    r.sums = r.at - 2 * in + 2 * p.tile_rows + (long long)in * D;
    return r;
}

__device__ __forceinline__ Before before_of(const KvSharedParams& p, int i) {
    const int4* at = reinterpret_cast<const int4*>(p.before + i);
    const int4 x = __ldcg(at), y = __ldcg(at + 1);
    return Before{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}

// One warp joins a row of one query head, 32 pieces at a time, those of the prefix before those of
// the own tokens: lane i takes the weight of piece i, then all lanes add the pieces' sums in order.
//   A chain of loads: what comes before the item, the pieces' maxima, the sums.  7 us of a call with 64 rows of 32
// heads, 4 of them until the kernel before has ended for it too; 25 us for 256 rows with 34 MB of pieces, which are
// in L2.
template <int D>
__global__ void __launch_bounds__(256) kv_shared_join_kernel(const __grid_constant__ KvSharedParams a,
                                                             const __grid_constant__ KvSharedParams b) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31, s = blockIdx.x;
    const int head = blockIdx.y * 8 + threadIdx.x / 32;
    pdl_wait();
    if (s == 0 && head == 0 && blockIdx.z == 0) a.totals[1] = 0;  // (see say_sms)
    if (head >= b.Hq) return;
    const long long prefix_run = __ldcg(a.totals), own_run = __ldcg(b.totals);
    const Before own = before_of(b, s);
    // (without a list of groups this does not wait for `own`)
    const int g = a.groups ? own.group : s / (a.S / a.groups_n);
    Before pre{};
    if (g >= 0) pre = before_of(a, g);
    if ((int)blockIdx.z >= own.rows) return;
    if (g >= 0) {
        if (own.row0 < pre.row0 || own.row0 + own.rows > pre.row0 + pre.rows) {
            if (lane == 0) flag_status(a.status, MXQ_DEV_BAD_SEQUENCE);
            return;
        }
    }
    for (int j = blockIdx.z; j < own.rows; j += gridDim.z) {
        const RowPieces x = pieces_of(a, pre, prefix_run, own.row0 + j - pre.row0, head, D);
        const RowPieces y = pieces_of(b, own, own_run, j, head, D);
        const long long x_stride = (long long)a.tile_rows * (D + 2), y_stride = (long long)b.tile_rows * (D + 2);
        const int n = x.n + y.n;
        float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.f;
        for (int k0 = 0; k0 < n; k0 += 32) {
            const int mine = k0 + lane, many = min(32, n - k0);
            float2 ml = make_float2(-INFINITY, 0.f);
            if (mine < n)
                ml = __ldcg(reinterpret_cast<const float2*>(mine < x.n ? a.partial + x.at + (mine >> x.twice) * x_stride + (mine & x.twice) * 256
                                                                       : b.partial + y.at + (mine - x.n) * y_stride));
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
#pragma unroll 16
            for (int k = 0; k < many; ++k) {
                const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
                if (wk == 0.f) continue;  // (of a half without units there is no sum)
                const int at = k0 + k;
                const float* from = (at < x.n ? a.partial + x.sums + (at >> x.twice) * x_stride + (at & x.twice) * (128 * D)
                                              : b.partial + y.sums + (at - x.n) * y_stride) + lane * V;
                float v[V];
                if constexpr (V == 2) {
                    *reinterpret_cast<float2*>(v) = __ldcg(reinterpret_cast<const float2*>(from));
                } else {
#pragma unroll
                    for (int i = 0; i < V; i += 4)
                        *reinterpret_cast<float4*>(v + i) = __ldcg(reinterpret_cast<const float4*>(from + i));
                }
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = fmaf(v[i], wk, o[i]);
            }
        }
        const long long to = (long long)(own.row0 + j) * b.Hq + head;
        const float inv = l > 0.f ? 1.f / l : l;  // (0, or not a number)
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

size_t kv_shared_before_bytes() { return sizeof(Before); }

cudaError_t launch_kv_shared_many(const KvSharedParams& prefix, const KvSharedParams& own, int D, int G,
                                  cudaStream_t stream) {
#define MXQ_KV_SHARED(d, g) \
    if (D == d && G == g) return launch<d, g>(prefix, own, stream);
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
    cfg.gridDim = dim3((unsigned)own.S, (unsigned)(own.Hq + 7) / 8, (unsigned)(own.max_q < 64 ? own.max_q : 64));
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
