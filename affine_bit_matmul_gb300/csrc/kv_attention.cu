// Attention of a few query rows over a paged 4-bit key/value cache: the launches of
// kv_few.cuh's kernel, and the joining of row tiles that its runs cut.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_few.cuh"

namespace mxq {
namespace {

// Joins the pieces of the row tiles that were cut: the CTA whose last piece
// begins one is followed by those that go on with it, in order.  One CTA a row
// tile; its threads share the pieces out and add their sums in a fixed order.  Bound by
// three dependent loads (who follows, their maxima, their sums): 5.7 us for 304 pieces,
// of which the launch beside the first kernel's end hides a part.
constexpr int kJoinThreads = 512;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const KvAttnParams p, int tile_rows) {
    extern __shared__ float weight[];        // [piece][row]: 2^(max - overall max)
    __shared__ float4 sums[kJoinThreads];
    __shared__ float row_inv[16], row_lse[16];
    __shared__ int last_piece;
    pdl_wait();
    const int cta = blockIdx.x;
    const Seg* segs = reinterpret_cast<const Seg*>(p.segs);
    const Seg g = segs[cta * 2 + 1];
    if (g.flags < 0 || !(g.flags & kBegins) || (g.flags & kEnds)) return;
    // after a wait that gave up the descriptors may be anything
    if (g.toks <= 0 || g.heads <= 0 || g.toks > tile_rows || g.heads > tile_rows ||
        g.toks * g.heads > tile_rows || g.row0 < 0 || g.row0 > p.T - g.toks || g.head0 < 0 ||
        g.head0 > p.Hq - g.heads)
        return;
    const int tid = threadIdx.x;
    if (tid == 0) last_piece = p.ctas - 1;
    __syncthreads();
    for (int c = cta + 1 + tid; c < p.ctas; c += kJoinThreads) {
        const int f = segs[c * 2].flags;
        if (f < 0 || (f & kEnds)) {
            atomicMin(&last_piece, c);
            break;
        }
    }
    __syncthreads();
    const int rows = g.toks * g.heads, n = last_piece - cta + 1;
    const long long stride = (long long)tile_rows * (D + 2);
    // piece 0 is the CTA's second, piece k the first of CTA cta + k
    auto piece = [&](int k) {
        return p.partial + ((cta + k) * 2LL + (k ? 0 : 1)) * stride;
    };
    for (int i = tid; i < n * rows; i += kJoinThreads)
        weight[i] = piece(i / rows)[2 * (i % rows)];
    __syncthreads();
    const int lane = tid & 31;
    for (int row = tid / 32; row < rows; row += kJoinThreads / 32) {
        float mm = -INFINITY;
        for (int k = lane; k < n; k += 32) mm = fmaxf(mm, weight[k * rows + row]);
#pragma unroll
        for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
        const float ref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        for (int k = lane; k < n; k += 32) {
            const float f = exp2_approx(weight[k * rows + row] - ref);
            weight[k * rows + row] = f;
            ll = fmaf(piece(k)[2 * row + 1], f, ll);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) ll += __shfl_xor_sync(0xFFFFFFFFu, ll, o);
        if (lane == 0) {
            row_inv[row] = ll > 0.f ? 1.f / ll : 0.f;
            row_lse[row] = log_sum_of(mm, ll);
        }
    }
    __syncthreads();
    const int items = rows * (D / 4);                           // of 4 values
    const int parts = items < kJoinThreads ? kJoinThreads / items : 1;
    for (int i0 = 0; i0 < items; i0 += kJoinThreads) {
        const int part = parts > 1 ? tid / items : 0, i = parts > 1 ? tid % items : i0 + tid;
        const bool mine = part < parts && i < items;
        const int row = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mine) {
#pragma unroll 8
            for (int k = part; k < n; k += parts) {
                const float4 y =
                    *reinterpret_cast<const float4*>(piece(k) + 2 * tile_rows + row * D + d);
                const float f = weight[k * rows + row];
                o.x = fmaf(y.x, f, o.x);
                o.y = fmaf(y.y, f, o.y);
                o.z = fmaf(y.z, f, o.z);
                o.w = fmaf(y.w, f, o.w);
            }
        }
        if (parts > 1) {
            sums[tid] = o;
            __syncthreads();
            if (part == 0)
                for (int k = 1; k < parts; ++k) {
                    const float4 y = sums[k * items + i];
                    o.x += y.x;
                    o.y += y.y;
                    o.z += y.z;
                    o.w += y.w;
                }
        }
        if (mine && part == 0) {
            const long long to = (long long)(g.row0 + row / g.heads) * p.Hq + g.head0 + row % g.heads;
            const float inv = row_inv[row];
            uint2 v;
            v.x = cvt_bf16x2(o.x * inv, o.y * inv);
            v.y = cvt_bf16x2(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2*>(p.out + to * D + d) = v;
            if (p.lse && d == 0) p.lse[to] = row_lse[row];
        }
    }
}

template <int D, int G, int KT>
cudaError_t launch(const KvAttnParams& p, cudaStream_t stream) {
    using SH = Shape<D, G, KT>;
    static std::atomic<uint64_t> asked{0};  // devices on which the kernel may take its memory
    cudaError_t err = allow_shared(kv_attn_kernel<D, G, KT, KvAttnParams>, SH::kSmem, asked);
    if (err != cudaSuccess) return err;
    // Where each CTA can have a row tile of its own and the longest possible one is short, and
    // longer than an equal share of row tiles like it by at most 2 tiles a warp, nothing is
    // cut and no second kernel needed.  (The lengths are not known here, only how many
    // pages or which window they are in.)  1 sequence of 573 tokens: 11.1 us cut, 7.6
    // whole; 32 of 4 rows with a window of 1024: 30.8 cut, 23.3 whole.
    long long most = ((long long)p.max_pages * p.page_size + SH::kTile - 1) / SH::kTile;
    if (p.window) {
        const long long seen = ((long long)p.window + p.tile_toks - 2) / SH::kTile + 2 +
                               ((long long)p.sinks + SH::kTile - 1) / SH::kTile;
        most = most < seen ? most : seen;
    }
    const long long row_tiles = (long long)p.S * p.Hkv * p.head_parts;
    if (row_tiles <= p.ctas && most <= kUncutTiles &&
        most * (p.ctas - row_tiles) <= 2LL * SH::kWarps * p.ctas) {
        KvAttnParams one = p;
        one.whole = 1;
        kv_attn_kernel<D, G, KT, KvAttnParams><<<(unsigned)row_tiles, SH::kThreads, SH::kSmem, stream>>>(one);
        return cudaGetLastError();
    }
    const unsigned grid = (unsigned)p.ctas;
    kv_attn_kernel<D, G, KT, KvAttnParams><<<grid, SH::kThreads, SH::kSmem, stream>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    // the second kernel's blocks are placed as the first one's finish
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = (size_t)p.ctas * SH::kRows * sizeof(float);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_join_kernel<D>, p, (int)SH::kRows);
}

}  // namespace

size_t kv_attn_seg_bytes(int ctas) { return (size_t)ctas * 2 * sizeof(Seg); }

size_t kv_attn_partial_bytes(int ctas, int tile_rows, int D) {
    return (size_t)ctas * 2 * tile_rows * (D + 2) * sizeof(float);
}

int kv_attn_ctas_per_sm() { return Shape<128, 64, 1>::kCtas; }

cudaError_t launch_kv_attn(const KvAttnParams& p, int D, int G, int tile_rows,
                           cudaStream_t stream) {
#define MXQ_KV_ATTN(d, g)                                        \
    if (D == d && G == g)                                        \
        return tile_rows <= 4   ? launch<d, g, 1>(p, stream)     \
               : tile_rows <= 8 ? launch<d, g, 2>(p, stream)     \
                                : launch<d, g, 4>(p, stream);
    MXQ_KV_ATTN(64, 32)
    MXQ_KV_ATTN(64, 64)
    MXQ_KV_ATTN(128, 32)
    MXQ_KV_ATTN(128, 64)
    MXQ_KV_ATTN(128, 128)
    MXQ_KV_ATTN(256, 32)
    MXQ_KV_ATTN(256, 64)
    MXQ_KV_ATTN(256, 128)
#undef MXQ_KV_ATTN
    return cudaErrorInvalidValue;
}

}  // namespace mxq
