// Attention of many query rows over a paged 4-bit key/value cache: the plan of the row
// tiles, the launches of kv_many.cuh's kernel, and the joining of row tiles that its runs cut.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_many.cuh"

namespace mxq {
namespace {

// ---------------------------------------------------------------- plan and join

__device__ int block_scan(int x, int* total) {  // exclusive; 1024 threads
    __shared__ int sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int w = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xFFFFFFFFu, w, 31);
    const int before = warp ? __shfl_sync(0xFFFFFFFFu, w, warp - 1) : 0;
    __syncthreads();
    return before + incl - x;
}

// The row tiles of all sequences and the units before each: one block, 3.5 us, most of
// it the chain of three scans.
__global__ void __launch_bounds__(1024) kv_plan_kernel(const KvAttnParams p) {
    pdl_launch_dependents();
    Entry* entries = reinterpret_cast<Entry*>(p.entries);
    int* starts = p.seq_tiles;  // first row tile of each sequence
    int run = 0;
    bool bad = false;
    for (int s0 = 0; s0 < p.S; s0 += 1024) {
        const int s = s0 + threadIdx.x;
        int n = 0;
        if (s < p.S) {
            const Span sp = span_of<kTile>(p, s, 0);
            bad |= sp.bad != 0;
            if (sp.toks > 0) {
                const int rows = p.q_starts ? __ldg(p.q_starts + s + 1) - __ldg(p.q_starts + s) : 1;
                n = (rows + p.tile_toks - 1) / p.tile_toks;
            }
        }
        int total;
        const int at = run + block_scan(n, &total);
        if (s < p.S) starts[s] = at;
        run += total;
    }
    // rows that overlap (decreasing starts) can make more row tiles than there is room for
    bad |= run > p.max_entries;
    const int n_entries = min(run, p.max_entries);
    if (bad) flag_status(p.status, MXQ_DEV_BAD_SEQUENCE);
    __syncthreads();
    run = 0;
    for (int e0 = 0; e0 < n_entries; e0 += 1024) {
        const int e = e0 + threadIdx.x;
        int tiles = 0;
        if (e < n_entries) {
            int lo = 0, hi = p.S - 1;  // the last sequence that starts at or before e
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (starts[mid] <= e) lo = mid;
                else hi = mid - 1;
            }
            const Span sp = span_of<kTile>(p, lo, e - starts[lo]);
            Entry en;
            en.s = lo;
            en.row0 = sp.row0;
            en.toks = sp.toks;
            en.p0 = sp.p0;
            en.tiles = sp.tiles;
            tiles = sp.tiles + kEndUnits;
            en.head_tiles = sp.head_tiles;
            en.tail = sp.tail;
            en.pad = 0;
            entries[e] = en;
        }
        int total;
        const int at = run + block_scan(tiles, &total);
        if (e < n_entries) p.before[e] = at;
        run += total;
    }
    if (threadIdx.x == 0) {
        p.counts[0] = n_entries;
        p.counts[1] = run;
    }
}

// Joins the pieces of cut row tiles; blockIdx.y takes a share of the rows.  13 us for
// 151 cut tiles of 256 rows of 128 values (40 MB of fp32 sums, in L2).
template <int D>
__global__ void __launch_bounds__(256) kv_join_rows_kernel(const KvAttnParams p, int tile_rows) {
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
    int last = cta;
    while (last + 1 < p.ctas) {
        ++last;
        const int f = segs[last * 2].flags;
        if (f < 0 || (f & kEnds)) break;
    }
    const int n = last - cta + 1, rows = g.toks * g.heads;
    const long long stride = (long long)tile_rows * (D + 2);
    auto piece = [&](int k) { return p.partial + ((cta + k) * 2LL + (k ? 0 : 1)) * stride; };
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < rows * (D / 4);
         i += gridDim.y * blockDim.x) {
        const int row = i / (D / 4), d = (i % (D / 4)) * 4;
        float mm = -INFINITY;
        for (int k = 0; k < n; ++k) mm = fmaxf(mm, piece(k)[2 * row]);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float* q = piece(k);
            const float2 ml = *reinterpret_cast<const float2*>(q + 2 * row);
            const float4 y =
                *reinterpret_cast<const float4*>(q + 2 * tile_rows + (long long)row * D + d);
            const float f = exp2_approx(ml.x - ref);
            ll = fmaf(ml.y, f, ll);
            o.x = fmaf(y.x, f, o.x);
            o.y = fmaf(y.y, f, o.y);
            o.z = fmaf(y.z, f, o.z);
            o.w = fmaf(y.w, f, o.w);
        }
        const long long to = (long long)(g.row0 + row / g.heads) * p.Hq + g.head0 + row % g.heads;
        const float inv = ll > 0.f ? 1.f / ll : 0.f;
        uint2 v;
        v.x = cvt_bf16x2(o.x * inv, o.y * inv);
        v.y = cvt_bf16x2(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2*>(p.out + to * D + d) = v;
        if (p.lse && d == 0) p.lse[to] = log_sum_of(mm, ll);
    }
}

template <int D, int G>
cudaError_t launch(const KvAttnParams& p, cudaStream_t stream) {
    using SH = Shape<D, G>;
    static std::atomic<uint64_t> asked{0};  // devices on which the kernel may take its memory
    cudaError_t err = allow_shared(kv_prefill_kernel<D, G, KvAttnParams, NoPart>, SH::kSmem, asked);
    if (err != cudaSuccess) return err;
    kv_plan_kernel<<<1, 1024, 0, stream>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    // each kernel's blocks are placed while the one before it finishes
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = SH::kSmem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kv_prefill_kernel<D, G, KvAttnParams, NoPart>, p, NoPart{});
    if (err != cudaSuccess) return err;
    cfg.gridDim = dim3((unsigned)p.ctas, 16);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv_join_rows_kernel<D>, p, (int)SH::kRows);
}

}  // namespace

int kv_prefill_rows(int D) { return D == 256 ? 128 : 256; }

size_t kv_prefill_entry_bytes() { return sizeof(Entry); }

cudaError_t launch_kv_prefill(const KvAttnParams& p, int D, int G, cudaStream_t stream) {
#define MXQ_KV_PREFILL(d, g) \
    if (D == d && G == g) return launch<d, g>(p, stream);
    MXQ_KV_PREFILL(64, 32)
    MXQ_KV_PREFILL(64, 64)
    MXQ_KV_PREFILL(128, 32)
    MXQ_KV_PREFILL(128, 64)
    MXQ_KV_PREFILL(128, 128)
    MXQ_KV_PREFILL(256, 32)
    MXQ_KV_PREFILL(256, 64)
    MXQ_KV_PREFILL(256, 128)
#undef MXQ_KV_PREFILL
    return cudaErrorInvalidValue;
}

}  // namespace mxq
