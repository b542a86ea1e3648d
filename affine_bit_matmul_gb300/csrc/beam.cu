// Selection of beams: the best K of a prompt's W beams times V tokens.
//
//   cand(w, v) = score[w] + x[w, v] - log sum_u exp x[w, u]
//
// A row's candidates are in the order of its logits x, so each CTA takes a chunk of one row,
// keeps it in registers, and gives the K largest logits of it with their tokens, the
// chunk's largest logit m and sum exp(x - m).  A second kernel, one CTA a prompt, adds the
// sums to the rows' logarithms in 64 bits, turns the lists' logits into candidates and takes
// the best K of all.
//   Selecting without sorting: the largest logits of groups of threads are known, and at
// least K logits are at or above the K-th largest of those; it is found bit by bit (16 bits
// are enough), and what is not below it, little more than K logits, goes to shared memory,
// where each counts how many are ahead of it.  Keys are (value, ~token), so no two are equal and
// the order of arrival does not matter.  Where too many are level (rows of equal logits) the
// K largest are taken one by one.
//   Candidates are compared in 64 bits: two beams' are sums of different scores.  The chunks
// of a row begin at the same tokens whatever the row's alignment, so that equal rows have equal
// sums, and equal candidates of equal beams go to the lowest beam.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mxq_internal.h"
#include "tc_common.cuh"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRoom = 512;   // keys that are compared with each other
constexpr int kMostK = 64;
constexpr int kMostW = 64;

struct BeamParams {
    const void* logits;
    long long row_stride;  // in bytes
    const float* scores;
    const uint8_t* done;
    float* out_scores;
    int32_t *parents, *tokens;
    uint8_t* out_done;
    int N, W, V, K, chunks, end;
    float2* stats;         // workspace: [row][chunk] largest logit, sum
    unsigned long long* lists;  // workspace: [row][chunk][K] keys, 0 where there is none
};

// Whether x orders before y as fp32 numbers is whether these order so as unsigned ones.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ unsigned long long ordered(double x) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(x);
    return u ^ ((unsigned long long)((long long)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double from_ordered(unsigned long long u) {
    return __longlong_as_double((long long)(u ^ ((u >> 63) ? 0x8000000000000000ull : ~0ull)));
}

// A logit as a candidate's first key: -0 as +0, what is not a number as -inf.
__device__ __forceinline__ uint32_t value_key(float x) { return ordered(x == x ? x + 0.f : -INFINITY); }

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 bytes of a row, in registers.
template <bool F32>
struct Vec {
    static constexpr int kSize = F32 ? 4 : 8, kBytes = F32 ? 4 : 2;
    uint32_t w[4];
    __device__ __forceinline__ float at(int i) const {
        if constexpr (F32) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void none() {
        w[0] = w[1] = w[2] = w[3] = F32 ? 0xFF800000u : 0xFF80FF80u;  // -inf
    }
    // the largest that is a number
    __device__ __forceinline__ float most() const {
        if constexpr (F32) {
            return fmaxf(fmaxf(at(0), at(1)), fmaxf(at(2), at(3)));
        } else {
            const uint32_t m = max_bf16x2(max_bf16x2(w[0], w[1]), max_bf16x2(w[2], w[3]));
            return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
        }
    }
    // values v .. of a row of V at `row`; -inf past the end
    __device__ __forceinline__ void load(const uint8_t* row, int v, int V) {
        const uint8_t* at = row + (long long)v * kBytes;
        const int off = (int)(reinterpret_cast<uintptr_t>(at) & 15);
        if (off == 0 && v + kSize <= V) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(at));
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else if (v > 0 && v + 2 * kSize - off / kBytes <= V) {
            // between two aligned pieces, both within the row
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(at - off));
            const uint4 y = __ldg(reinterpret_cast<const uint4*>(at - off) + 1);
            const int bits = (off & 3) * 8;
            const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            switch (off >> 2) {
                case 0: shift<0>(u, bits); break;
                case 1: shift<1>(u, bits); break;
                case 2: shift<2>(u, bits); break;
                default: shift<3>(u, bits);
            }
        } else {
            none();
#pragma unroll
            for (int i = 0; i < kSize; ++i) {
                if (v + i >= V) continue;
                if constexpr (F32) {
                    w[i] = __ldg(reinterpret_cast<const uint32_t*>(at) + i);
                } else {
                    const uint32_t x = __ldg(reinterpret_cast<const uint16_t*>(at) + i);
                    w[i / 2] = i & 1 ? (w[i / 2] & 0xFFFFu) | x << 16 : (w[i / 2] & 0xFFFF0000u) | x;
                }
            }
        }
    }

private:
    template <int FROM>
    __device__ __forceinline__ void shift(const uint32_t (&u)[8], int bits) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(u[FROM + i], u[FROM + i + 1], bits);
    }
};

// The groups' largest values of a block, in shared memory, and from them the largest and a
// lower bound of the K-th largest of all: 2^SHIFT below it at most.
template <int SHIFT>
__device__ __forceinline__ uint32_t bound_of(const uint32_t* groups, int n, int K, uint32_t* top) {
    const int lane = threadIdx.x & 31;
    uint32_t x[kThreads / 32];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        x[i] = i * 32 < n ? groups[i * 32 + lane] : 0u;
        m = max(m, x[i]);
    }
    *top = __reduce_max_sync(0xFFFFFFFFu, m);
    uint32_t t = 0;
#pragma unroll 1
    for (int bit = 31; bit >= SHIFT; --bit) {
        const uint32_t c = t | 1u << bit;
        int count = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i)
            if (i * 32 < n) count += __popc(__ballot_sync(0xFFFFFFFFu, x[i] >= c));
        if (count >= K) t = c;
    }
    return t;
}

// How many threads make a group, of 256: the K-th largest of their maxima is then not far
// below the K-th largest of all.
__device__ __forceinline__ int group_threads(int K) { return K <= 10 ? 8 : K <= 40 ? 2 : 1; }

__device__ __forceinline__ uint32_t group_max(uint32_t x, int threads) {
    for (int o = 1; o < threads; o <<= 1) x = max(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    return x;
}

struct Key {
    unsigned long long value;  // ordered
    uint32_t back;             // ~index
};
__device__ __forceinline__ bool ahead(const Key& a, const Key& b) {
    return a.value > b.value || (a.value == b.value && a.back > b.back);
}

// The largest key of the block, in all threads.
__device__ __forceinline__ Key block_first(Key k, Key* room) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        Key x;
        x.value = __shfl_xor_sync(0xFFFFFFFFu, k.value, o);
        x.back = __shfl_xor_sync(0xFFFFFFFFu, k.back, o);
        if (ahead(x, k)) k = x;
    }
    __syncthreads();
    if (lane == 0) room[warp] = k;
    __syncthreads();
    Key best = room[0];
    for (int i = 1; i < kWarps; ++i)
        if (ahead(room[i], best)) best = room[i];
    return best;
}

// One chunk of a row, NV vectors a thread.
//   Bound by the memory.
template <bool F32, int NV>
__global__ void __launch_bounds__(kThreads, 4) beam_rows_kernel(const BeamParams p) {
    using V4 = Vec<F32>;
    __shared__ uint32_t groups[kThreads];
    __shared__ unsigned long long keys[kRoom];
    __shared__ float sums[kWarps];
    __shared__ Key room[kWarps];
    __shared__ int count;
    pdl_launch_dependents();
    const int row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    // a beam that has ended, or that is not in use, has no candidates here
    const float score = __ldg(p.scores + row);
    if (!(fabsf(score) < INFINITY) || (p.done && __ldg(p.done + row))) return;
    const uint8_t* x = static_cast<const uint8_t*>(p.logits) + row * p.row_stride;
    const int first = (chunk * NV * kThreads + (int)threadIdx.x) * V4::kSize;
    auto token = [&](int i) { return first + i * kThreads * V4::kSize; };
    if (threadIdx.x == 0) count = 0;
    V4 v[NV];
    if (((reinterpret_cast<uintptr_t>(x) & 15) == 0) &&
        (chunk + 1) * NV * kThreads * V4::kSize <= p.V) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint4 y = __ldg(reinterpret_cast<const uint4*>(x + (long long)token(i) * V4::kBytes));
            v[i].w[0] = y.x, v[i].w[1] = y.y, v[i].w[2] = y.z, v[i].w[3] = y.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (token(i) < p.V) v[i].load(x, token(i), p.V);
            else v[i].none();
        }
    }
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) most = fmaxf(most, v[i].most());
    const int each = group_threads(p.K), n_groups = kThreads / each;
    const uint32_t g = group_max(value_key(most), each);
    if (threadIdx.x % each == 0) groups[threadIdx.x / each] = g;
    __syncthreads();
    uint32_t top;
    const uint32_t bound = bound_of<16>(groups, n_groups, p.K, &top);
    // ---- sum of exponentials
    const float m = from_ordered(top), ref = m == -INFINITY ? 0.f : m;
    float l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V4::kSize; e += 2) {
            l0 += exp2_of((v[i].at(e) - ref) * 1.4426950408889634f);
            l1 += exp2_of((v[i].at(e + 1) - ref) * 1.4426950408889634f);
        }
    float l = l0 + l1;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    if (lane == 0) sums[warp] = l;
    // ---- keys at or above the bound
    auto key_of = [&](float y, int t) {
        return (unsigned long long)value_key(y) << 32 | (uint32_t)~t;
    };
    if (value_key(most) >= bound) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (value_key(v[i].most()) < bound) continue;
#pragma unroll
            for (int e = 0; e < V4::kSize; ++e) {
                if (value_key(v[i].at(e)) >= bound && token(i) + e < p.V) {
                    const int at = atomicAdd(&count, 1);
                    if (at < kRoom) keys[at] = key_of(v[i].at(e), token(i) + e);
                }
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float sum = 0.f;
        for (int i = 0; i < kWarps; ++i) sum += sums[i];
        p.stats[blockIdx.x] = make_float2(m, sum);
    }
    unsigned long long* out = p.lists + (long long)blockIdx.x * p.K;
    const int n = count;
    if (n <= kRoom) {
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const unsigned long long k = keys[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += keys[j] > k;
            if (rank < p.K) out[rank] = k;
        }
        for (int i = n + threadIdx.x; i < p.K; i += kThreads) out[i] = 0;
        return;
    }
    // level logits: the largest, the next one, ...
    Key last{~0ull, 0};
    for (int r = 0; r < p.K; ++r) {
        Key k{0, 0};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V4::kSize; ++e)
                if (token(i) + e < p.V) {
                    const unsigned long long y = key_of(v[i].at(e), token(i) + e);
                    if (y < last.value && y > k.value) k.value = y;
                }
        last = block_first(k, room);
        if (threadIdx.x == 0) out[r] = last.value;
    }
}

// One prompt: the best K of the lists of its rows.
__global__ void __launch_bounds__(kThreads) beam_best_kernel(const BeamParams p) {
    __shared__ double offset[kMostW];
    __shared__ uint8_t live[kMostW];
    __shared__ uint32_t groups[kThreads];
    __shared__ Key keys[kRoom];
    __shared__ Key room[kWarps];
    __shared__ int count;
    const int prompt = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int row0 = prompt * p.W, each_row = max(p.chunks * p.K, p.K + 1), all = p.W * each_row;
    if (threadIdx.x == 0) count = 0;
    pdl_wait();
    // ---- the rows' logarithms
    for (int w = warp; w < p.W; w += kWarps) {
        const float score = __ldg(p.scores + row0 + w);
        const bool in = fabsf(score) < INFINITY && !(p.done && __ldg(p.done + row0 + w));
        double off = 0.0;
        bool ok = in;
        if (in) {
            const float2* st = p.stats + (long long)(row0 + w) * p.chunks;
            float m = -INFINITY;
            for (int c = lane; c < p.chunks; c += 32) m = fmaxf(m, __ldcg(st + c).x);
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            double l = 0.0;
            for (int c = lane; c < p.chunks; c += 32) {
                const float2 s = __ldcg(st + c);
                // (a chunk of -inf has the sum 0)
                l += s.x == -INFINITY ? (double)s.y : (double)s.y * exp((double)s.x - (double)m);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
            off = (double)score - ((double)m + log(l));
            ok = off - off == 0.0;  // a number: some logit is finite, none is +inf or not a number
        }
        if (lane == 0) {
            offset[w] = off;
            live[w] = ok;
        }
    }
    __syncthreads();
    // candidate e of row w
    auto candidate = [&](int w, int e) {
        Key k{0, 0};
        if (live[w]) {
            if (e >= p.chunks * p.K) return k;
            const unsigned long long x = __ldcg(p.lists + (long long)(row0 + w) * p.chunks * p.K + e);
            if (x == 0) return k;
            k.value = ordered((double)from_ordered((uint32_t)(x >> 32)) + offset[w]);
            k.back = ~((uint32_t)w * (uint32_t)p.V + ~(uint32_t)x);
        } else if (e <= p.K) {
            // a beam that has ended: its end token as it stands; then, as for one without
            // candidates, the lowest tokens at -inf
            const float score = __ldg(p.scores + row0 + w);
            const bool ended = p.done && __ldg(p.done + row0 + w) && fabsf(score) < INFINITY;
            int t = e - 1;
            double x = -INFINITY;
            if (e == 0) {
                if (!ended) return k;
                t = p.end;
                x = (double)score;
            } else if (t >= p.V || (ended && t == p.end)) {
                return k;
            }
            k.value = ordered(x);
            k.back = ~((uint32_t)w * (uint32_t)p.V + (uint32_t)t);
        }
        return k;
    };
    uint32_t most = 0;
    for (int i = threadIdx.x; i < all; i += kThreads)
        most = max(most, (uint32_t)(candidate(i / each_row, i % each_row).value >> 32));
    const int each = group_threads(p.K), n_groups = kThreads / each;
    const uint32_t g = group_max(most, each);
    if (threadIdx.x % each == 0) groups[threadIdx.x / each] = g;
    __syncthreads();
    uint32_t top;
    const uint32_t bound = bound_of<0>(groups, n_groups, p.K, &top);
    for (int i = threadIdx.x; i < all; i += kThreads) {
        const Key k = candidate(i / each_row, i % each_row);
        if (k.value != 0 && (uint32_t)(k.value >> 32) >= bound) {
            const int at = atomicAdd(&count, 1);
            if (at < kRoom) keys[at] = k;
        }
    }
    __syncthreads();
    auto give = [&](int rank, const Key& k) {
        const uint32_t flat = ~k.back;
        const int w = (int)(flat / (uint32_t)p.V), t = (int)(flat % (uint32_t)p.V);
        const long long to = (long long)prompt * p.K + rank;
        p.out_scores[to] = (float)from_ordered(k.value);
        p.parents[to] = w;
        p.tokens[to] = t;
        if (p.out_done) p.out_done[to] = (p.done && p.done[row0 + w]) || t == p.end;
    };
    const int n = count;
    if (n <= kRoom) {
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const Key k = keys[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += ahead(keys[j], k);
            if (rank < p.K) give(rank, k);
        }
        return;
    }
    Key last{~0ull, ~0u};
    for (int r = 0; r < p.K; ++r) {
        Key k{0, 0};
        for (int i = threadIdx.x; i < all; i += kThreads) {
            const Key y = candidate(i / each_row, i % each_row);
            if (ahead(last, y) && ahead(y, k)) k = y;
        }
        last = block_first(k, room);
        if (threadIdx.x == 0) give(r, last);
    }
}

// Vectors of a thread: as many as leave four CTAs for each SM, up to 8.
struct Cut {
    int vectors, chunks;
};
Cut cut_of(long long rows, int V, int fp32) {
    Cut c{8, 1};
    for (;; c.vectors /= 2) {
        const int size = c.vectors * kThreads * (fp32 ? 4 : 8);
        c.chunks = (V - 1) / size + 1;
        if (c.vectors == 1 || rows * c.chunks >= 4 * 152) return c;
    }
}

template <bool F32>
cudaError_t launch_rows(const BeamParams& p, int vectors, cudaStream_t s) {
    const unsigned grid = (unsigned)((long long)p.N * p.W * p.chunks);
    switch (vectors) {
        case 8: beam_rows_kernel<F32, 8><<<grid, kThreads, 0, s>>>(p); break;
        case 4: beam_rows_kernel<F32, 4><<<grid, kThreads, 0, s>>>(p); break;
        case 2: beam_rows_kernel<F32, 2><<<grid, kThreads, 0, s>>>(p); break;
        default: beam_rows_kernel<F32, 1><<<grid, kThreads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

size_t stat_bytes(long long rows, int chunks) { return ((size_t)rows * chunks * sizeof(float2) + 255) / 256 * 256; }

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool shape_ok(int N, int W, int V, int K) {
    return N >= 0 && W > 0 && W <= kMostW && V > 0 && K > 0 && K <= kMostK && K <= (long long)W * V;
}

}  // namespace
}  // namespace mxq

extern "C" {

size_t mxq_beam_select_workspace_bytes(int N, int W, int V, int K, int fp32) {
    if (!mxq::shape_ok(N, W, V, K)) return 0;
    const long long rows = (long long)N * W;
    const mxq::Cut c = mxq::cut_of(rows, V, fp32);
    return mxq::stat_bytes(rows, c.chunks) + (size_t)rows * c.chunks * K * sizeof(unsigned long long);
}

mxq_status mxq_beam_select(const void* logits, long long row_stride, int fp32, const float* scores,
                           const uint8_t* done, float* out_scores, int32_t* parents, int32_t* tokens,
                           uint8_t* out_done, int N, int W, int V, int K, int end_token, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (!mxq::shape_ok(N, W, V, K) || row_stride < 0) return MXQ_ERR_INVALID_ARG;
    if ((done || out_done) && (end_token < 0 || end_token >= V)) return MXQ_ERR_INVALID_ARG;
    if (N > 0 && (!logits || !scores || !out_scores || !parents || !tokens)) return MXQ_ERR_INVALID_ARG;
    if (!mxq::aligned(logits, fp32 ? 4 : 2) || !mxq::aligned(scores, 4) || !mxq::aligned(out_scores, 4) ||
        !mxq::aligned(parents, 4) || !mxq::aligned(tokens, 4) || !mxq::aligned(workspace, 256))
        return MXQ_ERR_MISALIGNED;
    const long long rows = (long long)N * W;
    const mxq::Cut c = mxq::cut_of(rows, V, fp32);
    // tokens are counted in 32 bits, over a prompt's beams too; CTAs as well
    if ((long long)W * V > 0x7FFFFFFF - 65536 || rows * c.chunks > 0x7FFFFFFF ||
        (long long)W * c.chunks * K > 0x7FFFFFFF)
        return MXQ_ERR_UNSUPPORTED;
    if (N > 0 && (!workspace || workspace_bytes < mxq_beam_select_workspace_bytes(N, W, V, K, fp32)))
        return MXQ_ERR_WORKSPACE;
    const mxq_status st = mxq::check_current_device(nullptr);
    if (st != MXQ_OK) return st;
    if (N == 0) return MXQ_OK;
    mxq::BeamParams p;
    p.logits = logits;
    p.row_stride = row_stride * (fp32 ? 4 : 2);
    p.scores = scores;
    p.done = done;
    p.out_scores = out_scores;
    p.parents = parents;
    p.tokens = tokens;
    p.out_done = out_done;
    p.N = N;
    p.W = W;
    p.V = V;
    p.K = K;
    p.chunks = c.chunks;
    p.end = end_token;
    p.stats = static_cast<float2*>(workspace);
    p.lists = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(workspace) +
                                                    mxq::stat_bytes(rows, c.chunks));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = fp32 ? mxq::launch_rows<true>(p, c.vectors, s) : mxq::launch_rows<false>(p, c.vectors, s);
    if (err != cudaSuccess) return MXQ_ERR_CUDA;
    // the second kernel's blocks are placed while the first one finishes
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)N);
    cfg.blockDim = dim3(mxq::kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, mxq::beam_best_kernel, p);
    return err == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

}  // extern "C"
