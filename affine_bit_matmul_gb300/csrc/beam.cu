// Selection of beams: the best K of a prompt's W beams times V tokens.
//
//   cand(w, v) = score[w] + x[w, v] - log sum_u exp x[w, u]
//
// A row's candidates are in the order of its logits x, so each warp takes parts of rows, on
// its own: it reads a part once, keeps the K largest logits with their tokens, the largest one
// m and sum exp(x - m).  Then one CTA a prompt adds the sums to the rows' logarithms in 64 bits,
// turns the lists' logits into candidates and takes the best K of all.
//   Selecting without sorting: a lane's vectors at one place of all steps are a slot, 128 of
// them a warp, whose largest logits are known in the end.  At least K logits are at or above the K-th
// largest of those.  Only the slots that reach it, few more than K, are looked at again, and what is not below it goes to shared memory, where
// each of those logits counts how many are ahead of it.  Keys are (value, ~token), so no two are
// equal.  When there are too many (level logits) the K best stay, and equal logits with later
// tokens than all that were there cannot come in.
//   Candidates are compared in 48 bits, none past the 53rd: two beams' are sums of different scores.  All rows are
// cut at the same tokens, whatever their alignment, so that equal rows have equal sums, and equal
// candidates of equal beams go to the lowest beam.
//   A lane copies what it will look at (and its neighbour, where a row does not begin at 16
// bytes) with asynchronous 16-byte copies two steps ahead; nothing in the loop waits for another
// warp.
//   64 prompts of 8 beams of 131072 bf16 logits, 134 MB: 42 us, of which the first kernel takes some 34, 3.9 TB/s. It
// issues 10 instructions a logit of its lanes, 2.4 a cycle and SM while it runs, and the looks at slots of all warps
// fall together at the end, when the memory is idle.  Small calls are a chain: scores, logits, slots, lists, a second
// launch: 10 us for 1 prompt of 4 beams of 32768.
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_attn_common.cuh"
#include "mxq_internal.h"
#include "tc_common.cuh"

namespace mxq {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMostK = 64;
constexpr int kMostW = 64;
constexpr int kVecs = 4;       // 16-byte vectors of a lane in a step
constexpr int kRoom = 96;      // keys of a warp: K and those of one look at 32 lanes
constexpr int kStages = 3;
constexpr int kLook = 2;       // vectors of a lane that are looked at again at once
constexpr int kPieces = kVecs * 32;              // of 16 bytes in a step
constexpr int kStageBytes = (kPieces + 1) * 16;  // and one more, where rows are not aligned
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kSmem = kRingBytes + kWarps * (kRoom * 8 + kPieces);

constexpr float kLog2e = 1.4426950408889634f;

struct BeamParams {
    const uint8_t* logits;
    long long row_stride;  // in bytes
    const float* scores;
    const uint8_t* done;
    float* out_scores;
    int32_t *parents, *tokens;
    uint8_t* out_done;
    int N, W, V, K, steps, parts, end;
    float2* stats;              // workspace: [prompt][row][part] largest logit, sum
    unsigned long long* lists;  // workspace: [prompt][K][row][part] keys, 0 where there is none
};

// Whether x orders before y as fp32 numbers is whether these order so as unsigned ones.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// a + b and, if it is finite, what its rounding left.
__device__ __forceinline__ float sum_of(float a, float b, float* left) {
    const float s = a + b, y = s - a;
    *left = (a - (s - y)) + (b - y);
    return s;
}
// A candidate, a logit, its row's largest one and the row's offset (two fp32 numbers, the second within
// half a step of the first), as a key: the sum, an fp32 number and what its rounding left.  The two of them
// can say more than 53 bits, where the second is far smaller: beside a logit of -1e30 or of the type's lowest
// number, which stands for a token that is not allowed, a beam's score would still count, and such tokens of
// all beams are level as 64-bit numbers.  So the rest is rounded to them.
__device__ __forceinline__ unsigned long long sum_key(float x, float top, float2 off) {
    float e0, e;
    const float d = sum_of(x, -top, &e0);
    float s = sum_of(d, off.x, &e);
    if (fabsf(s) < INFINITY) {
        e = e0 + e + off.y;
        const float t = s + e;
        e = e - (t - s);
        s = t;
        // steps of 2^-52 of s's power of two (rests above 2^-30 of it have no finer bits but for one)
        const uint32_t pow = __float_as_uint(s) & 0x7F800000u;
        if (pow > (30u << 23) && fabsf(e) < __uint_as_float(pow - (30u << 23))) {
            const float c = __uint_as_float((pow - (29u << 23)) | 0x00400000u);
            e = (e + c) - c;
        }
    } else {
        e = 0.f;
    }
    return (unsigned long long)ordered(s + 0.f) << 32 | ordered(e + 0.f);
}

// A logit as a candidate's first key: -0 as +0, what is not a number as -inf.
__device__ __forceinline__ uint32_t value_key(float x) { return ordered(x == x ? x + 0.f : -INFINITY); }

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void parts_of(uint64_t p, float* a, float* b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(p));
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
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
    // the same, where i is not known to the compiler
    __device__ __forceinline__ float any(int i) const {
        const int k = F32 ? i : i / 2;
        const uint32_t x = k < 2 ? (k ? w[1] : w[0]) : k == 2 ? w[2] : w[3];
        return __uint_as_float(F32 ? x : i & 1 ? x & 0xFFFF0000u : x << 16);
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
    // values past the first n: -inf
    __device__ __forceinline__ void cut(int n) {
#pragma unroll
        for (int i = 0; i < kSize; ++i) {
            if (i < n) continue;
            if constexpr (F32) w[i] = 0xFF800000u;
            else w[i / 2] = i & 1 ? (w[i / 2] & 0xFFFFu) | 0xFF800000u : (w[i / 2] & 0xFFFF0000u) | 0xFF80u;
        }
    }
    // values v .. of a row of V in memory, v < V
    __device__ __forceinline__ void load(const uint8_t* row, int v, int V) {
        const uint8_t* at = row + (long long)v * kBytes;
        const int off = (int)(reinterpret_cast<uintptr_t>(at) & 15);
        if (off == 0 && v + kSize <= V) {
            const uint4 x = *(reinterpret_cast<const uint4*>(at));
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            return;
        }
        w[0] = w[1] = w[2] = w[3] = 0;
#pragma unroll
        for (int i = 0; i < kSize; ++i) {
            if (v + i >= V) continue;
            if constexpr (F32) w[i] = *(reinterpret_cast<const uint32_t*>(at) + i);
            else w[i / 2] |= (uint32_t)*(reinterpret_cast<const uint16_t*>(at) + i) << (i & 1 ? 16 : 0);
        }
        cut(V - v);
    }
    // from two aligned pieces in shared memory, `off` bytes into the first
    __device__ __forceinline__ void load(uint32_t at, int off) {
        const uint4 x = ld_shared_v4(at);
        if (off == 0) {
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            return;
        }
        const uint4 y = ld_shared_v4(at + 16);
        const int bits = (off & 3) * 8;
        const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        switch (off >> 2) {
            case 0: shift<0>(u, bits); break;
            case 1: shift<1>(u, bits); break;
            case 2: shift<2>(u, bits); break;
            default: shift<3>(u, bits);
        }
    }

private:
    template <int FROM>
    __device__ __forceinline__ void shift(const uint32_t (&u)[8], int bits) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(u[FROM + i], u[FROM + i + 1], bits);
    }
};

__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
    const uint32_t x = max(a, b);
    b = min(a, b);
    a = x;
}

// The K-th largest of four values of each lane, taken away from the top (bit by bit instead: 1 to 6 us more
// for K up to 32, 5 us less of 112 for 64 of 64 x 8 x 50001).
__device__ __forceinline__ uint32_t kth_of(uint32_t (&x)[4], int K) {
    order(x[0], x[1]);
    order(x[2], x[3]);
    order(x[0], x[2]);
    order(x[1], x[3]);
    order(x[1], x[2]);
    for (;;) {
        const uint32_t t = __reduce_max_sync(0xFFFFFFFFu, x[0]);
        const bool mine = x[0] == t;
        K -= __popc(__ballot_sync(0xFFFFFFFFu, mine));
        if (K <= 0 || t == 0) return t;
        if (mine) {
            x[0] = x[1];
            x[1] = x[2];
            x[2] = x[3];
            x[3] = 0;
        }
    }
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

struct Rows {
    float score[kMostW];
    bool ended[kMostW];
    float2 offset[kMostW];
    float top[kMostW];
    unsigned long long sum[kMostW];
    bool used[kMostW];      // neither ended nor without a score
    uint8_t row[kMostW];    // those that are
    int live;               // and their number
};

// Whether beam `row` of all has logits that count.
__device__ __forceinline__ bool in_use(const BeamParams& p, long long row) {
    return fabsf(p.scores[row]) < INFINITY && !(p.done && p.done[row]);
}

// A prompt's rows in use, by one warp: beams that have ended, or have no score, have no candidates
// in their logits.  Scores and ends are kept, as the results may take their place, and are read in L2:
// this kernel starts when the first one has waited for what comes before the call.
__device__ __forceinline__ void find_rows(const BeamParams& p, Rows& r, long long row0) {
    const int lane = threadIdx.x & 31;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kMostW; i += 32) {
        const int w = i + lane;
        const float score = w < p.W ? __ldcg(p.scores + row0 + w) : 0.f;
        const bool ended = w < p.W && p.done && __ldcg(p.done + row0 + w);
        const bool in = w < p.W && fabsf(score) < INFINITY && !ended;
        r.score[w] = score;
        r.ended[w] = ended;
        const uint32_t live = __ballot_sync(0xFFFFFFFFu, in);
        const int at = n + __popc(live & ((1u << lane) - 1u));
        r.used[w] = in;
        if (in) r.row[at] = w;
        n += __popc(live);
    }
    if (lane == 0) r.live = n;
}

// What a CTA selects with.
struct Best {
    static constexpr int kKeys = 1024;
    Key keys[kKeys];
    uint32_t groups[kThreads / 4];
    Key first[kWarps];
    int count;
};

// The best K candidates of a prompt out of its rows' lists; one CTA.
__device__ __forceinline__ void best_of_prompt(const BeamParams& p, Rows& r, Best& s, int prompt) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, parts = p.parts, span = p.W * parts;
    const long long row0 = (long long)prompt * p.W;
    // entries: the first of the lists of the rows in use, the second ones, ...; and K + 1 of each row, for
    // those that have no other ones
    const int lists = r.live * parts, in_lists = lists * p.K, all = in_lists + p.W * (p.K + 1);
    auto entry = [&](int i, int* w) {
        *w = 0;
        if (i >= in_lists) return 0ull;
        const unsigned rank = (unsigned)i / lists, list = i - rank * lists, n = list / (unsigned)parts;
        *w = r.row[n];
        return __ldcg(p.lists + ((long long)prompt * p.K + rank) * span + *w * parts + (list - n * parts));
    };
    constexpr int kHeld = 2;  // entries that a thread keeps
    unsigned long long held[kHeld];
    int held_row[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = entry(tid + i * kThreads, &held_row[i]);
    // ---- the rows' logarithms
    if (tid == 0) s.count = 0;
    for (int w = warp; w < p.W; w += kWarps) {
        if (!r.used[w]) continue;
        const float2* st = p.stats + (row0 + w) * parts;
        const float2 x = lane < parts ? __ldcg(st + lane) : make_float2(-INFINITY, 0.f);
        float m = x.x;
        for (int i = lane + 32; i < parts; i += 32) m = fmaxf(m, __ldcg(st + i).x);
        m = from_ordered(__reduce_max_sync(0xFFFFFFFFu, ordered(m)));
        // the parts' sums in units of 2^-31, which are added without rounding (there are less than
        // 2^31 terms of at most 1; a part of -inf has the sum 0)
        bool ok = true;
        auto scaled = [&](float2 y) {
            const float l = y.x == -INFINITY ? y.y : y.y * exp2_approx((y.x - m) * kLog2e);
            ok = ok && l < INFINITY;  // (a number)
            return ok ? (unsigned long long)((double)l * 0x1p31) : 0ull;
        };
        unsigned long long l = scaled(x);
        for (int i = lane + 32; i < parts; i += 32) l += scaled(__ldcg(st + i));
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (lane == 0) {
            r.top[w] = m;
            r.sum[w] = ok ? l : 0;
        }
    }
    __syncthreads();
    for (int w = tid; w < p.W; w += kThreads) {
        // in 64 bits, as two fp32 numbers, of a candidate with the row's largest logit; not a number where
        // no logit is finite, or one is +inf or not a number
        float2 off = make_float2(NAN, 0.f);
        if (r.used[w] && r.sum[w]) {
            const double x = (double)r.score[w] - (log((double)r.sum[w]) - 21.487562597358306);  // 31 ln 2
            off.x = (float)x;
            off.y = (float)(x - (double)off.x);
        }
        r.offset[w] = off;
    }
    __syncthreads();
    // what entry i, x in a list of a row, is as a candidate
    auto candidate = [&](int i, unsigned long long x, int list_row) {
        Key k{0, 0};
        if (i < in_lists) {
            const int w = list_row;
            const float2 off = r.offset[w];
            if (x == 0 || off.x - off.x != 0.f) return k;
            k.value = sum_key(from_ordered((uint32_t)(x >> 32)), r.top[w], off);
            k.back = ~((uint32_t)w * (uint32_t)p.V + ~(uint32_t)x);
            return k;
        }
        // a beam that has ended: its end token as it stands; then, as for one without
        // candidates, the lowest tokens at -inf
        const int w = (i - in_lists) / (p.K + 1), e = (i - in_lists) - w * (p.K + 1);
        const float off = r.offset[w].x;
        if (off - off == 0.f) return k;
        const float score = r.score[w];
        const bool ended = r.ended[w] && fabsf(score) < INFINITY;
        int t = e - 1;
        float y = -INFINITY;
        if (e == 0) {
            if (!ended) return k;
            t = p.end;
            y = score;
        } else if (t >= p.V || (ended && t == p.end)) {
            return k;
        }
        k.value = sum_key(y, 0.f, make_float2(0.f, 0.f));
        k.back = ~((uint32_t)w * (uint32_t)p.V + (uint32_t)t);
        return k;
    };
    auto nth = [&](int i) {
        int w;
        const unsigned long long x = entry(i, &w);
        return candidate(i, x, w);
    };
    Key mine[kHeld];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        mine[i] = Key{0, 0};
        if (tid + i * kThreads < all) mine[i] = candidate(tid + i * kThreads, held[i], held_row[i]);
        most = max(most, (uint32_t)(mine[i].value >> 32));
    }
    for (int i = tid + kHeld * kThreads; i < all; i += kThreads) most = max(most, (uint32_t)(nth(i).value >> 32));
    // the K-th largest of groups of 4 threads
    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
    if (tid % 4 == 0) s.groups[tid / 4] = most;
    __syncthreads();
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = s.groups[i * 32 + lane];
    const uint32_t bound = kth_of(x, p.K);
    auto take = [&](const Key& k) {
        if (k.value == 0 || (uint32_t)(k.value >> 32) < bound) return;
        const int at = atomicAdd(&s.count, 1);
        if (at < Best::kKeys) s.keys[at] = k;
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) take(mine[i]);
    for (int i = tid + kHeld * kThreads; i < all; i += kThreads) take(nth(i));
    __syncthreads();
    auto give = [&](int rank, const Key& k) {
        const uint32_t flat = ~k.back;
        const int w = (int)(flat / (uint32_t)p.V), t = (int)(flat % (uint32_t)p.V);
        const long long to = (long long)prompt * p.K + rank;
        p.out_scores[to] = from_ordered((uint32_t)(k.value >> 32));
        p.parents[to] = w;
        p.tokens[to] = t;
        if (p.out_done) p.out_done[to] = r.ended[w] || t == p.end;
    };
    const int n = s.count;
    if (n <= Best::kKeys) {
        for (int i = tid; i < n; i += kThreads) {
            const Key k = s.keys[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += ahead(s.keys[j], k);
            if (rank < p.K) give(rank, k);
        }
        return;
    }
    // level candidates: the best, the next one, ...
    Key last{~0ull, ~0u};
    for (int rank = 0; rank < p.K; ++rank) {
        Key k{0, 0};
        for (int i = tid; i < all; i += kThreads) {
            const Key y = nth(i);
            if (ahead(last, y) && ahead(y, k)) k = y;
        }
        last = block_first(k, s.first);
        if (tid == 0) give(rank, last);
    }
}

// The best K of a warp's n keys (at most kRoom), in order where `to` is.
__device__ __forceinline__ void rank_keys(const unsigned long long* keys, int n, int K, unsigned long long* to,
                                          long long step = 1) {
    const int lane = threadIdx.x & 31;
    unsigned long long k[kRoom / 32];
    int rank[kRoom / 32];
#pragma unroll
    for (int i = 0; i < kRoom / 32; ++i) {
        k[i] = i * 32 + lane < n ? keys[i * 32 + lane] : 0;
        rank[i] = 0;
    }
    for (int j = 0; j < n; ++j) {
        const unsigned long long x = keys[j];
#pragma unroll
        for (int i = 0; i < kRoom / 32; ++i) rank[i] += x > k[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kRoom / 32; ++i)
        if (k[i] && rank[i] < K) to[rank[i] * step] = k[i];
    __syncwarp();
}

template <bool F32>
__global__ void __launch_bounds__(kThreads, 2) beam_kernel(const BeamParams p) {
    using V4 = Vec<F32>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int all_steps = (p.V - 1) / (kPieces * V4::kSize) + 1, parts = p.parts;
    pdl_wait();
    pdl_launch_dependents();
    // this warp's parts: every so many of all rows
    const long long items = (long long)p.N * p.W * parts;
    const int stride = (int)gridDim.x * kWarps;
    const uint32_t ring = smem_u32(smem) + warp * (kStages * kStageBytes);
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(smem + kRingBytes) + warp * kRoom;
    uint8_t* slots = smem + kRingBytes + kWarps * kRoom * 8 + warp * kPieces;
    // Steps one after the other: of a part of the row at x, from step0 to `end`.
    struct At {
        long long item;
        int step0, step, end;
        const uint8_t* x;
    };
    auto begin = [&](At& a, long long item) {
        for (a.item = item; a.item < items; a.item += stride) {
            const long long i = a.item / parts;
            if (!in_use(p, i)) continue;
            a.x = p.logits + i * p.row_stride;
            a.step = a.step0 = (int)(a.item - i * parts) * p.steps;
            a.end = min(a.step + p.steps, all_steps);
            return;
        }
    };
    auto next = [&](At& a) {
        if (++a.step == a.end) begin(a, a.item + stride);
    };
    // the copies of a step's pieces that are within its row
    At ahead_at{};
    int to_stage = 0;
    auto issue = [&]() {
        if (ahead_at.item < items) {
            const uint8_t* row = ahead_at.x;
            const uint8_t* end = row + (long long)p.V * V4::kBytes;
            const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15);
            const uint32_t to = ring + to_stage * kStageBytes;
            const uint8_t* from = row - off + (long long)ahead_at.step * (kPieces * 16);
            auto piece = [&](int i) {
                const uint8_t* at = from + i * 16;
                if (at >= end) return;
                if (at >= row) {
                    const long long left = end - at;
                    cp_async_16(to + i * 16, at, left < 16 ? (uint32_t)left : 16u);
                } else {
                    // what is before the row is not read
                    for (int b = off; b < 16 && at + b < end; b += V4::kBytes) {
                        if constexpr (F32)
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + i * 16 + b),
                                         "r"(*(reinterpret_cast<const uint32_t*>(at + b)))
                                         : "memory");
                        else
                            asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + i * 16 + b),
                                         "h"(*(reinterpret_cast<const uint16_t*>(at + b)))
                                         : "memory");
                    }
                }
            };
            if (off == 0 && from + kPieces * 16 <= end) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i) cp_async_16(to + (i * 32 + lane) * 16, from + (i * 32 + lane) * 16, 16u);
            } else {
#pragma unroll 1
                for (int i = 0; i < kVecs; ++i) piece(i * 32 + lane);
                if (lane == 0 && off) piece(kPieces);
            }
            if (++to_stage == kStages) to_stage = 0;
            next(ahead_at);
        }
        cp_async_commit();
    };
    begin(ahead_at, (int)blockIdx.x * kWarps + warp);
    At at = ahead_at;
    issue();
    issue();
    int stage = 0;
    float m = -INFINITY, l = 0.f;
    float so_far[kVecs];  // largest logits of the slots
#pragma unroll
    for (int i = 0; i < kVecs; ++i) so_far[i] = -INFINITY;
    while (at.item < items) {
        cp_async_wait<1>();
        __syncwarp();
        issue();
        const int off = (int)(reinterpret_cast<uintptr_t>(at.x) & 15);
        const uint32_t from = ring + stage * kStageBytes + lane * 16;
        if (++stage == kStages) stage = 0;
        const int token0 = (at.step * kPieces + lane) * V4::kSize;
        auto token = [&](int i) { return token0 + i * (32 * V4::kSize); };
        V4 v[kVecs];
        float top[kVecs], most = -INFINITY;
        if (off == 0 && at.step + 1 < all_steps) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i].load(from + i * 512, 0);
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                v[i].load(from + i * 512, off);
                if (token(i) + V4::kSize > p.V) v[i].cut(p.V - token(i));
            }
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            top[i] = v[i].most();
            most = fmaxf(most, top[i]);
        }
        // ---- sum of exponentials
        // of x - m: a row of one large number of either sign is level, too
        const float was = m;
        m = fmaxf(m, most);
        const float ref = m == -INFINITY ? 0.f : m;
        l *= exp2_approx((was - ref) * kLog2e);
        const uint64_t ref2 = pair_of(-ref, -ref), log2 = pair_of(kLog2e, kLog2e);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            uint64_t sum = 0;
#pragma unroll
            for (int j = 0; j < V4::kSize; j += 2) {
                float a, b;
                parts_of(mul_pair(add_pair(pair_of(v[i].at(j), v[i].at(j + 1)), ref2), log2), &a, &b);
                const uint64_t e = pair_of(exp2_approx(a), exp2_approx(b));
                sum = j ? add_pair(sum, e) : e;
            }
            float a, b;
            parts_of(sum, &a, &b);
            l += a + b;
        }
        // ---- keys at or above the bound
#pragma unroll
        for (int i = 0; i < kVecs; ++i) so_far[i] = fmaxf(so_far[i], top[i]);
        const At was_at = at;
        next(at);
        if (at.item == was_at.item) continue;
        // ---- the part is done: a bound of its K best logits
        uint32_t slot_key[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) slot_key[i] = value_key(so_far[i]);
        const uint32_t t = kth_of(slot_key, p.K);
        // (what is left of the bits of -inf may be no number)
        float bound = from_ordered(max(t, ordered(-INFINITY)));
        // the slots that reach it, in order
        int n_slots = 0;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, so_far[i] >= bound);
            if ((who >> lane) & 1u) slots[n_slots + __popc(who & ((1u << lane) - 1u))] = (uint8_t)(i * 32 + lane);
            n_slots += __popc(who);
        }
        __syncwarp();
        // their vectors of all steps, by token
        const int step0 = was_at.step0, n_vecs = n_slots * (was_at.end - step0);
        int have = 0;  // keys
        for (int q0 = 0; q0 < n_vecs; q0 += 32 * kLook) {
            // the loads of several then take the time of one
            V4 x[kLook];
            int first_token[kLook];
            uint32_t mine[kLook];
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                const int q = q0 + i * 32 + lane, step = q / n_slots;
                first_token[i] = q < n_vecs ? ((step0 + step) * kPieces + slots[q - step * n_slots]) * V4::kSize : p.V;
                if (first_token[i] < p.V) x[i].load(was_at.x, first_token[i], p.V);
            }
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                mine[i] = 0;
#pragma unroll
                for (int j = 0; j < V4::kSize; ++j)
                    mine[i] |= (first_token[i] + j < p.V && x[i].at(j) >= bound ? 1u : 0u) << j;
            }
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                bool full = false;  // the bound is a key's
                for (uint32_t any = __reduce_or_sync(0xFFFFFFFFu, mine[i]); any; any &= any - 1) {
                    const int j = __ffs(any) - 1;
                    const float y = x[i].any(j);
                    const bool take = ((mine[i] >> j) & 1u) && y >= bound;
                    uint32_t who = __ballot_sync(0xFFFFFFFFu, take);
                    if (have + __popc(who) > kRoom) {
                        rank_keys(keys, have, p.K, keys);
                        have = p.K;
                        bound = from_ordered((uint32_t)(keys[p.K - 1] >> 32));
                        full = true;
                        who = __ballot_sync(0xFFFFFFFFu, take && y >= bound);
                    }
                    if ((who >> lane) & 1u)
                        keys[have + __popc(who & ((1u << lane) - 1u))] =
                            (unsigned long long)value_key(y) << 32 | (uint32_t)~(first_token[i] + j);
                    have += __popc(who);
                    __syncwarp();
                }
                // tokens only grow from here on: equal values are not ahead of any of K keys
                if (full) bound = from_ordered(min(ordered(bound) + 1u, ordered(INFINITY)));
            }
        }
        const long long span = (long long)p.W * parts, place0 = was_at.item / span * span;
        unsigned long long* list = p.lists + place0 * p.K + (was_at.item - place0);
        rank_keys(keys, have, p.K, list, span);
        for (int i = have + lane; i < p.K; i += 32) list[i * span] = 0ull;
        const float mw = from_ordered(__reduce_max_sync(0xFFFFFFFFu, ordered(m)));
        l *= exp2_approx((m - (mw == -INFINITY ? 0.f : mw)) * kLog2e);
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        if (lane == 0) p.stats[was_at.item] = make_float2(mw, l);
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) so_far[i] = -INFINITY;
    }
    cp_async_wait<0>();
}

__global__ void __launch_bounds__(kThreads) beam_best_kernel(const BeamParams p) {
    __shared__ Rows rows;
    __shared__ Best best;
    if (threadIdx.x < 32) find_rows(p, rows, (long long)blockIdx.x * p.W);
    __syncthreads();
    pdl_wait();
    best_of_prompt(p, rows, best, blockIdx.x);
}

// How a call is cut: steps of a part of a row, its parts.  Each warp has one part of two steps at least: a
// step each makes twice the lists (8 beams of 50001 tokens for 8 prompts: 15.6 us, of single steps 21.6).  One CTA
// an SM up to 16384 steps, two above, where the memory counts more than the lists: 24 and 64 prompts of these
// 19.4 and 35.0 us with one, 22.6 and 31.8 with two; 32 and 64 of 4 beams of 131072 tokens 14.6 and 21.2, 16.9 and
// 20.8.  (A cluster for each prompt, whose first CTA takes the best: 18.3 us for the 8 prompts, 25.3 for the 24.)
struct Cut {
    int ctas, steps, parts;
    long long places;
};
constexpr int kSms = 152;
Cut cut_of(int N, int W, int V, int fp32) {
    const int steps = (V - 1) / (kPieces * (fp32 ? 4 : 8)) + 1;
    const long long rows = (long long)N * W, most = (rows * steps <= 16384 ? 1 : 2) * kSms;  // CTAs
    const long long each = rows ? most * kWarps / rows : steps;
    Cut c{};
    c.parts = each < 1 ? 1 : each < steps ? (int)each : steps;
    c.steps = (steps - 1) / c.parts + 1;
    if (c.steps == 1 && steps > 1) c.steps = 2;
    c.parts = (steps - 1) / c.steps + 1;
    c.places = rows * c.parts;
    c.ctas = (int)(c.places <= (most - 1) * kWarps ? (c.places + kWarps - 1) / kWarps : most);
    return c;
}

template <bool F32>
cudaError_t launch_of(const BeamParams& p, int ctas, cudaStream_t s) {
    static std::atomic<uint64_t> asked{0};  // devices on which the kernel may take its memory
    cudaError_t err = allow_shared(beam_kernel<F32>, kSmem, asked);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    // a kernel's blocks are placed while the one before it finishes
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, beam_kernel<F32>, p);
    if (err != cudaSuccess) return err;
    cfg.gridDim = dim3((unsigned)p.N);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, beam_best_kernel, p);
}

size_t stat_bytes(const Cut& c) { return ((size_t)c.places * sizeof(float2) + 255) / 256 * 256; }

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool shape_ok(int N, int W, int V, int K) {
    return N >= 0 && W > 0 && W <= kMostW && V > 0 && K > 0 && K <= kMostK && K <= (long long)W * V;
}

}  // namespace
}  // namespace mxq

extern "C" {

size_t mxq_beam_select_workspace_bytes(int N, int W, int V, int K, int fp32) {
    if (!mxq::shape_ok(N, W, V, K)) return 0;
    const mxq::Cut c = mxq::cut_of(N, W, V, fp32);
    return mxq::stat_bytes(c) + (size_t)c.places * K * sizeof(unsigned long long);
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
    const mxq::Cut c = mxq::cut_of(N, W, V, fp32);
    // tokens are counted in 32 bits, over a prompt's beams too, and CTAs
    if ((long long)W * V > 0x7FFFFFFF - 65536 || N > 0x7FFFFFFF / 8 ||
        (long long)W * (c.parts + 1) * (K + 1) > 0x7FFFFFFF) return MXQ_ERR_UNSUPPORTED;
    // a prompt's results take the place of its own scores only
    if (N > 1 && K != W && (out_scores == scores || (done && out_done == done))) return MXQ_ERR_INVALID_ARG;
    if (N > 0 && (!workspace || workspace_bytes < mxq_beam_select_workspace_bytes(N, W, V, K, fp32)))
        return MXQ_ERR_WORKSPACE;
    const mxq_status st = mxq::check_current_device(nullptr);
    if (st != MXQ_OK) return st;
    if (N == 0) return MXQ_OK;
    mxq::BeamParams p;
    p.logits = static_cast<const uint8_t*>(logits);
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
    p.steps = c.steps;
    p.parts = c.parts;
    p.end = end_token;
    p.stats = static_cast<float2*>(workspace);
    p.lists = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(workspace) +
                                                    mxq::stat_bytes(c));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t err = fp32 ? mxq::launch_of<true>(p, c.ctas, s) : mxq::launch_of<false>(p, c.ctas, s);
    return err == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

}  // extern "C"
