// Attention of a few query rows over a paged 4-bit key/value cache.
//
// For a row at position p and the keys t it sees (t <= p; with a window also
// t > p - window or t < sinks):
//   S_t = scale * q . k^_t,  P = softmax(S),  out = sum_t P_t v^_t
//   k^_td = s_tg q_td + b_tg, the same for v, g the group of value d
// The codes never become rounded values.  Per group,
//   q . k^_t = sum_g s_tg (q_g . c_t) + b_tg sum(q_g)
//   sum_t P_t v^_td = sum_t (P_t s_tg) c_td + sum_t P_t b_tg
// so the matrix instructions (m16n8k16, bf16 operands, fp32 sums) multiply the
// bf16 queries, or P_t s_tg rounded to bf16, with 16 + code, which bf16 holds
// exactly and which one shift and one logic operation make out of a pair of
// nibbles; scales, biases and the offset of 16 are applied in fp32 to a few
// numbers per token.  The rounding of P_t s_tg is the only one before the
// output's; it is taken against codes centred on 7.5 (the sum of the rounded
// P_t s_tg is kept beside the products), which halves its weight.
//
// Tokens are the instruction's rows (K) or its depth (V) and query rows its
// columns, so 8 rows of a key/value head's queries cost one instruction per
// 256 codes and 16 rows two.
//
// Work split: a unit is (row tile, tile of 64 tokens that it sees); the units
// of a plane, in order, are cut into equal runs, one per CTA, whatever the
// lengths of the sequences.  A run that begins or ends inside a row tile
// leaves its (max, sum, weighted sum) in the workspace and a second kernel
// joins them in order, so the result does not depend on timing.
//
// A CTA is one warp that copies whole page blocks (K codes, K pairs, V codes
// and V pairs of a head are contiguous: one bulk copy per page) into a ring of
// 64-token stages, and four warps that take 16 tokens of each stage with a
// softmax state of their own, joined at the end of a row tile.  The running
// maximum is only moved when a score exceeds it by 2^8, so most stages have no
// reductions across lanes at all.
// Bound by HBM for long contexts: 2 (D / 2 + 4 D / G) bytes per token and head.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_format.cuh"
#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "tc_common.cuh"

namespace mxq {
namespace {

constexpr int kWarps = 4;                       // compute warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStages = 4;
constexpr int kChunk = 64;                      // values joined at a time
constexpr int kRowPad = kChunk + 4;

enum : int { kNew = 1, kEnd = 2, kBegins = 4, kEnds = 8, kFull = 16, kLast = 32, kEmpty = 64 };

// What the compute warps need to know about a stage.
struct Stage {
    int row0;    // first row of q of the row tile
    int toks;    // its tokens
    int head0;   // its first query head
    int heads;   // its query heads
    int p0;      // position of its first token
    int t0;      // first token of this stage
    int flags;
    int valid;   // bit i: the 16 tokens from t0 + 16 i were copied
};

// Descriptor of a run's first or last piece of a row tile (workspace).
struct Seg {
    int row0, toks, head0, heads;
    int flags;  // kBegins, kEnds; -1: none
    int pad[3];
};

// What a row tile of a sequence sees.
struct Span {
    int row0, toks, p0;  // rows of q, tokens, position of the first
    int tiles;           // tiles of 64 tokens (at least 1 when it has rows)
    int head_tiles;      // the first of them, from token 0 on (sinks) ...
    int tail;            // ... and the tile where the rest begins
    int bad;             // the sequence's arguments are out of range
};

__device__ __forceinline__ Span span_of(const KvAttnParams& p, int s, int plane) {
    Span r;
    r.bad = 0;
    r.tiles = 0;
    r.head_tiles = 0;
    r.tail = 0;
    int a = s, b = s + 1;
    if (p.q_starts) {
        a = __ldg(p.q_starts + s);
        b = __ldg(p.q_starts + s + 1);
    }
    int len = __ldg(p.ctx_lens + s);
    const int most = p.max_pages * p.page_size;
    if (a < 0 || b > p.T || a > b || b - a > p.max_q || len < 0 || len > most) {
        r.bad = 1;
        if (a < 0 || b > p.T || a > b || b - a > p.max_q) b = a;  // none of its rows
        len = min(max(len, 0), most);
    }
    const int n = b - a;
    const int j0 = plane * p.tile_toks;
    r.row0 = a + j0;
    r.toks = min(p.tile_toks, n - j0);
    r.p0 = len - n + j0;
    if (r.toks <= 0) return r;
    const int hi = r.p0 + r.toks - 1;           // position of the last row
    const int end = hi < 0 ? 0 : hi / kKvTile + 1;
    int lo = 0;
    if (p.window) lo = max(0, r.p0 - p.window + 1) / kKvTile;
    int first = min((min(p.sinks, hi + 1) + kKvTile - 1) / kKvTile, end);
    if (first < 0) first = 0;
    if (first >= lo) first = lo = 0;
    lo = min(lo, end);
    r.head_tiles = first;
    r.tail = lo;
    r.tiles = max(1, first + end - lo);
    return r;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Nibble N of both halves of a word -> two bf16 numbers 16 + code.
template <int N>
__device__ __forceinline__ uint32_t codes16(uint32_t w) {
    constexpr uint32_t mask = 0x00780078u, base = 0x41804180u;
    const uint32_t x = N == 0 ? w << 3 : w >> (N == 1 ? 1 : N == 2 ? 5 : 9);
    return (x & mask) | base;
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

template <int D, int G, int NT>
struct Shape {
    static constexpr int kRows = NT * 8;
    static constexpr int kStageBytes = kv_block_bytes(D, G, kKvTile);
    static constexpr int kJoinBytes = kWarps * kRows * kRowPad * 4;
    static constexpr int kStatBytes = kWarps * kRows * 8;
    static constexpr int kSmem = kStages * kStageBytes + kJoinBytes + kStatBytes;
    static constexpr int kPartialFloats = kRows * (D + 2);
};

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t (&w)[W]) {
    if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {  // slabs of 128 values are 512 bytes apart
            const uint4 v = *reinterpret_cast<const uint4*>(at + 512 * i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
}

template <int NG>
__device__ __forceinline__ void load_pairs(const uint8_t* at, uint32_t (&w)[NG]) {
    if constexpr (NG == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(at);
    } else if constexpr (NG == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < NG / 4; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(at + 16 * i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
}

// One thread: walks the CTA's run of units, copies the stages' page blocks and
// describes each stage.
template <int D, int G>
__device__ void produce(const KvAttnParams& p, int plane, int cta, long long u0, long long u1,
                        int s, long long base, uint8_t* ring, Stage* stages, uint64_t* full,
                        uint64_t* empty) {
    constexpr int kStageBytes = kv_block_bytes(D, G, kKvTile);
    const int vheads = p.Hkv * p.head_parts;
    const int page = p.page_size;
    const int piece = page < kKvTile ? page : kKvTile;
    const long long block = kv_block_bytes(D, G, page);
    const int rep = p.Hq / p.Hkv;
    Seg* seg = reinterpret_cast<Seg*>(p.segs) + ((long long)plane * p.ctas + cta) * 2;
    if (p.segs) seg[0].flags = seg[1].flags = -1;
    long long issued = 0;
    uint32_t parity = 1;  // the first round of waits passes at once
    int slot = 0;
    bool ok = true;

    Span sp = span_of(p, s, plane);
    long long u = u0;
    while (u < u1 && ok) {
        while (u >= base + (long long)sp.tiles * vheads) {
            base += (long long)sp.tiles * vheads;
            sp = span_of(p, ++s, plane);
        }
        const int vh = (int)((u - base) / sp.tiles);
        int k = (int)((u - base) % sp.tiles);
        const int kend = (int)(u1 - u < sp.tiles - k ? k + (u1 - u) : sp.tiles);
        const int h = vh / p.head_parts, part = vh % p.head_parts;
        Stage st;
        st.row0 = sp.row0;
        st.toks = sp.toks;
        st.head0 = h * rep + part * p.part_heads;
        st.heads = min(p.part_heads, rep - part * p.part_heads);
        st.p0 = sp.p0;
        const int whole = (k == 0 ? kBegins : 0) | (kend == sp.tiles ? kEnds : 0);
        if (whole != (kBegins | kEnds)) {
            Seg g;
            g.row0 = st.row0;
            g.toks = st.toks;
            g.head0 = st.head0;
            g.heads = st.heads;
            g.flags = whole;
            seg[(whole & kBegins) ? 1 : 0] = g;
        }
        const int p1 = sp.p0 + sp.toks - 1;
        const int first = k;
        for (; k < kend; ++k, ++u) {
            const int tile = k < sp.head_tiles ? k : sp.tail + (k - sp.head_tiles);
            st.t0 = tile * kKvTile;
            st.flags = whole | (k == first ? kNew : 0) | (k == kend - 1 ? kEnd : 0) |
                       (u == u1 - 1 ? kLast : 0);
            const int tend = st.t0 + kKvTile - 1;
            if (tend <= sp.p0 && (!p.window || st.t0 > p1 - p.window || tend < p.sinks))
                st.flags |= kFull;
            if (!mbar_wait(&empty[slot], parity, p.wait_budget)) {
                flag_status(p.status, MXQ_DEV_TIMEOUT);
                ok = false;
                break;
            }
            // which pieces of the tile are there, and where
            st.valid = 0;
            uint32_t bytes = 0;
            const uint8_t* src[4] = {nullptr, nullptr, nullptr, nullptr};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = st.t0 + i * piece;
                if (i * piece < kKvTile && t <= p1) {
                    const int id = __ldg(p.table + (long long)s * p.max_pages + t / page);
                    if (id >= 0 && id < p.n_pages) {
                        src[i] = p.pages + ((long long)id * p.Hkv + h) * block;
                        const int sixteens = piece / 16;
                        st.valid |= ((1 << sixteens) - 1) << (i * sixteens);
                        bytes += page <= kKvTile ? (uint32_t)block : (uint32_t)kStageBytes;
                    } else {
                        // a page that some row sees has to exist
                        const int te = min(t + piece - 1, p1);
                        if (!p.window || te > sp.p0 - p.window || t < p.sinks)
                            flag_status(p.status, MXQ_DEV_BAD_PAGE);
                    }
                }
            }
            if (st.valid != 15) st.flags &= ~kFull;
            stages[slot] = st;
            mbar_expect_tx(&full[slot], bytes);
            const uint32_t dst = smem_u32(ring + slot * kStageBytes);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!src[i]) continue;
                if (page <= kKvTile) {
                    bulk_copy(dst + i * (uint32_t)block, src[i], (uint32_t)block, &full[slot]);
                } else {  // a 64-token part of a longer page: its four regions
                    const int o = st.t0 % page;
                    const uint32_t cb = kv_code_bytes(D, kKvTile), pb = kv_pair_bytes(D, G, kKvTile);
                    const uint8_t* kc = src[i] + kv_code_bytes(D, o);
                    const uint8_t* kp = src[i] + kv_code_bytes(D, page) + kv_pair_bytes(D, G, o);
                    const long long v = block / 2;
                    bulk_copy(dst, kc, cb, &full[slot]);
                    bulk_copy(dst + cb, kp, pb, &full[slot]);
                    bulk_copy(dst + cb + pb, kc + v, cb, &full[slot]);
                    bulk_copy(dst + 2 * cb + pb, kp + v, pb, &full[slot]);
                }
            }
            ++issued;
            if (++slot == kStages) {
                slot = 0;
                parity ^= 1u;
            }
        }
    }
    drain_ring(full, kStages, issued, kStages);
}

template <int D, int G, int NT>
__global__ void __launch_bounds__(kThreads, (D == 256 || NT == 2) ? 2 : 3)
    kv_attn_kernel(const KvAttnParams p) {
    using SH = Shape<D, G, NT>;
    constexpr int NG = D / G;       // groups
    constexpr int U = D / 32;       // code words of a lane per 8 tokens
    constexpr int MT = D / 16;      // output tiles of 16 values
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kStages], empty[kStages], joined;
    __shared__ Stage stages[kStages];
    __shared__ long long sums[kThreads];
    uint8_t* ring = smem;
    float* join = reinterpret_cast<float*>(smem + kStages * SH::kStageBytes);
    float2* stat = reinterpret_cast<float2*>(smem + kStages * SH::kStageBytes + SH::kJoinBytes);

    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int plane = blockIdx.x / p.ctas, cta = blockIdx.x % p.ctas;

    // every CTA finds its own run: the units of all sequences, then its share
    const int per = (p.S + kThreads - 1) / kThreads;
    {
        long long sum = 0;
        for (int i = 0; i < per; ++i) {
            const int s = threadIdx.x * per + i;
            if (s >= p.S) break;
            const Span sp = span_of(p, s, plane);
            sum += sp.tiles;
            if (sp.bad && blockIdx.x == 0) flag_status(p.status, MXQ_DEV_BAD_SEQUENCE);
        }
        sums[threadIdx.x] = sum * (p.Hkv * p.head_parts);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWarps);
        }
        mbar_init(&joined, kWarps);
        mbar_init_fence();
    }
    __syncthreads();

    if (warp == kWarps) {
        // scan of the threads' sums: 5 of them a lane
        constexpr int kPer = kThreads / 32;
        long long mine = 0;
        for (int i = 0; i < kPer; ++i) mine += sums[lane * kPer + i];
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += x;
        }
        const long long total = __shfl_sync(0xFFFFFFFFu, incl, 31);
        const long long runs = total < p.ctas ? total : p.ctas;
        const long long u0 = cta < runs ? cta * total / runs : 0;
        const long long u1 = cta < runs ? (cta + 1) * total / runs : 0;
        if (u0 == u1) {
            if (lane == 0) {
                Seg* seg = reinterpret_cast<Seg*>(p.segs) + ((long long)plane * p.ctas + cta) * 2;
                if (p.segs) seg[0].flags = seg[1].flags = -1;
                stages[0].flags = kLast | kEmpty;
                mbar_arrive(&full[0]);
            }
        } else {
            const uint32_t here = __ballot_sync(0xFFFFFFFFu, u0 >= incl - mine && u0 < incl);
            if (lane == __ffs(here) - 1) {
                long long base = incl - mine;
                int i = lane * kPer;
                while (u0 >= base + sums[i]) base += sums[i++];
                // sequences of that thread, one by one (produce skips on)
                produce<D, G>(p, plane, cta, u0, u1, i * per, base, ring, stages, full, empty);
            }
        }
        return;
    }

    // ------------------------------------------------------- compute warps
    const int r = lane >> 2, i4 = lane & 3;
    uint32_t qf[NT][U][4];
    float qsum[NT][NG][2];     // sum of q over a group, rows 2 i4 and 2 i4 + 1
    float acc[NT][MT][4], psum[NT][NG][4];
    float pb[NT][NG][2], l[NT][2], m[NT][2], mu[NT][2];
    int pos[NT][2];
    int slot = 0;
    uint32_t parity = 0, jparity = 0;

    const int piece = p.page_size < kKvTile ? p.page_size : kKvTile;
    const int in_piece = (warp * 16) % piece;
    const int piece_at = (warp * 16) / piece * kv_block_bytes(D, G, piece);
    const int kc_at = piece_at + kv_code_bytes(D, in_piece) + lane * (D == 64 ? 8 : 16);
    const int kp_at = piece_at + kv_code_bytes(D, piece) + (in_piece + r) * NG * 4;
    const int v_off = kv_block_bytes(D, G, piece) / 2;

    for (;;) {
        if (!warp_wait(&full[slot], parity, p.wait_budget)) {
            if (lane == 0) flag_status(p.status, MXQ_DEV_TIMEOUT);
            return;
        }
        const Stage st = stages[slot];
        if (st.flags & kEmpty) return;
        if (st.flags & kNew) {
            // a row tile begins: its queries as the instruction's columns
            const int rows = st.toks * st.heads;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int rr = nt * 8 + r;
                const bool in = rr < rows;
                const int j = in ? rr / st.heads : 0, hh = in ? rr % st.heads : 0;
                const __nv_bfloat16* src = p.q + (long long)(st.row0 + j) * p.q_row_stride +
                                           (long long)(st.head0 + hh) * p.q_head_stride + 8 * i4;
                float part[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) part[g] = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (in) v = __ldg(reinterpret_cast<const uint4*>(src + 32 * u));
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    // pairs (0, 4), (1, 5), (2, 6), (3, 7), as a code word's nibbles
                    qf[nt][u][0] = prmt(w[0], w[2], 0x5410u);
                    qf[nt][u][1] = prmt(w[0], w[2], 0x7632u);
                    qf[nt][u][2] = prmt(w[1], w[3], 0x5410u);
                    qf[nt][u][3] = prmt(w[1], w[3], 0x7632u);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        part[u * 32 / G] += __uint_as_float(w[e] << 16) +
                                            __uint_as_float(w[e] & 0xFFFF0000u);
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float x = part[g];
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
                    qsum[nt][g][0] = __shfl_sync(0xFFFFFFFFu, x, 8 * i4);
                    qsum[nt][g][1] = __shfl_sync(0xFFFFFFFFu, x, 8 * i4 + 4);
                    pb[nt][g][0] = pb[nt][g][1] = 0.f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) psum[nt][g][c] = 0.f;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = nt * 8 + 2 * i4 + c;
                    pos[nt][c] = col < rows ? st.p0 + col / st.heads : -1;
                    m[nt][c] = -INFINITY;
                    mu[nt][c] = 0.f;
                    l[nt][c] = 0.f;
                }
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[nt][t][c] = 0.f;
            }
        }

        const uint8_t* at = ring + slot * SH::kStageBytes;
        // ---- scores of 16 tokens: rows r and r + 8 of the instruction
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[nt][c] = 0.f;
        {
            uint32_t w0[U], w1[U], pr0[NG], pr1[NG];
            load_words<U>(at + kc_at, w0);
            load_words<U>(at + kc_at + 4 * D, w1);
            load_pairs<NG>(at + kp_at, pr0);
            load_pairs<NG>(at + kp_at + 8 * NG * 4, pr1);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float a[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) a[nt][c] = 0.f;
#pragma unroll
                for (int u = g * G / 32; u < (g + 1) * G / 32; ++u) {
                    const uint32_t x0 = codes16<0>(w0[u]), y0 = codes16<0>(w1[u]);
                    const uint32_t x1 = codes16<1>(w0[u]), y1 = codes16<1>(w1[u]);
                    const uint32_t x2 = codes16<2>(w0[u]), y2 = codes16<2>(w1[u]);
                    const uint32_t x3 = codes16<3>(w0[u]), y3 = codes16<3>(w1[u]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_bf16(a[nt], x0, y0, x1, y1, qf[nt][u][0], qf[nt][u][1]);
                        mma_bf16(a[nt], x2, y2, x3, y3, qf[nt][u][2], qf[nt][u][3]);
                    }
                }
                const float s0 = __uint_as_float(pr0[g] << 16) * p.scale_log2;
                const float s1 = __uint_as_float(pr1[g] << 16) * p.scale_log2;
                const float b0 = fmaf(-16.f, s0, __uint_as_float(pr0[g] & 0xFFFF0000u) * p.scale_log2);
                const float b1 = fmaf(-16.f, s1, __uint_as_float(pr1[g] & 0xFFFF0000u) * p.scale_log2);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    sc[nt][0] = fmaf(s0, a[nt][0], fmaf(b0, qsum[nt][g][0], sc[nt][0]));
                    sc[nt][1] = fmaf(s0, a[nt][1], fmaf(b0, qsum[nt][g][1], sc[nt][1]));
                    sc[nt][2] = fmaf(s1, a[nt][2], fmaf(b1, qsum[nt][g][0], sc[nt][2]));
                    sc[nt][3] = fmaf(s1, a[nt][3], fmaf(b1, qsum[nt][g][1], sc[nt][3]));
                }
            }
        }
        bool live0 = true, live1 = true;  // tokens r and r + 8 are seen by some row
        if (!(st.flags & kFull)) {
            const int t0 = st.t0 + warp * 16 + r, t1 = t0 + 8;
            const bool there = (st.valid >> warp) & 1;
            const int p1 = st.p0 + st.toks - 1;
            live0 = there && t0 <= p1 && (!p.window || t0 > st.p0 - p.window || t0 < p.sinks);
            live1 = there && t1 <= p1 && (!p.window || t1 > st.p0 - p.window || t1 < p.sinks);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int q = pos[nt][c];
                    if (!(live0 && t0 <= q && (!p.window || t0 > q - p.window || t0 < p.sinks)))
                        sc[nt][c] = -INFINITY;
                    if (!(live1 && t1 <= q && (!p.window || t1 > q - p.window || t1 < p.sinks)))
                        sc[nt][2 + c] = -INFINITY;
                }
            }
        }
        // ---- running maximum: moved only when a score is far above it
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                over |= fmaxf(sc[nt][c], sc[nt][2 + c]) > m[nt][c] + 8.f;
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x = fmaxf(sc[nt][c], sc[nt][2 + c]);
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                    const float mn = fmaxf(m[nt][c], x);
                    const float ref = mn == -INFINITY ? 0.f : mn;
                    const float f = exp2_approx(m[nt][c] - ref);
                    m[nt][c] = mn;
                    mu[nt][c] = ref;
                    l[nt][c] *= f;
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        pb[nt][g][c] *= f;
                        psum[nt][g][c] *= f;
                    }
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        acc[nt][t][c] *= f;
                        acc[nt][t][2 + c] *= f;
                    }
                }
            }
        }
        // ---- weights
        float w[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 4; ++c) w[nt][c] = exp2_approx(sc[nt][c] - mu[nt][c & 1]);
            l[nt][0] += w[nt][0] + w[nt][2];
            l[nt][1] += w[nt][1] + w[nt][3];
        }
        // ---- weighted sum of the values
        {
            uint32_t w0[U], w1[U], pr0[NG], pr1[NG];
            load_pairs<NG>(at + v_off + kp_at, pr0);
            load_pairs<NG>(at + v_off + kp_at + 8 * NG * 4, pr1);
            load_words<U>(at + v_off + kc_at, w0);
            load_words<U>(at + v_off + kc_at + 4 * D, w1);
            constexpr uint32_t one = 0x3F803F80u;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float s0 = live0 ? __uint_as_float(pr0[g] << 16) : 0.f;
                const float s1 = live1 ? __uint_as_float(pr1[g] << 16) : 0.f;
                const float b0 = live0 ? fmaf(7.5f, s0, __uint_as_float(pr0[g] & 0xFFFF0000u)) : 0.f;
                const float b1 = live1 ? fmaf(7.5f, s1, __uint_as_float(pr1[g] & 0xFFFF0000u)) : 0.f;
                uint32_t f0[NT], f1[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    f0[nt] = transpose_8x8(cvt_bf16x2(w[nt][0] * s0, w[nt][1] * s0));
                    f1[nt] = transpose_8x8(cvt_bf16x2(w[nt][2] * s1, w[nt][3] * s1));
                    pb[nt][g][0] = fmaf(w[nt][0], b0, fmaf(w[nt][2], b1, pb[nt][g][0]));
                    pb[nt][g][1] = fmaf(w[nt][1], b0, fmaf(w[nt][3], b1, pb[nt][g][1]));
                    mma_bf16(psum[nt][g], one, one, one, one, f0[nt], f1[nt]);
                }
#pragma unroll
                for (int u = g * G / 32; u < (g + 1) * G / 32; ++u) {
                    const uint32_t x0 = codes16<0>(w0[u]), y0 = codes16<0>(w1[u]);
                    const uint32_t x1 = codes16<1>(w0[u]), y1 = codes16<1>(w1[u]);
                    const uint32_t x2 = codes16<2>(w0[u]), y2 = codes16<2>(w1[u]);
                    const uint32_t x3 = codes16<3>(w0[u]), y3 = codes16<3>(w1[u]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_bf16(acc[nt][2 * u], x0, x1, y0, y1, f0[nt], f1[nt]);
                        mma_bf16(acc[nt][2 * u + 1], x2, x3, y2, y3, f0[nt], f1[nt]);
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (++slot == kStages) {
            slot = 0;
            parity ^= 1u;
        }

        if (st.flags & kEnd) {
            // ---- the four warps' results of this row tile become one
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x = l[nt][c];
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
                    if (r == 0)
                        stat[warp * SH::kRows + nt * 8 + 2 * i4 + c] = make_float2(m[nt][c], x);
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        float y = pb[nt][g][c];
                        y += __shfl_xor_sync(0xFFFFFFFFu, y, 4);
                        y += __shfl_xor_sync(0xFFFFFFFFu, y, 8);
                        y += __shfl_xor_sync(0xFFFFFFFFu, y, 16);
                        pb[nt][g][c] = fmaf(-23.5f, psum[nt][g][c], y);
                    }
                }
            }
            const bool whole = (st.flags & kBegins) && (st.flags & kEnds);
            float* part = p.partial + (((long long)plane * p.ctas + cta) * 2 +
                                       ((st.flags & kBegins) ? 1 : 0)) *
                                          SH::kPartialFloats;
            const int rows = st.toks * st.heads;
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += kChunk) {
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if (t / (kChunk / 16) != d0 / kChunk) continue;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            join[(warp * SH::kRows + nt * 8 + 2 * i4 + (c & 1)) * kRowPad +
                                 (t % (kChunk / 16)) * 16 + r + (c >> 1) * 8] =
                                acc[nt][t][c] + pb[nt][t * 16 / G][c & 1];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&joined);
                if (!warp_wait(&joined, jparity, p.wait_budget)) {
                    if (lane == 0) flag_status(p.status, MXQ_DEV_TIMEOUT);
                    return;
                }
                jparity ^= 1u;
#pragma unroll
                for (int e = 0; e < NT; ++e) {
                    const int row = e * 8 + threadIdx.x / 16, d = (threadIdx.x % 16) * 4;
                    float mm = -INFINITY;
#pragma unroll
                    for (int wi = 0; wi < kWarps; ++wi)
                        mm = fmaxf(mm, stat[wi * SH::kRows + row].x);
                    const float ref = mm == -INFINITY ? 0.f : mm;
                    float ll = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int wi = 0; wi < kWarps; ++wi) {
                        const float2 ml = stat[wi * SH::kRows + row];
                        const float f = exp2_approx(ml.x - ref);
                        ll = fmaf(ml.y, f, ll);
                        const float4 x = *reinterpret_cast<const float4*>(
                            join + (wi * SH::kRows + row) * kRowPad + d);
                        o.x = fmaf(x.x, f, o.x);
                        o.y = fmaf(x.y, f, o.y);
                        o.z = fmaf(x.z, f, o.z);
                        o.w = fmaf(x.w, f, o.w);
                    }
                    if (row >= rows) continue;
                    if (whole) {
                        const long long to = (long long)(st.row0 + row / st.heads) * p.Hq +
                                             st.head0 + row % st.heads;
                        const float inv = ll > 0.f ? 1.f / ll : 0.f;
                        uint2 v;
                        v.x = cvt_bf16x2(o.x * inv, o.y * inv);
                        v.y = cvt_bf16x2(o.z * inv, o.w * inv);
                        *reinterpret_cast<uint2*>(p.out + to * D + d0 + d) = v;
                        if (p.lse && d0 + d == 0)
                            p.lse[to] = ll > 0.f ? (mm + log2f(ll)) * 0.69314718f : -INFINITY;
                    } else {
                        *reinterpret_cast<float4*>(part + 2 * SH::kRows + row * D + d0 + d) = o;
                        if (d0 + d == 0) {
                            part[2 * row] = mm;
                            part[2 * row + 1] = ll;
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&joined);
                if (!warp_wait(&joined, jparity, p.wait_budget)) {
                    if (lane == 0) flag_status(p.status, MXQ_DEV_TIMEOUT);
                    return;
                }
                jparity ^= 1u;
            }
        }
        if (st.flags & kLast) return;
    }
}

// Joins the pieces of the row tiles that were cut: the CTA whose last piece
// begins one is followed by those that go on with it, in order.
template <int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const KvAttnParams p, int tile_rows) {
    const int plane = blockIdx.x / p.ctas, cta = blockIdx.x % p.ctas;
    const long long base = (long long)plane * p.ctas;
    const Seg* segs = reinterpret_cast<const Seg*>(p.segs);
    const Seg g = segs[(base + cta) * 2 + 1];
    if (g.flags < 0 || !(g.flags & kBegins) || (g.flags & kEnds)) return;
    // after a wait that gave up the descriptors may be anything
    if (g.toks <= 0 || g.heads <= 0 || g.toks > tile_rows || g.heads > tile_rows ||
        g.toks * g.heads > tile_rows || g.row0 < 0 || g.row0 > p.T - g.toks || g.head0 < 0 ||
        g.head0 > p.Hq - g.heads)
        return;
    int last = cta;
    while (last + 1 < p.ctas) {
        ++last;
        const int f = segs[(base + last) * 2].flags;
        if (f < 0 || (f & kEnds)) break;
    }
    const long long stride = (long long)tile_rows * (D + 2);
    const float* first = p.partial + ((base + cta) * 2 + 1) * stride;
    const float* next = p.partial + (base + cta) * 2 * stride;  // piece 0 of CTA cta + k: + 2 k
    const int rows = g.toks * g.heads, n = last - cta;
    for (int i = threadIdx.x; i < rows * (D / 4); i += blockDim.x) {
        const int row = i / (D / 4), d = (i % (D / 4)) * 4;
        float mm = first[2 * row];
        for (int k = 1; k <= n; ++k) mm = fmaxf(mm, next[2 * k * stride + 2 * row]);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float f = exp2_approx(first[2 * row] - ref);
        float ll = first[2 * row + 1] * f;
        const float4 x = *reinterpret_cast<const float4*>(first + 2 * tile_rows + row * D + d);
        float4 o = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
#pragma unroll 4
        for (int k = 1; k <= n; ++k) {
            const float* q = next + 2 * k * stride;
            const float2 ml = *reinterpret_cast<const float2*>(q + 2 * row);
            const float4 y = *reinterpret_cast<const float4*>(q + 2 * tile_rows + row * D + d);
            f = exp2_approx(ml.x - ref);
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
        if (p.lse && d == 0) p.lse[to] = ll > 0.f ? (mm + log2f(ll)) * 0.69314718f : -INFINITY;
    }
}

template <int D, int G, int NT>
cudaError_t launch(const KvAttnParams& p, cudaStream_t stream) {
    using SH = Shape<D, G, NT>;
    cudaError_t err = cudaFuncSetAttribute(kv_attn_kernel<D, G, NT>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, SH::kSmem);
    if (err != cudaSuccess) return err;
    const unsigned grid = (unsigned)(p.planes * p.ctas);
    kv_attn_kernel<D, G, NT><<<grid, kThreads, SH::kSmem, stream>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess || !p.segs) return err;
    kv_join_kernel<D><<<grid, 256, 0, stream>>>(p, SH::kRows);
    return cudaGetLastError();
}

}  // namespace

size_t kv_attn_seg_bytes(int planes, int ctas) { return (size_t)planes * ctas * 2 * sizeof(Seg); }

size_t kv_attn_partial_bytes(int planes, int ctas, int tile_rows, int D) {
    return (size_t)planes * ctas * 2 * tile_rows * (D + 2) * sizeof(float);
}

int kv_attn_ctas_per_sm(int D, int tile_rows) { return D == 256 || tile_rows > 8 ? 2 : 3; }

cudaError_t launch_kv_attn(const KvAttnParams& p, int D, int G, int tile_rows,
                           cudaStream_t stream) {
#define MXQ_KV_ATTN(d, g)                                                     \
    if (D == d && G == g)                                                     \
        return tile_rows <= 8 ? launch<d, g, 1>(p, stream) : launch<d, g, 2>(p, stream);
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
