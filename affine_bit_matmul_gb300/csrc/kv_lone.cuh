// Attention of a few query rows over a paged 4-bit key/value cache by warps on their own, for
// the parts of a call over shared prefixes: a run of a warp (kv_shared.cuh) is a few hundred tokens.
//
// The mathematics is kv_attention.cu's: codes as f16 subnormals in m16n8k16, scales and biases in
// fp32, the running maximum moved only when a score exceeds it by 2^8, sums centred every 512
// tokens.  What differs is who does what: each warp has a run and a ring of tiles of its own, into
// which it copies pages (bulk copies) as far ahead as there is room, past the ends of row tiles, and a
// piece of a row tile leaves its (largest score, sum, weighted sum) in the workspace as it is.  No warp
// waits for another, and nothing is shared but the list of items.  Where contexts are short, the ends of
// row tiles are most of the work, and they cost a few stores here.
//   16 groups of 8 sequences, 32 query heads over 8 of 128 values, 2048 + 256 tokens (51 MB of cache): some 53 us of
// 57 for the call.  Bound by instructions, 18.7 million of its warps at 1.35 a cycle and SM: 38% of a warp's time
// goes by without the next one having been fetched, since the warps of an SM are at different places of loops that
// are longer than the nearest caches.  12 us are the start (lists, pieces, page numbers, queries, first tiles).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_attn_common.cuh"
#include "kv_shared.cuh"

namespace mxq {
namespace {

constexpr int kLoneThreads = 128;
constexpr int kLoneWarps = kLoneThreads / 32;
constexpr int kLoneChain = 512;  // tokens whose value products are added before the means are taken out

constexpr int kLonePieces = 8;   // of which a warp knows ahead

// Row tiles of 4 KT rows.
template <int D, int G, int KT>
struct Lone {
    static constexpr int kRows = 4 * KT;
    static constexpr int kTile = D == 256 ? 16 : 32;  // tokens
    static constexpr int kColumns = (KT + 1) / 2;  // tiles of 8 columns
    // the queries lie in shared memory where they would take 32 registers or more
    static constexpr bool kQueryShared = D * kColumns >= 256;
    // Rows of up to 8 come as they are into shared memory while the piece before is worked on.
    static constexpr bool kQueryAhead = KT <= 2;
    static constexpr int kRawBytes = kQueryAhead ? kRows * D * 2 : 0;  // of a warp
    static constexpr int kQueryBytes = (kQueryShared ? kColumns * D * 16 : 0) + kRawBytes;
    // CTAs of an SM, by the registers of a thread: 128, 168, 255
    static constexpr int kCtas = D == 256 ? (KT == 1 ? 3 : 2) : KT == 4 ? 3 : 4;
};

// What two kinds of row tiles in one kernel have.
template <int D, int G, int KT1, int KT2>
struct LoneBoth {
    using A = Lone<D, G, KT1>;
    using B = Lone<D, G, KT2>;
    static constexpr int kCtas = A::kCtas < B::kCtas ? A::kCtas : B::kCtas;
    static constexpr int kQueryBytes = A::kQueryBytes > B::kQueryBytes ? A::kQueryBytes : B::kQueryBytes;
    static constexpr int kStageBytes = kv_block_bytes(D, G, A::kTile);
    static constexpr int kRoom = (222 * 1024 / kCtas - 6 * 1024) / kLoneWarps - kQueryBytes;  // (6 KB: static)
    static constexpr int kSlots = kRoom / kStageBytes < 4 ? kRoom / kStageBytes : 4;
    static constexpr int kWarpBytes = kSlots * kStageBytes + kQueryBytes;
    static constexpr int kSmem = kLoneWarps * kWarpBytes;
    static_assert(kSlots >= 2 && kSlots <= 4);
};

// A warp's ring, what is known of the pieces ahead, and where the copies are: at a tile of piece
// number `piece`; the one after it is known too.
template <int SLOTS>
struct LoneRing {
    uint64_t full[SLOTS], query;
    int there[SLOTS];  // bit b: the slot's 16 tokens from 16 b on exist
    SharedPiece pieces[kLonePieces];  // count 0: the run is over
    SharedWalk walk;
    int n, piece;      // tiles copied so far
    int left, t0;      // of the piece: tiles not copied yet (-1: the run is over), the first of them
};

// The page numbers that a warp holds: lane i that of a piece's page `first` + i; -2: not needed.
struct LonePages {
    int id, first;
};

// Finds piece `number` of the run.
template <int SLOTS>
__device__ __forceinline__ void lone_walk(const KvSharedParams& p, LoneRing<SLOTS>& ring, int number) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        SharedPiece q;
        if (ring.walk.next(p, &q)) find_rows(p, q);
        ring.pieces[number % kLonePieces] = q;
    }
    __syncwarp();
}

// A piece's page numbers from the page of token t0 on.
__device__ __forceinline__ LonePages lone_pages(const KvSharedParams& p, const SharedPiece& q, int t0) {
    LonePages r;
    r.first = t0 >> p.page_shift;
    const int page = r.first + (threadIdx.x & 31);
    r.id = q.count && page <= q.p1 >> p.page_shift ? *(p.table + (long long)q.item * p.max_pages + page) : -2;
    return r;
}

// Goes to the next piece, and looks up what the one after it needs.
template <int TILE, int SLOTS>
__device__ __forceinline__ void lone_next(const KvSharedParams& p, LoneRing<SLOTS>& ring, LonePages& pages,
                                          LonePages& later) {
    __syncwarp();
    const int n = ring.piece + 1;
    const SharedPiece& q = ring.pieces[n % kLonePieces];
    pages = later;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        ring.piece = n;
        ring.left = q.count ? q.count : -1;
        ring.t0 = q.k0 * TILE;
    }
    __syncwarp();
    if (ring.left < 0) return;
    lone_walk(p, ring, n + 1);
    const SharedPiece& r = ring.pieces[(n + 1) % kLonePieces];
    later = lone_pages(p, r, r.k0 * TILE);
}

// Copies the next tile; the whole warp.
template <int D, int G, int TILE, int SLOTS>
__device__ __forceinline__ void lone_copy(const KvSharedParams& p, LoneRing<SLOTS>& ring, uint32_t data,
                                          LonePages& pages, LonePages& later) {
    if (ring.left == 0) lone_next<TILE>(p, ring, pages, later);
    if (ring.left < 0) return;
    constexpr uint32_t stage = kv_block_bytes(D, G, TILE);
    const SharedPiece& q = ring.pieces[ring.piece % kLonePieces];
    const int lane = threadIdx.x & 31, slot = ring.n % SLOTS, size = p.page_size, t0 = ring.t0, p1 = q.p1;
    const uint32_t to = data + slot * stage;
    const long long block = kv_block_bytes(D, G, size);
    if (min(t0 + TILE - 1, p1) >> p.page_shift >= pages.first + 32) pages = lone_pages(p, q, t0);
    int id[TILE / 16];
#pragma unroll
    for (int b = 0; b < TILE / 16; ++b) {
        const int t = t0 + 16 * b, x = __shfl_sync(0xFFFFFFFFu, pages.id, ((t >> p.page_shift) - pages.first) & 31);
        id[b] = t <= p1 ? x : -2;
    }
    const bool a = (unsigned)id[0] < (unsigned)p.n_pages;
    const bool b = TILE == 32 && (unsigned)id[TILE / 16 - 1] < (unsigned)p.n_pages;
    const bool halves = TILE == 32 && size == 16;  // two pages a tile
    const uint8_t* src = p.pages + ((long long)id[0] * p.Hkv + q.h) * block;
    __syncwarp();
    if (lane == 0) {
        ring.there[slot] = (a ? 1 : 0) | (b ? 2 : 0);
        // a page that some row sees has to exist
        if ((!a && id[0] != -2) || (TILE == 32 && !b && id[TILE / 16 - 1] != -2)) flag_status(p.status, MXQ_DEV_BAD_PAGE);
        mbar_expect_tx(&ring.full[slot], halves ? (a ? stage / 2 : 0) + (b ? stage / 2 : 0) : a ? stage : 0);
        ++ring.n;
        --ring.left;
        ring.t0 = t0 + TILE;
    }
    __syncwarp();
    if (size <= TILE) {
        // whole blocks
        if (lane == 0 && a) bulk_copy(to, src, (uint32_t)block, &ring.full[slot]);
        if (halves && lane == 1 && b)
            bulk_copy(to + stage / 2, p.pages + ((long long)id[TILE / 16 - 1] * p.Hkv + q.h) * block, stage / 2, &ring.full[slot]);
    } else if (a && lane < 4) {
        // the part of each region that the tile is
        constexpr uint32_t cb = kv_code_bytes(D, TILE), pb = kv_pair_bytes(D, G, TILE);
        const int skip = t0 & (size - 1);
        src += (lane >> 1) * (block / 2) +
               (lane & 1 ? kv_code_bytes(D, size) + kv_pair_bytes(D, G, skip) : kv_code_bytes(D, skip));
        bulk_copy(to + (lane >> 1) * (cb + pb) + (lane & 1) * cb, src, lane & 1 ? pb : cb, &ring.full[slot]);
    }
}

// Copies the queries of piece q, up to 8 rows.
template <int D, int SLOTS>
__device__ __forceinline__ void lone_queries(const KvSharedParams& p, LoneRing<SLOTS>& ring, const SharedPiece& q,
                                             uint32_t to) {
    const int lane = threadIdx.x & 31;
    if (q.count == 0) return;
    if (lane == 0) mbar_expect_tx(&ring.query, q.rows * D * 2);
    __syncwarp();
    if (lane < q.rows) {
        const int flat = q.flat0 + lane, j = flat / q.heads;
        bulk_copy(to + lane * D * 2,
                  p.q + (long long)(q.it.row0 + j) * p.q_row_stride + (long long)(q.head0 + flat - j * q.heads) * p.q_head_stride,
                  D * 2, &ring.query);
    }
}

// After a wait that gave up: no copy may land after the CTA is gone.
template <int SLOTS>
__device__ __noinline__ bool lone_stop(LoneRing<SLOTS>& ring, int tiles, bool queries, int queried) {
    for (int i = tiles; i < ring.n; ++i) mbar_wait(&ring.full[i % SLOTS], (uint32_t)(i / SLOTS) & 1u);
    if (queries) mbar_wait(&ring.query, (uint32_t)queried & 1u);
    return false;
}

// A warp's pieces of the run.  False if a wait gave up.
template <int D, int G, int KT, int SLOTS>
__device__ __forceinline__ bool lone_run(const KvSharedParams& p, int runner, LoneRing<SLOTS>& ring, uint8_t* data,
                                         uint4* queries) {
    using LN = Lone<D, G, KT>;
    constexpr int NG = D / G, U = D / 32, MT = D / 16, VT = LN::kColumns, TILE = LN::kTile, SUB = TILE / 16;
    constexpr int kStage = kv_block_bytes(D, G, TILE);
    const int lane = threadIdx.x & 31, r = lane >> 2, i4 = lane & 3;
    const uint32_t slots = smem_u32(data);
    // the queries as they come, behind those as operands
    const uint8_t* raw_rows = reinterpret_cast<const uint8_t*>(queries) + (LN::kQueryBytes - LN::kRawBytes);
    // the first two pieces
    lone_walk(p, ring, 0);
    lone_walk(p, ring, 1);
    LonePages pages{-2, 0}, later = lone_pages(p, ring.pieces[0], ring.pieces[0].k0 * TILE);
    if (LN::kQueryAhead) lone_queries<D>(p, ring, ring.pieces[0], smem_u32(raw_rows));
    {
        const LonePages first = later;
        later = lone_pages(p, ring.pieces[1], ring.pieces[1].k0 * TILE);
        pages = first;
        __syncwarp();
        if (lane == 0) {
            ring.piece = 0;
            ring.left = ring.pieces[0].count;
            ring.t0 = ring.pieces[0].k0 * TILE;
        }
        __syncwarp();
    }
    for (int i = 0; i < SLOTS; ++i) lone_copy<D, G, TILE>(p, ring, slots, pages, later);
    // offsets in a slot of this lane's words and pairs of 16 tokens: a page's block of `unit` tokens
    // after another
    const int page = p.page_size < TILE ? p.page_size : TILE, page_block = kv_block_bytes(D, G, page);
    const int v_off = page_block / 2;
    const int words_1 = page == 32 ? 8 * D : page_block, pairs_1 = page == 32 ? 64 * NG : page_block;
    const int words_0 = lane * (D == 64 ? 8 : 16), pairs_0 = kv_code_bytes(D, page) + r * NG * 4;
    int u = 0, queried = 0;  // tiles, pieces' queries so far
    for (int n_piece = 0;; ++n_piece) {
        __syncwarp();
        const SharedPiece& pc = ring.pieces[n_piece % kLonePieces];
        const int count = pc.count;
        if (count == 0) return true;
        const int head0 = pc.head0, heads = pc.heads, flat0 = pc.flat0, rows = pc.rows, p1 = pc.p1;
        const int row0 = pc.it.row0, k0 = pc.k0, place = pc.tile + runner;
        // positions of the first and of the last row: the tokens that they see
        const int pos0 = p.prefix ? pc.it.len - 1 : pc.it.len - pc.it.rows;
        const int p0 = p.prefix ? pos0 : pos0 + flat0 / heads;
        auto position = [&](int kt) {
            const int row = kt * 4 + i4;
            return row < rows ? (p.prefix ? pos0 : pos0 + (flat0 + row) / heads) : -1;
        };
        // ---- the queries as the instruction's columns: column r of tile vt is row 8 vt + r / 2, and 4
        // more where r is odd
        uint4 qf[VT][LN::kQueryShared ? 1 : U];
        float qsum[KT][NG];  // sum of a row's values over a group, in the products' unit
        float unit[KT];      // the factor that makes scores (times log2 e) of the sums
        float acc[VT][MT][4];
        float pb[KT][NG], l[KT], m[KT], mu[KT];
        int v_exp = 20;        // the values' scales are below 2^(v_exp - 126) ...
        uint32_t v_bound = 0;  // ... whose bf16 bits these are
        float v_up = 0.f;      // 2^7 over that
        if (LN::kQueryShared) __syncwarp();  // (the last piece's have been used)
        if (LN::kQueryAhead) {
            if (!warp_wait_sleep(&ring.query, (uint32_t)queried & 1u, p.wait_budget)) return lone_stop(ring, u, true, queried);
            ++queried;
        }
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
            const int rr = vt * 8 + (r >> 1) + (r & 1) * 4;
            const bool in = rr < rows && (KT > 1 || !(r & 1));
            const int flat = flat0 + (in ? rr : 0), j = flat / heads;
            const __nv_bfloat16* src = p.q + (long long)(row0 + j) * p.q_row_stride +
                                       (long long)(head0 + flat - j * heads) * p.q_head_stride + 8 * i4;
            uint4 raw[U];
            uint32_t big = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw[u] = make_uint4(0u, 0u, 0u, 0u);
                if (in)
                    raw[u] = LN::kQueryAhead
                                 ? *reinterpret_cast<const uint4*>(raw_rows + rr * (D * 2) + (8 * i4 + 32 * u) * 2)
                                 : *(reinterpret_cast<const uint4*>(src + 32 * u));
                big = max_u16x2(big, max_u16x2(raw[u].x & 0x7FFF7FFFu, raw[u].y & 0x7FFF7FFFu));
                big = max_u16x2(big, max_u16x2(raw[u].z & 0x7FFF7FFFu, raw[u].w & 0x7FFF7FFFu));
            }
            big = max(big & 0xFFFFu, big >> 16);
            big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
            big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
            const int ex = max((int)(big >> 7), 16);  // biased exponent of the largest
            const float up = pow2_of(267 - ex);       // 2^(140 - ex)
            float sums[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) sums[g] = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * e] = __uint_as_float(w[e] << 16) * up;
                    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u) * up;
                    sums[u * 32 / G] += x[2 * e] + x[2 * e + 1];
                }
                // as a code word's nibbles pair up; the odd ones are 16 times as large
                const uint4 f = make_uint4(
                    cvt_f16x2(x[0], x[4]), cvt_f16x2(x[1] * 0.0625f, x[5] * 0.0625f),
                    cvt_f16x2(x[2], x[6]), cvt_f16x2(x[3] * 0.0625f, x[7] * 0.0625f));
                if (LN::kQueryShared) queries[(vt * U + u) * 32 + lane] = f;
                else qf[vt][LN::kQueryShared ? 0 : u] = f;
            }
#pragma unroll
            for (int c = 0; c < (KT == 1 ? 1 : 2); ++c) {
                const int kt = 2 * vt + c, from = 8 * i4 + 4 * c;  // a lane of column 2 i4 + c
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float x = sums[g];
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
                    qsum[kt][g] = __shfl_sync(0xFFFFFFFFu, x, from) * 0x1p-24f;
                    pb[kt][g] = 0.f;
                }
                const int ec = __shfl_sync(0xFFFFFFFFu, ex, from);
                unit[kt] = fmaxf(p.scale_log2 * 0x1p24f * pow2_of(ec - 13), 0x1p-126f);
                l[kt] = 0.f;
                m[kt] = -INFINITY;
                mu[kt] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[vt][t][c] = 0.f;
        }
        __syncwarp();  // the queries have been read
        bool asked = false;  // the next piece's
        if (LN::kQueryAhead) {
            const SharedPiece& q = ring.pieces[(n_piece + 1) % kLonePieces];
            asked = q.count;
            lone_queries<D>(p, ring, q, smem_u32(raw_rows));
        }

        for (int n = 0; n < count; ++n, ++u) {
            const int t0 = (k0 + n) * TILE, slot = u % SLOTS;
            if (n % (kLoneChain / TILE) == kLoneChain / TILE - 1) {
                // ---- the mean of a row's sums over a group goes to where its biases are summed, an eighth
                // in each of the column's lanes
                const float down = pow2_of(max(v_exp - 6, 1));
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const int vt = kt / 2, c = kt & 1;
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        float x = 0.f;
#pragma unroll
                        for (int t = g * G / 16; t < (g + 1) * G / 16; ++t)
                            x += fmaf(acc[vt][t][2 + c], 0.0625f, acc[vt][t][c]);
                        x = sum_rows(x) * (1.f / G);
#pragma unroll
                        for (int t = g * G / 16; t < (g + 1) * G / 16; ++t) {
                            acc[vt][t][c] -= x;
                            acc[vt][t][2 + c] = fmaf(x, -16.f, acc[vt][t][2 + c]);
                        }
                        pb[kt][g] = fmaf(x * down, 0x1p21f, pb[kt][g]);
                    }
                }
            }
            if (!warp_wait_sleep(&ring.full[slot], (uint32_t)(u / SLOTS) & 1u, p.wait_budget)) {
                return lone_stop(ring, u, asked, queried);
            }
            const uint8_t* at = data + slot * kStage;
            const int there = ring.there[slot];
            // 16 tokens at a time, in a loop that the instruction caches hold: the warps of an SM are all
            // at different places of it
#pragma unroll 1
            for (int b = 0; b < SUB; ++b) {
            // ---- sums q . c, tokens r and r + 8 in a lane
            float sc[KT][2];
            {
                uint32_t w0[U], w1[U], pr0[NG], pr1[NG];
                load_words<U>(at + words_0 + b * words_1, w0);
                load_words<U>(at + words_0 + b * words_1 + 4 * D, w1);
                load_pairs<NG>(at + pairs_0 + b * pairs_1, pr0);
                load_pairs<NG>(at + pairs_0 + b * pairs_1 + 8 * NG * 4, pr1);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float a[VT][4];
#pragma unroll
                    for (int u = g * G / 32; u < (g + 1) * G / 32; ++u) {
                        uint32_t x[4], y[4];
                        codes_of(w0[u], x);
                        codes_of(w1[u], y);
#pragma unroll
                        for (int vt = 0; vt < VT; ++vt) {
                            const uint4 f = LN::kQueryShared ? queries[(vt * U + u) * 32 + lane]
                                                             : qf[vt][LN::kQueryShared ? 0 : u];
                            if (u == g * G / 32)
                                mma_f16_first(a[vt], x[0], y[0], x[1], y[1], f.x, f.y);
                            else
                                mma_f16(a[vt], x[0], y[0], x[1], y[1], f.x, f.y);
                            mma_f16(a[vt], x[2], y[2], x[3], y[3], f.z, f.w);
                        }
                    }
                    const float s0 = __uint_as_float(pr0[g] << 16);
                    const float s1 = __uint_as_float(pr1[g] << 16);
                    const float b0 = __uint_as_float(pr0[g] & 0xFFFF0000u);
                    const float b1 = __uint_as_float(pr1[g] & 0xFFFF0000u);
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        const float qs = qsum[kt][g];
                        const float z0 = g ? fmaf(b0, qs, sc[kt][0]) : b0 * qs;
                        const float z1 = g ? fmaf(b1, qs, sc[kt][1]) : b1 * qs;
                        sc[kt][0] = fmaf(s0, a[kt / 2][kt & 1], z0);
                        sc[kt][1] = fmaf(s1, a[kt / 2][2 + (kt & 1)], z1);
                    }
                }
            }
            // ---- the values' pairs; what no row sees may hold anything
            uint32_t vp0[NG], vp1[NG];
            load_pairs<NG>(at + v_off + pairs_0 + b * pairs_1, vp0);
            load_pairs<NG>(at + v_off + pairs_0 + b * pairs_1 + 8 * NG * 4, vp1);
            if (there != (1 << SUB) - 1 || t0 + TILE - 1 > p0) {
                // some row does not see some token
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = t0 + 16 * b + r + 8 * i;
                        const bool is = ((there >> b) & 1) && t <= p1;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            if (!is && i == 0) vp0[g] = 0u;
                            if (!is && i == 1) vp1[g] = 0u;
                        }
#pragma unroll
                        for (int kt = 0; kt < KT; ++kt)
                            if (!(is && t <= position(kt))) sc[kt][i] = -INFINITY;
                    }
            }
            // ---- running maximum: moved only when a score is far above it, and the
            // values' power of two, when a scale is above it
            uint32_t scales = 0;  // the low half word
#pragma unroll
                for (int g = 0; g < NG; ++g) scales = max_u16x2(scales, max_u16x2(vp0[g], vp1[g]));
            scales &= 0xFFFFu;
            float top[KT];
            bool over = scales > v_bound;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                top[kt] = fmaxf(sc[kt][0] * unit[kt], sc[kt][1] * unit[kt]);
                over |= top[kt] > m[kt] + 8.f;
            }
            if (__any_sync(0xFFFFFFFFu, over)) {
                uint32_t big = __reduce_max_sync(0xFFFFFFFFu, scales);
                if (big > 0x7FFFu) {
                    // a scale with its sign set, which comes here every time: only the sizes count
                    uint32_t size = 0;
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            size = max(size, max(vp0[g] & 0x7FFFu, vp1[g] & 0x7FFFu));
                    big = __reduce_max_sync(0xFFFFFFFFu, size);
                }
                const int e_new = max(v_exp, min((int)(big >> 7), 254));
                const float fv = pow2_of(max(v_exp - e_new + 127, 1));
                v_exp = e_new;
                v_bound = ((uint32_t)e_new << 7) | 127u;
                v_up = pow2_of(260 - e_new);  // 2^(133 - e_new)
                float f[KT];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    float x = top[kt];
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                    const float mn = fmaxf(m[kt], x);
                    mu[kt] = mn == -INFINITY ? 0.f : mn;
                    f[kt] = exp2_approx(m[kt] - mu[kt]);
                    m[kt] = mn;
                    l[kt] *= f[kt];
#pragma unroll
                    for (int g = 0; g < NG; ++g) pb[kt][g] *= f[kt];
                    f[kt] *= fv;
                }
#pragma unroll
                for (int vt = 0; vt < VT; ++vt)
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[vt][t][c] *= f[KT == 1 ? 0 : 2 * vt + (c & 1)];
            }
            // ---- weighted sum of the values
            {
                uint32_t w0[U], w1[U];
                load_words<U>(at + v_off + words_0 + b * words_1, w0);
                load_words<U>(at + v_off + words_0 + b * words_1 + 4 * D, w1);
                float e0[KT], e1[KT], h0[KT], h1[KT];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    e0[kt] = exp2_approx(fmaf(sc[kt][0], unit[kt], -mu[kt]));
                    e1[kt] = exp2_approx(fmaf(sc[kt][1], unit[kt], -mu[kt]));
                    l[kt] += e0[kt] + e1[kt];
                    h0[kt] = e0[kt] * v_up;
                    h1[kt] = e1[kt] * v_up;
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float s0 = __uint_as_float(vp0[g] << 16);
                    const float s1 = __uint_as_float(vp1[g] << 16);
                    const float b0 = __uint_as_float(vp0[g] & 0xFFFF0000u);
                    const float b1 = __uint_as_float(vp1[g] & 0xFFFF0000u);
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
                        pb[kt][g] = fmaf(b0, e0[kt], fmaf(b1, e1[kt], pb[kt][g]));
                    uint32_t f0[VT], f1[VT];
#pragma unroll
                    for (int vt = 0; vt < VT; ++vt) {
                        constexpr int other = KT == 1 ? 0 : 1;
                        f0[vt] = transpose_8x8(
                            cvt_f16x2(s0 * h0[2 * vt], other ? s0 * h0[2 * vt + other] : 0.f));
                        f1[vt] = transpose_8x8(
                            cvt_f16x2(s1 * h1[2 * vt], other ? s1 * h1[2 * vt + other] : 0.f));
                    }
#pragma unroll
                    for (int u = g * G / 32; u < (g + 1) * G / 32; ++u) {
                        uint32_t x[4], y[4];
                        codes_of(w0[u], x);
                        codes_of(w1[u], y);
#pragma unroll
                        for (int vt = 0; vt < VT; ++vt) {
                            mma_f16(acc[vt][2 * u], x[0], x[1], y[0], y[1], f0[vt], f1[vt]);
                            mma_f16(acc[vt][2 * u + 1], x[2], x[3], y[2], y[3], f0[vt], f1[vt]);
                        }
                    }
                }
            }
            }
            __syncwarp();  // the slot has been read
            lone_copy<D, G, TILE>(p, ring, slots, pages, later);
        }

        // ---- the piece's result
        const float v_down = pow2_of(max(v_exp - 6, 1));  // 1 / v_up
        float* to = p.partial + (long long)place * (LN::kRows * (D + 2));
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            const int row = kt * 4 + i4;
            const float x = sum_rows(l[kt]);
            if (r == 0 && row < rows) *reinterpret_cast<float2*>(to + 2 * row) = make_float2(m[kt], x);
#pragma unroll
            for (int g = 0; g < NG; ++g) pb[kt][g] = sum_rows(pb[kt][g]);
            if (row < rows) {
                float* o = to + 2 * LN::kRows + row * D + r;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        o[t * 16 + c * 8] = fmaf(acc[kt / 2][t][2 * c + (kt & 1)] * (c ? 0x1p20f : 0x1p24f),
                                                 v_down, pb[kt][t * 16 / G]);
            }
        }
    }
}

// Both parts (KT1, KT2: row tiles of the groups' and of the sequences' rows), or the sequences'
// beside the tensor cores' kernel.
template <int D, int G, int KT1, int KT2>
__global__ void __launch_bounds__(kLoneThreads, (LoneBoth<D, G, KT1, KT2>::kCtas))
    kv_lone_kernel(const __grid_constant__ KvSharedParams a, const __grid_constant__ KvSharedParams b) {
    using LB = LoneBoth<D, G, KT1, KT2>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Sums<kLoneThreads> prefix_sums, own_sums;
    __shared__ LoneRing<LB::kSlots> rings[kLoneWarps];
    if (threadIdx.x < kLoneWarps) {
        for (int i = 0; i < LB::kSlots; ++i) mbar_init(&rings[threadIdx.x].full[i], 1);
        mbar_init(&rings[threadIdx.x].query, 1);
        mbar_init_fence();
    }
    // The tensor cores' kernel has waited for what comes before the call, and is not waited for here: what is read
    // comes behind its word.
    if (!a.on_tensor_cores) {
        pdl_wait();
        pdl_launch_dependents();
    }
    // Runners of the two parts.  Beside the other kernel they are the first CTAs, which are on the SMs
    // that it leaves; else consecutive ones are on different SMs.
    const int all = gridDim.x * kLoneWarps;
    int first = 0, second = all;
    if (a.on_tensor_cores) {
        // the SMs that the other kernel leaves; it needs them all for itself if there is nothing else
        const int sms = said_sms(a);
        pdl_launch_dependents();
        if (sms < a.sms) second = (int)((long long)all * (a.sms - sms) / a.sms);
        if ((int)blockIdx.x * kLoneWarps >= second) {
            // (a CTA that begins when the other kernel ends, with 3 us of lists before it would find nothing to do)
            pdl_wait();
            return;
        }
        heard();
    }
    if (!a.on_tensor_cores) sum_items(a, prefix_sums);
    else prefix_sums.units[threadIdx.x] = prefix_sums.planes[threadIdx.x] = 0;
    sum_items(b, own_sums);
    __syncthreads();
    const int warp = threadIdx.x / 32;
    Scan prefix, own;
    scan_sums(prefix_sums, own_sums, prefix, own);
    const long long prefix_cost = all_units(a, prefix) * a.unit_cost, own_cost = all_units(b, own) * b.unit_cost;
    const int runner = a.on_tensor_cores ? blockIdx.x * kLoneWarps + warp : warp * gridDim.x + blockIdx.x;
    if (!a.on_tensor_cores) {
        first = share_of(prefix_cost, own_cost, all);
        second = all - first;
    }
    const long long own_run = run_length(b, all_units(b, own), second);
    const long long prefix_run = a.on_tensor_cores ? 0 : run_length(a, all_units(a, prefix), first);
    if (blockIdx.x == (a.on_tensor_cores ? (second - 1) / kLoneWarps : gridDim.x - 1)) {
        write_before(b, own_sums, own, own_run);
        if (!a.on_tensor_cores) write_before(a, prefix_sums, prefix, prefix_run);
    }
    uint8_t* data = smem + warp * LB::kWarpBytes;
    uint4* queries = reinterpret_cast<uint4*>(data + LB::kSlots * LB::kStageBytes);
    auto& ring = rings[warp];
    // (all lanes write the same)
    ring.n = 0;
    bool ok = true;
    if (!a.on_tensor_cores && runner < first) {
        SharedWalk walk;
        walk.start(a, prefix_sums, prefix, prefix_run, runner);
        ring.walk = walk;
        __syncwarp();
        if (walk.left > 0) ok = lone_run<D, G, KT1>(a, runner, ring, data, queries);
    } else if (runner - first < second) {
        SharedWalk walk;
        walk.start(b, own_sums, own, own_run, runner - first);
        ring.walk = walk;
        __syncwarp();
        if (walk.left > 0) ok = lone_run<D, G, KT2>(b, runner - first, ring, data, queries);
    }
    if (!ok) flag_status(b.status, MXQ_DEV_TIMEOUT);
    // The tensor cores' kernel may still run; the joining kernel waits for this one only.
    if (a.on_tensor_cores) pdl_wait();
}

}  // namespace
}  // namespace mxq
