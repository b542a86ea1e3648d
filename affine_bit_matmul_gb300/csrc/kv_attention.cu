// Attention of a few query rows over a paged 4-bit key/value cache.
//
// For a row at position p and the keys t it sees (t <= p; with a window also
// t > p - window or t < sinks):
//   S_t = scale * q . k^_t,  P = softmax(S),  out = sum_t P_t v^_t
//   k^_td = s_tg q_td + b_tg, the same for v, g the group of value d
// The codes never become rounded values.  Per group,
//   q . k^_t = sum_g s_tg (q_g . c_t) + b_tg sum(q_g)
//   sum_t P_t v^_td = sum_t (P_t s_tg) c_td + sum_t P_t b_tg
// so the matrix instructions (m16n8k16, f16 operands, fp32 sums) multiply codes,
// and scales and biases are applied in fp32 to a few numbers per token.  A code
// in the lowest 4 bits of an f16 number is 2^-24 times its value, in the next 4
// bits 2^-20 times it (both are subnormals, which the instructions take as they
// are): a code word's 8 nibbles become 4 operand registers by 4 masks and one
// shift, with no offset to take out again.
//   Keys: the other operand is a query row, scaled by a power of two so that its
// largest value is 2^13 .. 2^14; f16 then holds its bf16 values exactly down to
// 2^-24 of the largest.
//   Values: P_t s_tg, scaled by a power of two that keeps it below 2^15 for the
// scales met so far, rounded to f16: 11 bits down to 2^-29 of the largest, which
// is the only rounding before the output's.
// Tokens are the instruction's rows (K) or depth (V), query rows the columns: row
// i in column 2 i, row 4 + i in column 2 i + 1, so up to 4 rows leave half of a
// lane's numbers unused and not computed.
//
// Work split: a unit is (row tile, tile of tokens that it sees); the units of a
// call, in order, are cut into equal runs, one per CTA, whatever the lengths
// of the sequences.  A run that begins or ends inside a row tile leaves its
// (max, sum, weighted sum) in the workspace and a second kernel joins them in
// order, so the result does not depend on timing.  Short calls whose row tiles can have
// a CTA each are not cut.
//
// A CTA's warps take the units of its run in turn, each with a softmax state of
// its own; they are joined at the end of a row tile.  One more warp fills the
// ring of tiles, lane i slot i, by copying whole page blocks (K codes, K pairs,
// V codes and V pairs of a head are contiguous: one bulk copy per page), and
// works out what a tile's tokens are to the rows.  The running maximum is only
// moved when a score exceeds it by 2^8, so most tiles have no reductions across
// lanes at all.
// Bound by HBM for long contexts, 2 (D / 2 + 4 D / G) bytes per token and head: 8
// sequences of 65536 to 131072 tokens, 5 query heads to a key head of 128 values,
// 164 us, 5.8 TB/s; 64 of 1024 to 8192 tokens, 4 query heads, 71 us, 4.8 TB/s with the
// ends of the row tiles.  From 16 rows on by the instructions around the products: 32
// sequences of 8192 tokens 117 us, 2.6 TB/s.  One sequence of 573 tokens takes 7.6 us: a
// chain of loads (length, pages, tiles) and two rounds of tiles in each warp.
//   The matrix instructions' fp32 sums round towards zero.  Codes and weights are not
// negative, so their products add up to sums of which the biases then take most away
// again, and what a long chain of them loses is a good part of a small result: of 40 sequences of
// 131072 tokens of values around zero 1.2e-2 of the norm for 4 rows, 5.9e-2 for 16, where the
// rounding to bf16 is 1.7e-3.  The values of a group share most of that sum.  So every 512
// tokens a warp moves a group's mean from the sums to the biases': what stays is no larger
// than the result, and a chain loses parts of 512 tokens' products only.  The same
// calls are off by 1.8e-3 in all, the rest beside the rounding being the weights' 11 bits; 256 tokens
// gain 1e-5 more.  Time: none at 4 rows, 2% at 16.
#include <climits>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_attn_common.cuh"
#include "kv_shared.cuh"

namespace mxq {
namespace {

// What a sequence of a call over shared prefixes sees when its prefix is taken for it alone: the prefix's
// tiles (head_tiles), then those of its own tokens.
template <int TILE>
__device__ __forceinline__ Span span_of(const KvTwoParams& p, int s, int plane) {
    Span r = span_of<TILE>(static_cast<const KvAttnParams&>(p), s, plane);
    const int own = r.p0 + r.toks > 0 ? (r.p0 + r.toks - 1) / TILE + 1 : 0;
    r.head_tiles = r.tail = 0;
    const int g = group_with(p, s);
    if (g < 0) {
        r.tiles = r.toks > 0 ? max(1, own) : 0;
        return r;
    }
    const Item pre = item_of(p, g);
    if (pre.bad) r.bad = 1;
    if (r.toks > 0 && (r.row0 < pre.row0 || r.row0 + r.toks > pre.row0 + pre.rows)) {
        // the group is left out, or the sequence's rows are not its
        r.bad = 1;
        r.toks = 0;
    }
    r.head_tiles = (pre.len + TILE - 1) / TILE;
    r.tiles = r.toks > 0 ? max(1, r.head_tiles + own) : 0;
    return r;
}

// Tokens whose value products a warp adds before it takes out what the values of a group
// have in common.
constexpr int kChainTokens = 512;

// What the end of a row tile costs a CTA (joining its warps, the next queries), in
// tokens: the runs are cut equal with so many tokens that take no work after each
// row tile.  64 sequences of 1024 to 8192 tokens take 88 us without it (the CTAs of
// short ones 81 us, those of long ones 52), 78 with 128 tokens, 76 with 256, 74 with
// 512.
constexpr int kEndTokens = 512;

// A call is left uncut only if none of its row tiles can have more tiles than this: however
// ragged the batch, the others then do not wait long for the block of the longest.  38
// sequences, 8 key heads of 128 values, one as long as possible and the others of 64 tokens,
// uncut and cut: 4 rows 12.2 and 14.5 us for 32 tiles, 19.6 and 15.3 for 64, 242 and 27 for
// 1024; 16 rows 17.1 and 19.2 for 32, 25.4 and 20.5 for 64.
constexpr int kUncutTiles = 40;

// Sizes of a kernel for row tiles of 4 KT rows: tokens of a tile, compute warps,
// CTAs per SM, tiles in the ring.  Warps: as many as their registers allow, 16 an SM
// with 128 registers each (D <= 128, up to 8 rows), 12 with 168, 8 with 255.  16 rows:
// tiles of 32 tokens, which take 31 us for 32 sequences with a window of 1024 and 115
// for 32 of 8192 tokens (64 tokens: 40 and 109).
template <int D, int G, int KT>
struct Shape {
    static constexpr int kRows = 4 * KT;
    static constexpr int kTile = D == 256 || KT == 4 ? 32 : 64;
    static constexpr int kCtas = 2;
    static constexpr int kStageBytes = kv_block_bytes(D, G, kTile);
    // the queries lie in shared memory where they would take 32 registers or more
    static constexpr int kColumns = (KT + 1) / 2;  // tiles of 8 columns
    static constexpr bool kQueryShared = D * kColumns >= 256;
    static constexpr int kQueryBytes = kQueryShared ? kColumns * D * 16 : 0;
    static constexpr int kWarps = KT == 4 ? 3 : D == 256 ? 5 : 7;
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int kChunk = KT == 1 && D > 64 ? 128 : 64;  // values joined at a time
    static constexpr int kRowPad = kChunk + 8;
    static constexpr int kJoinBytes = kWarps * kRows * kRowPad * 4;
    static constexpr int kStatBytes = kWarps * kRows * 8;
    static constexpr int kRoom = 107 * 1024 - kJoinBytes - kStatBytes - kQueryBytes;
    static constexpr int kSlots = kRoom / kStageBytes < 24 ? kRoom / kStageBytes : 24;
    static constexpr int kRingBytes = kSlots * kStageBytes;
    static constexpr int kSmem = kRingBytes + kJoinBytes + kStatBytes + kQueryBytes;
    static constexpr int kPartialFloats = kRows * (D + 2);
};

// A run's piece of one row tile, for the warps of a CTA (shared memory).
struct Piece {
    int row0, toks, p0;       // its rows of q, tokens, position of the first
    int head0, heads;         // its query heads
    int s, h;                 // sequence and key/value head
    int head_tiles, tail;     // which tiles its units are (Span)
    int k0, seq0, end;        // first unit; numbers of its units in the run
    int flags;                // kBegins, kEnds
    int last;                 // no piece: the run is over
    int group, prefix;        // shared prefixes: the sequence's group (-1: none), its tokens
};
// Pieces of the run that are known ahead: the copying warp looks up to two rounds of
// its ring (24 tiles at most) ahead of the unit that is being worked on.
constexpr int kPieces = 64;

// A row tile's units: its tiles of tokens, and what its end costs.
template <int TILE>
__device__ __forceinline__ int units_of(const Span& sp) {
    return sp.tiles ? sp.tiles + kEndTokens / TILE : 0;
}

// One thread: lists the pieces of the CTA's run, the first kPieces at once and
// one more whenever the warps are done with one; then one marked `last`.
template <int TILE>
struct Walk {  // (no constructors: it lies in shared memory)
    int s, h, part, k, seq, left;
    Span sp;

    // the run's first unit is unit `at` of sequence s (of all its heads)
    template <class P>
    __device__ void start(const P& p, int s_, long long at, int units) {
        s = s_;
        sp = span_of<TILE>(p, s, 0);
        const long long vheads = (long long)p.Hkv * p.head_parts;
        while (at >= units_of<TILE>(sp) * vheads) {
            at -= units_of<TILE>(sp) * vheads;
            sp = span_of<TILE>(p, ++s, 0);
        }
        const unsigned first = (unsigned)at;  // below 2^31 units a sequence
        const int vh = (int)(first / (unsigned)units_of<TILE>(sp));
        k = (int)(first % (unsigned)units_of<TILE>(sp));
        h = vh / p.head_parts;
        part = vh % p.head_parts;
        seq = 0;
        left = units;
    }
    // the run is one row tile
    template <class P>
    __device__ void whole(const P& p, int s_, int vh, const Span& span) {
        s = s_;
        sp = span;
        h = vh / p.head_parts;
        part = vh % p.head_parts;
        k = seq = 0;
        left = sp.tiles;
    }
    template <class P>
    __device__ bool next(const P& p, Piece* out, Seg* seg) {
        bool found = false;
        while (left && !found) {
            while (sp.tiles == 0) sp = span_of<TILE>(p, ++s, 0);
            const int units = units_of<TILE>(sp), n = min(left, units - k);
            const int tiles = min(k + n, sp.tiles) - k;  // the others are the row tile's end
            if (tiles > 0) {
                const int rep = p.Hq / p.Hkv;
                Piece q;
                q.row0 = sp.row0;
                q.toks = sp.toks;
                q.p0 = sp.p0;
                q.head0 = h * rep + part * p.part_heads;
                q.heads = min(p.part_heads, rep - part * p.part_heads);
                q.s = s;
                q.h = h;
                q.head_tiles = sp.head_tiles;
                q.tail = sp.tail;
                q.k0 = k;
                q.seq0 = seq;
                q.end = seq + tiles;
                q.flags = (k == 0 ? kBegins : 0) | (k + tiles == sp.tiles ? kEnds : 0);
                q.last = 0;
                if constexpr (P::kTwo) {
                    q.group = group_with(p, s);
                    q.prefix = q.group < 0 ? 0 : item_of(p, q.group).len;
                }
                *out = q;
                if (q.flags != (kBegins | kEnds)) {
                    Seg g;
                    g.row0 = q.row0;
                    g.toks = q.toks;
                    g.head0 = q.head0;
                    g.heads = q.heads;
                    g.flags = q.flags;
                    seg[(q.flags & kBegins) ? 1 : 0] = g;
                }
                seq += tiles;
                found = true;
            }
            left -= n;
            k += n;
            if (k == units && left) {
                k = 0;
                if (++part == p.head_parts) {
                    part = 0;
                    if (++h == p.Hkv) {
                        h = 0;
                        sp = span_of<TILE>(p, ++s, 0);
                    }
                }
            }
        }
        if (!found) {
            out->end = 1 << 30;
            out->last = 1;  // no piece: the run is over
        }
        return found;
    }
};

// What a tile in the ring is to the compute warps: the number of its unit, its
// first token, and in `state` bit i: its 16 tokens from 16 i on exist; kAll: every
// row sees all of them.  The warps may be a whole round of the ring apart, and
// the parity of a phase alone does not tell a round from the one two before it:
// a warp waits for the number first.
struct Tile {
    int unit, t0, state;
};
constexpr int kAll = 256;
constexpr int kPrefix = 512;  // its tokens are a shared prefix's

// Waits, within the budget, until a slot is given to unit n (whole warp).
__device__ __forceinline__ bool unit_comes(const int* unit, int n, long long budget) {
    const volatile int* u = unit;
    bool ok = true;
    if (*u != n) {
        const long long since = clock64();
        while (*u != n && ok) {
            __nanosleep(20);
            ok = clock64() - since <= budget;
        }
    }
    return __all_sync(0xFFFFFFFFu, ok);
}

// The copying warp, lane i filling slot i: units i, i + SLOTS, ...  Pages of at
// most a tile are copied whole, of longer ones the four regions of the tile's
// part.
template <int D, int G, int TILE, int SLOTS, class P>
__device__ void copy_tiles(const P& p, const Piece* pieces, int lane,
                           uint32_t ring, Tile* tiles, uint64_t* full, uint64_t* empty) {
    constexpr int kMost = TILE / 16;
    constexpr uint32_t cb = kv_code_bytes(D, TILE), pb = kv_pair_bytes(D, G, TILE);
    const int size = min(p.page_size, TILE), count = TILE / size;
    const uint32_t block = kv_block_bytes(D, G, size);
    const uint32_t slot = ring + lane * kv_block_bytes(D, G, TILE);
    int n = lane, end = 0, piece = -1;
    uint32_t parity = 1;  // the first wait passes at once
    bool work = lane < SLOTS;
    int t0 = 0, id[kMost];
    bool of_prefix = false;
    Piece q;

    auto look = [&]() {  // the pages of unit n, if there is one
        if (n >= end) {
            do ++piece;
            while (n >= pieces[piece % kPieces].end);
            q = pieces[piece % kPieces];
            end = q.end;
            if (q.last) {
                work = false;
                return;
            }
        }
        const int k = q.k0 + n - q.seq0;
        t0 = (k < q.head_tiles ? k : q.tail + k - q.head_tiles) * TILE;
        const int32_t* row = p.table + (long long)q.s * p.max_pages;
        if constexpr (P::kTwo) {
            of_prefix = k < q.head_tiles;
            if (of_prefix) row = p.prefix_table + (long long)q.group * p.max_prefix_pages;
        }
        const int end_token = P::kTwo && of_prefix ? q.prefix : q.p0 + q.toks;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int t = t0 + i * size;
            id[i] = -2;  // not needed
            if (i < count && t < end_token) id[i] = __ldg(row + (t >> p.page_shift));
        }
    };
    if (work) look();
    long long since = clock64();
    while (__any_sync(0xFFFFFFFFu, work)) {
        const bool ready = work && mbar_test_wait(&empty[lane], parity);
        if (ready) {
            const int p1 = q.p0 + q.toks - 1;
            uint32_t bytes = 0;
            int state = 0;
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                if ((unsigned)id[i] < (unsigned)p.n_pages) {
                    state |= ((1 << (size / 16)) - 1) << (i * (size / 16));
                    bytes += block;
                } else if (id[i] != -2) {
                    // a page that some row sees has to exist
                    const int t = t0 + i * size, te = min(t + size - 1, p1);
                    if (!p.window || te > q.p0 - p.window || t < p.sinks)
                        flag_status(p.status, MXQ_DEV_BAD_PAGE);
                }
            }
            if (state == (1 << kMost) - 1 && t0 + TILE - 1 <= (P::kTwo && of_prefix ? q.prefix - 1 : q.p0) &&
                (!p.window || t0 > p1 - p.window || t0 + TILE <= p.sinks))
                state |= kAll;
            if (P::kTwo && of_prefix) state |= kPrefix;
            tiles[lane].t0 = t0;
            tiles[lane].state = state;
            *const_cast<volatile int*>(&tiles[lane].unit) = n;
            mbar_expect_tx(&full[lane], bytes);
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                if ((unsigned)id[i] >= (unsigned)p.n_pages) continue;
                const uint8_t* src = p.pages + ((long long)id[i] * p.Hkv + q.h) *
                                                   kv_block_bytes(D, G, p.page_size);
                if (p.page_size <= TILE) {
                    bulk_copy(slot + i * block, src, block, &full[lane]);
                } else {
                    const int skip = t0 & (p.page_size - 1);
                    const uint8_t* codes = src + kv_code_bytes(D, skip);
                    const uint8_t* pairs =
                        src + kv_code_bytes(D, p.page_size) + kv_pair_bytes(D, G, skip);
                    const int v = kv_block_bytes(D, G, p.page_size) / 2;
                    bulk_copy(slot, codes, cb, &full[lane]);
                    bulk_copy(slot + cb, pairs, pb, &full[lane]);
                    bulk_copy(slot + cb + pb, codes + v, cb, &full[lane]);
                    bulk_copy(slot + 2 * cb + pb, pairs + v, pb, &full[lane]);
                }
            }
            parity ^= 1u;
            n += SLOTS;
            look();
        }
        if (__any_sync(0xFFFFFFFFu, ready)) {
            since = clock64();
        } else {
            if (clock64() - since > p.wait_budget) {
                if (work) flag_status(p.status, MXQ_DEV_TIMEOUT);
                break;
            }
            __nanosleep(100);
        }
    }
    // no copy may land after the CTA is gone
    if (lane < SLOTS && n > lane) mbar_wait(&full[lane], (uint32_t)((n - lane) / SLOTS - 1) & 1u);
}

template <int D, int G, int KT, class P>
__global__ void __launch_bounds__(Shape<D, G, KT>::kThreads, Shape<D, G, KT>::kCtas)
    kv_attn_kernel(const P p) {
    using SH = Shape<D, G, KT>;
    constexpr int TILE = SH::kTile, SUB = TILE / 16;  // a warp takes 16 tokens at a time
    constexpr int kWarps = SH::kWarps, kThreads = SH::kThreads, kSlots = SH::kSlots;
    constexpr int kChunk = SH::kChunk, kRowPad = SH::kRowPad;
    constexpr int NG = D / G;          // groups
    constexpr int U = D / 32;          // code words of a lane per 8 tokens
    constexpr int MT = D / 16;         // output tiles of 16 values
    constexpr int VT = SH::kColumns;   // tiles of 8 columns
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kSlots], empty[kSlots], joined, freed, queried;
    __shared__ Tile tiles[kSlots];
    __shared__ Piece pieces[kPieces];
    __shared__ Walk<TILE> walk;  // thread 0's
    __shared__ int sums[kThreads];
    // the joining kernel waits for this one's end by itself; what else follows may not
    if (!p.whole) pdl_launch_dependents();
    float* join = reinterpret_cast<float*>(smem + SH::kRingBytes);
    float2* stat = reinterpret_cast<float2*>(smem + SH::kRingBytes + SH::kJoinBytes);
    uint4* queries = reinterpret_cast<uint4*>(smem + SH::kSmem - SH::kQueryBytes);

    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    Seg* seg = reinterpret_cast<Seg*>(p.segs) + (long long)cta * 2;

    if constexpr (P::kTwo) {
        // groups that no sequence is found in are reported too
        if (cta == 0 && p.status)
            for (int g = threadIdx.x; g < p.groups_n; g += kThreads)
                if (item_of(p, g).bad) flag_status(p.status, MXQ_DEV_BAD_SEQUENCE);
    }
    // every CTA finds its own run: the tiles of all sequences, then its share (or its
    // row tile)
    const int per = (p.S + kThreads - 1) / kThreads;
    if (!p.whole) {
        int sum = 0;
        for (int i = 0; i < per; ++i) {
            const int s = threadIdx.x * per + i;
            if (s >= p.S) break;
            const Span sp = span_of<TILE>(p, s, 0);
            sum += units_of<TILE>(sp);
            if (sp.bad && blockIdx.x == 0) flag_status(p.status, MXQ_DEV_BAD_SEQUENCE);
        }
        sums[threadIdx.x] = sum;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            tiles[i].unit = -1;
        }
        mbar_init(&joined, kWarps);
        mbar_init(&freed, kWarps);
        mbar_init(&queried, kWarps);
        mbar_init_fence();
    }
    __syncthreads();
    if (p.whole) {
        if (threadIdx.x == 0) {
            const int vheads = p.Hkv * p.head_parts, s = cta / vheads, vh = cta % vheads;
            const Span sp = span_of<TILE>(p, s, 0);
            if (sp.bad && vh == 0) flag_status(p.status, MXQ_DEV_BAD_SEQUENCE);
            walk.whole(p, s, vh, sp);
            if (walk.next(p, &pieces[0], seg)) walk.next(p, &pieces[1], seg);
        }
    } else {
        // scan of the threads' sums, in every warp
        long long mine = 0;
#pragma unroll
        for (int i = 0; i < kWarps + 1; ++i) mine += sums[lane * (kWarps + 1) + i];
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += x;
        }
        const long long vheads = (long long)p.Hkv * p.head_parts;
        const long long all = __shfl_sync(0xFFFFFFFFu, incl, 31) * vheads;
        const long long runs = all < p.ctas ? all : p.ctas;
        if (threadIdx.x == 0) seg[0].flags = seg[1].flags = -1;
        if (cta >= runs) return;
        // the first `all % runs` runs have one unit more
        const long long each = all <= INT_MAX ? (int)all / (int)runs : all / runs;
        const int more = (int)(all - each * runs);
        const long long u0 = cta * each + min(cta, more);
        const int total = (int)each + (cta < more ? 1 : 0);
        if (warp == 0) {
            const uint32_t here = __ballot_sync(0xFFFFFFFFu, u0 >= (incl - mine) * vheads &&
                                                                 u0 < incl * vheads);
            const int owner = __ffs(here) - 1;
            long long at = u0 - __shfl_sync(0xFFFFFFFFu, incl - mine, owner) * vheads;
            if (lane == 0) {
                int i = owner * (kWarps + 1);  // the thread whose sequences the run starts in
                while (at >= sums[i] * vheads) at -= sums[i++] * vheads;
                walk.start(p, i * per, at, total);
                for (int n = 0; n < kPieces && walk.next(p, &pieces[n], seg); ++n) {
                }
            }
        }
    }
    __syncthreads();
    if (pieces[0].last) return;

    if (warp == kWarps) {
        copy_tiles<D, G, TILE, kSlots>(p, pieces, lane, smem_u32(smem), tiles, full, empty);
        return;
    }

    const int r = lane >> 2, i4 = lane & 3;
    // offsets in a slot of this lane's words and pairs of 16 tokens: a page's
    // block of `piece` tokens after another
    const int piece = p.page_size < TILE ? p.page_size : TILE;
    const int block = kv_block_bytes(D, G, piece), v_off = block / 2;
    const int words_1 = piece >= 32 ? 8 * D : block, pairs_1 = piece >= 32 ? 64 * NG : block;
    const int words_2 = piece >= 64 ? 16 * D : piece == 32 ? block : 2 * block;
    const int pairs_2 = piece >= 64 ? 128 * NG : piece == 32 ? block : 2 * block;
    auto words_at = [&](int b) {
        return lane * (D == 64 ? 8 : 16) + (b & 1) * words_1 + (b >> 1) * words_2;
    };
    auto pairs_at = [&](int b) {
        return kv_code_bytes(D, piece) + r * NG * 4 + (b & 1) * pairs_1 + (b >> 1) * pairs_2;
    };
    int n = warp;  // this warp's units: those whose number in the run is warp modulo kWarps
    auto gave_up = [&](bool ok) {
        if (!ok && lane == 0) flag_status(p.status, MXQ_DEV_TIMEOUT);
        return !ok;
    };

    int joins = 0;
    for (int at_piece = 0; !pieces[at_piece % kPieces].last; ++at_piece) {
        const Piece& sp = pieces[at_piece % kPieces];
        const int heads = sp.heads, rows = sp.toks * heads, head0 = sp.head0;
        const int p0 = sp.p0, p1 = p0 + sp.toks - 1, end = sp.end;
        // Queries as the instruction's columns: column r of tile vt is row 8 vt + r / 2,
        // and 4 more where r is odd.
        uint4 qf[VT][SH::kQueryShared ? 1 : U];
        float qsum[KT][NG];    // sum of a row's values over a group, in the products' unit
        float unit[KT];        // the factor that makes scores (times log2 e) of the sums
        float acc[VT][MT][4];
        float pb[KT][NG], l[KT], m[KT], mu[KT];
        // The rows' positions are held where there are registers for them (32 sequences of 16
        // rows with a window of 1024: 22.7 us, 23.4 without), and else worked out under a mask
        // (8 rows of 128 values in groups of 32: 93 us, 97 held).
        constexpr bool kHeld = KT == 4 && D <= 128;
        // (a row of a shared prefix may have any position)
        constexpr int kNoRow = P::kTwo ? INT_MIN : -1;
        auto position = [&](int kt) {
            const int row = kt * 4 + i4;
            return row < rows ? p0 + row / heads : kNoRow;  // (no row sees as little)
        };
        int held[KT];
#pragma unroll
        for (int kt = 0; kHeld && kt < KT; ++kt) held[kt] = position(kt);
        int v_exp = 20;        // the values' scales are below 2^(v_exp - 126) ...
        uint32_t v_bound = 0;  // ... whose bf16 bits these are
        float v_up = 0.f;      // 2^7 over that
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
            const int rr = vt * 8 + (r >> 1) + (r & 1) * 4;
            const bool in = rr < rows && (KT > 1 || !(r & 1));
            const int j = in ? rr / heads : 0, hh = in ? rr % heads : 0;
            const __nv_bfloat16* src = p.q + (long long)(sp.row0 + j) * p.q_row_stride +
                                       (long long)(head0 + hh) * p.q_head_stride + 8 * i4;
            uint4 raw[U];
            uint32_t big = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw[u] = make_uint4(0u, 0u, 0u, 0u);
                if (in) raw[u] = __ldg(reinterpret_cast<const uint4*>(src + 32 * u));
                big = max_u16x2(big, max_u16x2(raw[u].x & 0x7FFF7FFFu, raw[u].y & 0x7FFF7FFFu));
                big = max_u16x2(big, max_u16x2(raw[u].z & 0x7FFF7FFFu, raw[u].w & 0x7FFF7FFFu));
            }
            big = max(big & 0xFFFFu, big >> 16);
            big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
            big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
            const int ex = max((int)(big >> 7), 16);  // biased exponent of the largest
            const float up = pow2_of(267 - ex);       // 2^(140 - ex)
            float part[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) part[g] = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * e] = __uint_as_float(w[e] << 16) * up;
                    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u) * up;
                    part[u * 32 / G] += x[2 * e] + x[2 * e + 1];
                }
                // as a code word's nibbles pair up; the odd ones are 16 times as large
                const uint4 f = make_uint4(
                    cvt_f16x2(x[0], x[4]), cvt_f16x2(x[1] * 0.0625f, x[5] * 0.0625f),
                    cvt_f16x2(x[2], x[6]), cvt_f16x2(x[3] * 0.0625f, x[7] * 0.0625f));
                if (SH::kQueryShared) {
                    if (u % kWarps == warp) queries[(vt * U + u) * 32 + lane] = f;
                } else {
                    qf[vt][SH::kQueryShared ? 0 : u] = f;
                }
            }
#pragma unroll
            for (int c = 0; c < (KT == 1 ? 1 : 2); ++c) {
                const int kt = 2 * vt + c, from = 8 * i4 + 4 * c;  // a lane of column 2 i4 + c
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float x = part[g];
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
        if (SH::kQueryShared) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&queried);
            if (gave_up(warp_wait(&queried, (uint32_t)at_piece & 1u, p.wait_budget))) return;
        }

        for (; n < end; n += kWarps) {
            if (n / kWarps % (kChainTokens / TILE) == kChainTokens / TILE - 1) {
                // ---- the mean of a row's sums over a group goes to where its biases are summed,
                // an eighth in each of the column's lanes
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
            const int slot = n % kSlots;
            if (gave_up(unit_comes(&tiles[slot].unit, n, p.wait_budget) &&
                        warp_wait_sleep(&full[slot], (uint32_t)(n / kSlots) & 1u, p.wait_budget)))
                return;
            uint8_t* at = smem + slot * SH::kStageBytes;
            const Tile tile = tiles[slot];
            // ---- sums q . c of 16 tokens at a time, tokens r and r + 8 in a lane
            float sc[SUB][KT][2];
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
                uint32_t w0[U], w1[U], pr0[NG], pr1[NG];
                load_words<U>(at + words_at(b), w0);
                load_words<U>(at + words_at(b) + 4 * D, w1);
                load_pairs<NG>(at + pairs_at(b), pr0);
                load_pairs<NG>(at + pairs_at(b) + 8 * NG * 4, pr1);
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
                            const uint4 f = SH::kQueryShared ? queries[(vt * U + u) * 32 + lane]
                                                             : qf[vt][SH::kQueryShared ? 0 : u];
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
                        const float z0 = g ? fmaf(b0, qs, sc[b][kt][0]) : b0 * qs;
                        const float z1 = g ? fmaf(b1, qs, sc[b][kt][1]) : b1 * qs;
                        sc[b][kt][0] = fmaf(s0, a[kt / 2][kt & 1], z0);
                        sc[b][kt][1] = fmaf(s1, a[kt / 2][2 + (kt & 1)], z1);
                    }
                }
            }
            if (!(tile.state & kAll)) {
                // some row does not see some token; what no row sees may hold anything
                int pos[KT];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) pos[kt] = kHeld ? held[kt] : position(kt);
#pragma unroll
                for (int b = 0; b < SUB; ++b) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = tile.t0 + 16 * b + r + 8 * i;
                        // (all rows see the same of a shared prefix)
                        const bool flat = P::kTwo && (tile.state & kPrefix);
                        const bool live = ((tile.state >> b) & 1) && t <= (flat ? sp.prefix - 1 : p1) &&
                                          (!p.window || t > p0 - p.window || t < p.sinks);
                        if (!live) {
                            for (int g = i4; g < NG; g += 4)
                                *reinterpret_cast<uint32_t*>(at + v_off + pairs_at(b) + 8 * i * NG * 4 +
                                                             g * 4) = 0u;
                        }
#pragma unroll
                        for (int kt = 0; kt < KT; ++kt)
                            if (!(live && (flat ? pos[kt] != kNoRow : t <= pos[kt]) &&
                                  (!p.window || t > pos[kt] - p.window || t < p.sinks)))
                                sc[b][kt][i] = -INFINITY;
                    }
                }
                fence_proxy_async_smem();  // the slot's next copy comes after these stores
                __syncwarp();
            }
            // ---- running maximum: moved only when a score is far above it, and the
            // values' power of two, when a scale is above it
            uint32_t scales = 0;  // the low half word
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
                uint32_t pr0[NG], pr1[NG];
                load_pairs<NG>(at + v_off + pairs_at(b), pr0);
                load_pairs<NG>(at + v_off + pairs_at(b) + 8 * NG * 4, pr1);
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    scales = max_u16x2(scales, max_u16x2(pr0[g], pr1[g]));
            }
            scales &= 0xFFFFu;
            float top[KT];
            bool over = scales > v_bound;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                top[kt] = -INFINITY;
#pragma unroll
                for (int b = 0; b < SUB; ++b)
                    top[kt] = fmaxf(top[kt], fmaxf(sc[b][kt][0] * unit[kt], sc[b][kt][1] * unit[kt]));
                over |= top[kt] > m[kt] + 8.f;
            }
            if (__any_sync(0xFFFFFFFFu, over)) {
                uint32_t big = __reduce_max_sync(0xFFFFFFFFu, scales);
                if (big > 0x7FFFu) {
                    // a scale with its sign set, which comes here every time: only the sizes count
                    uint32_t size = 0;
#pragma unroll 1
                    for (int b = 0; b < SUB; ++b) {
                        uint32_t pr0[NG], pr1[NG];
                        load_pairs<NG>(at + v_off + pairs_at(b), pr0);
                        load_pairs<NG>(at + v_off + pairs_at(b) + 8 * NG * 4, pr1);
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            size = max(size, max(pr0[g] & 0x7FFFu, pr1[g] & 0x7FFFu));
                    }
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
                        for (int c = 0; c < 4; ++c)
                            acc[vt][t][c] *= f[KT == 1 ? 0 : 2 * vt + (c & 1)];
            }
            // ---- weighted sum of the values
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
                uint32_t w0[U], w1[U], pr0[NG], pr1[NG];
                load_pairs<NG>(at + v_off + pairs_at(b), pr0);
                load_pairs<NG>(at + v_off + pairs_at(b) + 8 * NG * 4, pr1);
                load_words<U>(at + v_off + words_at(b), w0);
                load_words<U>(at + v_off + words_at(b) + 4 * D, w1);
                float e0[KT], e1[KT], h0[KT], h1[KT];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    e0[kt] = exp2_approx(fmaf(sc[b][kt][0], unit[kt], -mu[kt]));
                    e1[kt] = exp2_approx(fmaf(sc[b][kt][1], unit[kt], -mu[kt]));
                    l[kt] += e0[kt] + e1[kt];
                    h0[kt] = e0[kt] * v_up;
                    h1[kt] = e1[kt] * v_up;
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float s0 = __uint_as_float(pr0[g] << 16);
                    const float s1 = __uint_as_float(pr1[g] << 16);
                    const float b0 = __uint_as_float(pr0[g] & 0xFFFF0000u);
                    const float b1 = __uint_as_float(pr1[g] & 0xFFFF0000u);
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
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
        }

        // ---- the warps' results of this row tile become one, once those of the last
        // have been read
        if (joins && gave_up(warp_wait(&freed, (uint32_t)(joins - 1) & 1u, p.wait_budget))) return;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            const float x = sum_rows(l[kt]);
            if (r == 0) stat[warp * SH::kRows + kt * 4 + i4] = make_float2(m[kt], x);
#pragma unroll
            for (int g = 0; g < NG; ++g) pb[kt][g] = sum_rows(pb[kt][g]);
        }
        const float v_down = pow2_of(max(v_exp - 6, 1));  // 1 / v_up
        const bool whole = sp.flags == (kBegins | kEnds);
        float* part = p.partial +
                      ((long long)cta * 2 + ((sp.flags & kBegins) ? 1 : 0)) *
                          SH::kPartialFloats;
#pragma unroll 1
        for (int d0 = 0; d0 < D; d0 += kChunk) {
            if (d0 && gave_up(warp_wait(&freed, (uint32_t)(joins - 1) & 1u, p.wait_budget))) return;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if (t / (kChunk / 16) != d0 / kChunk) continue;
#pragma unroll
                for (int vt = 0; vt < VT; ++vt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (KT == 1 && (c & 1)) continue;
                        const int kt = 2 * vt + (c & 1);
                        join[(warp * SH::kRows + kt * 4 + i4) * kRowPad + (t % (kChunk / 16)) * 16 +
                             r + (c >> 1) * 8] =
                            fmaf(acc[vt][t][c] * (c >> 1 ? 0x1p20f : 0x1p24f), v_down,
                                 pb[kt][t * 16 / G]);
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&joined);
            if (gave_up(warp_wait(&joined, (uint32_t)joins & 1u, p.wait_budget))) return;
            for (int e = threadIdx.x; e < SH::kRows * (kChunk / 4); e += kThreads - 32) {
                const int row = e / (kChunk / 4), d = (e % (kChunk / 4)) * 4;
                if (row >= rows) break;
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
                if (whole) {
                    const long long to =
                        (long long)(sp.row0 + row / heads) * p.Hq + head0 + row % heads;
                    const float inv = ll > 0.f ? 1.f / ll : 0.f;
                    uint2 v;
                    v.x = cvt_bf16x2(o.x * inv, o.y * inv);
                    v.y = cvt_bf16x2(o.z * inv, o.w * inv);
                    *reinterpret_cast<uint2*>(p.out + to * D + d0 + d) = v;
                    if (p.lse && d0 + d == 0)
                        p.lse[to] = log_sum_of(mm, ll);
                } else {
                    *reinterpret_cast<float4*>(part + 2 * SH::kRows + row * D + d0 + d) = o;
                    if (d0 + d == 0) {
                        part[2 * row] = mm;
                        part[2 * row + 1] = ll;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&freed);
            ++joins;
        }
        // everyone is done with the piece before this one: its place takes a later one
        if (threadIdx.x == 0 && at_piece > 0)
            walk.next(p, &pieces[(at_piece - 1) % kPieces], seg);
    }
}

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

template <int D, int G, int KT, class P>
cudaError_t launch(const P& p, cudaStream_t stream) {
    using SH = Shape<D, G, KT>;
    static std::atomic<uint64_t> asked{0};  // devices on which the kernel may take its memory
    cudaError_t err = allow_shared(kv_attn_kernel<D, G, KT, P>, SH::kSmem, asked);
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
    if constexpr (P::kTwo) most += ((long long)p.max_prefix_pages * p.page_size + SH::kTile - 1) / SH::kTile;
    if (row_tiles <= p.ctas && most <= kUncutTiles &&
        most * (p.ctas - row_tiles) <= 2LL * SH::kWarps * p.ctas) {
        P one = p;
        one.whole = 1;
        kv_attn_kernel<D, G, KT, P><<<(unsigned)row_tiles, SH::kThreads, SH::kSmem, stream>>>(one);
        return cudaGetLastError();
    }
    const unsigned grid = (unsigned)p.ctas;
    kv_attn_kernel<D, G, KT, P><<<grid, SH::kThreads, SH::kSmem, stream>>>(p);
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
    return cudaLaunchKernelEx(&cfg, kv_join_kernel<D>, static_cast<const KvAttnParams&>(p), (int)SH::kRows);
}

}  // namespace

#ifndef MXQ_KV_TWO
size_t kv_attn_seg_bytes(int ctas) { return (size_t)ctas * 2 * sizeof(Seg); }

size_t kv_attn_partial_bytes(int ctas, int tile_rows, int D) {
    return (size_t)ctas * 2 * tile_rows * (D + 2) * sizeof(float);
}

int kv_attn_ctas_per_sm() { return Shape<128, 64, 1>::kCtas; }
#endif

#define MXQ_KV_ATTN(d, g)                                        \
    if (D == d && G == g)                                        \
        return tile_rows <= 4   ? launch<d, g, 1>(p, stream)     \
               : tile_rows <= 8 ? launch<d, g, 2>(p, stream)     \
                                : launch<d, g, 4>(p, stream);
#define MXQ_KV_ATTN_ALL   \
    MXQ_KV_ATTN(64, 32)   \
    MXQ_KV_ATTN(64, 64)   \
    MXQ_KV_ATTN(128, 32)  \
    MXQ_KV_ATTN(128, 64)  \
    MXQ_KV_ATTN(128, 128) \
    MXQ_KV_ATTN(256, 32)  \
    MXQ_KV_ATTN(256, 64)  \
    MXQ_KV_ATTN(256, 128)

#ifdef MXQ_KV_TWO
cudaError_t launch_kv_two(const KvTwoParams& p, int D, int G, int tile_rows, cudaStream_t stream) {
    MXQ_KV_ATTN_ALL
    return cudaErrorInvalidValue;
}
#else
cudaError_t launch_kv_attn(const KvAttnParams& p, int D, int G, int tile_rows,
                           cudaStream_t stream) {
    MXQ_KV_ATTN_ALL
    return cudaErrorInvalidValue;
}
#endif
#undef MXQ_KV_ATTN_ALL
#undef MXQ_KV_ATTN

}  // namespace mxq
