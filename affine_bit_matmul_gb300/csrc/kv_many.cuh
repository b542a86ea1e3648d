// Attention of many query rows (prompts, chunks of them) over a paged 4-bit
// key/value cache, on the 5th-generation tensor cores.
//
// The formulas are kv_attention.cu's; here keys and values become f16 numbers,
// s q + b rounded once (11 bits), scaled by a power of two for each 32 tokens that
// keeps them within the type's range, and so do the queries (a
// power of two for each row, exact) and the weights P (11 bits).  Products are
// summed in fp32 in tensor memory; scores, maxima and sums are fp32.
//
// A row tile is up to 256 rows (128 for D = 256): all query heads of one
// key/value head at 128 / heads tokens, once or twice.  A unit is (row tile,
// 128 tokens); the units of all row tiles, in order, are cut into equal runs,
// one per SM, as for few rows.  Roles of a CTA's 19 warps:
//   0-3, 4-7  softmax of the first and second 128 rows, one row a thread:
//             scores from tensor memory, maximum, weights back into tensor
//             memory over the scores, and the output at the end
//   8-15      codes -> f16 operands in shared memory (128-byte swizzle; keys
//             along the values, values along the tokens): 32 tokens of the keys or
//             of the values of a unit each, loaded a unit ahead into registers
//   16, 17    the matrix instructions of one half each: Q K^T, then P V
//   18        the list of the run's pieces; tensor memory
// The two halves are independent chains (scores, weights, sum), and each has two
// score tiles in turn (of 64 tokens; D = 256 has one half with two tiles of 128), so that
// products run while the softmax warps work.  The running maximum is only moved when
// a score exceeds it by 2^8; the output's sums in tensor memory are rescaled then, by
// the softmax warps.
//   In a call over shared prefixes the rows are a group's (token, query head) pairs, as many as fill a
// tile, all of which see the whole prefix; the first SMs take them, by the costs of both parts, and all pieces go to
// the workspace.  Tiles of up to 128 rows are for both halves, which take alternate units: 2.4 us a unit of
// 128 tokens then, 2.6 to 3.1 of 256 rows.  256 rows of 32 heads, 8 of 128 values, over 32768 tokens and 512 of
// their own: 217 us, and 25 for the join.
//   4 D flops per visible pair and head: a chunk of 2048 tokens that ends at 8192, 32 query
// heads of 128 values, takes 285 us, 840 TFLOP/s (score tiles of 128 tokens, one a half:
// 333 us); a whole prompt of 8192, 642 us.  Bound by the softmax warps' instructions:
// the schedulers issue in 60% of the cycles, the tensor cores work in 36 to 48%.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <type_traits>

#include "kv_attn_common.cuh"
#include "kv_shared.cuh"

namespace mxq {
namespace {

constexpr int kTile = 128;           // tokens of a unit
constexpr int kThreads = 608;
constexpr int kPieceRing = 8;
constexpr int kMetaRing = 4;
// What the ends of a row tile cost (queries in, output out), in units, while the runs
// are cut.  8 whole prompts of 2048 tokens, 32 query heads of 128 values: 782, 625, 538,
// 469, 449, 460, 483 us with 0, 1, 2, 3, 4, 5, 8; 16 of 300: 110, 86, 85, 87, 81, 82, 87;
// the longest calls do not care.
constexpr int kEndUnits = 4;
constexpr int kPart = 32;            // tokens that share a power of two
constexpr int kParts = kTile / kPart;

template <int D, int G>
struct Shape {
    static constexpr int MT = D == 256 ? 1 : 2;    // halves of 128 rows
    // Tokens of one score tile; two of them in turn for each half, so that the tensor
    // cores work on the next while one is weighed.
    static constexpr int kCols = D == 256 ? 128 : 64;
    static constexpr int kSubs = kTile / kCols;
    static constexpr int KB = D == 256 ? 1 : 2;    // key and value buffers
    static constexpr int kRows = 128 * MT;
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kOpBytes = kTile * D * 2;
    static constexpr int kSmem = 1024 + kQBytes + 2 * KB * kOpBytes;
    static constexpr int kPartialFloats = kRows * (D + 2);
};

struct Piece {
    int row0, toks, p0, head0, heads, s, h, head_tiles, tail, k0, count, flags;
    // Shared prefixes: position of the last row, place of the result, and the first of its (token,
    // query head) rows, of which `toks` is the number.
    int p1, slot, flat0;
};
template <class P>
__device__ __forceinline__ int last_position(const Piece& q) {
    if constexpr (P::kShared) return q.p1;
    else return q.p0 + q.toks - 1;
}

// One row tile, in the workspace.
struct Entry {
    int s, row0, toks, p0, tiles, head_tiles, tail, pad;
};

// Of each part of a unit, one byte: the biased exponent e of the keys' and of the
// values' power of two (they are below 2^(e - 126)), and which 16 tokens exist.
struct Meta {
    uint8_t k_exp[kParts], v_exp[kParts], there[kParts];
};

__device__ __forceinline__ int unit_token(const Piece& q, int k) {
    return (k < q.head_tiles ? k : q.tail + k - q.head_tiles) * kTile;
}

// Whether a row tile of a shared prefix has rows for one half only: both halves then take all of them,
// for alternate units, and leave a result each.  (Every piece has rows: both the warps that issue the products and those
// that weigh the scores go by that.)
template <int D, int G, class P>
__device__ __forceinline__ bool is_narrow(const Piece& q) {
    return P::kShared && Shape<D, G>::MT == 2 && q.toks <= 128;
}

// Waits for this thread's tensor-memory loads; the registers named are not used
// before.
__device__ __forceinline__ void tmem_ld_wait_of(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// 8 columns of this thread's lane.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr)
        : "memory");
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
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t hmul2_f16(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Instruction descriptor for kind::f16: f16 A and B, fp32 D, both K-major.
__host__ __device__ constexpr uint32_t umma_idesc_f16(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ uint32_t hfma2_f16(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// The four pairs of a code word (nibbles 0 and 4, 1 and 5, ...) as s q + b in f16.
// As f16 numbers the masked codes are 2^-24 and 2^-20 times their values (both
// subnormal): s is 2^24 times what it is, and 2^20 for the odd ones.
__device__ __forceinline__ void dequant_word(uint32_t w, uint32_t s_even, uint32_t s_odd,
                                             uint32_t b2, uint32_t (&x)[4]) {
    const uint32_t v = w >> 8;
    x[0] = hfma2_f16(w & 0x000F000Fu, s_even, b2);
    x[1] = hfma2_f16(w & 0x00F000F0u, s_odd, b2);
    x[2] = hfma2_f16(v & 0x000F000Fu, s_even, b2);
    x[3] = hfma2_f16(v & 0x00F000F0u, s_odd, b2);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void sts32(uint32_t at, uint32_t a) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(a) : "memory");
}

// Barriers and small things that the warps share.  A wait names a phase by its parity, so
// each is placed where the phase before has ended and the one after cannot end without
// the waiting warp.  Those of the score tiles are two for each half, used in turn: the
// softmax warps may be a tile apart.
template <int D, int G>
struct Shared {
    using SH = Shape<D, G>;
    uint64_t piece_full[kPieceRing], piece_empty[kPieceRing];
    uint64_t k_full[SH::KB], k_empty[SH::KB], v_full[SH::KB], v_empty[SH::KB];
    uint64_t v_known[kMetaRing];  // the values' powers of two of a unit, before its buffer is free
    uint64_t q_full[SH::MT], s_full[2 * SH::MT], p_full[2 * SH::MT], pv_done[2 * SH::MT], drained[SH::MT];
    Piece pieces[kPieceRing];
    Meta meta[kMetaRing];
    uint32_t tmem;
};

// The pieces of the run in order, for one warp.
template <int D, int G>
struct Pieces {
    Shared<D, G>& sh;
    long long budget;
    int n;
    __device__ Pieces(Shared<D, G>& s, long long b) : sh(s), budget(b), n(0) {}
    // The next piece; null when a wait gave up.  count == 0: no more.
    __device__ const Piece* next() {
        if (!warp_wait_sleep(&sh.piece_full[n % kPieceRing], (uint32_t)(n / kPieceRing) & 1u, budget))
            return nullptr;
        return &sh.pieces[n % kPieceRing];
    }
    __device__ void done() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.piece_empty[n % kPieceRing]);
        ++n;
    }
};

// ---------------------------------------------------------------- pieces

template <int D, int G>
__device__ bool list_pieces(const KvAttnParams& p, Shared<D, G>& sh) {
    pdl_wait();  // for the plan
    const Entry* entries = reinterpret_cast<const Entry*>(p.entries);
    const int* before = p.before;
    const int n_entries = p.counts[0];
    const long long vheads = (long long)p.Hkv * p.head_parts;
    const long long all = p.counts[1] * vheads;
    const long long runs = all < p.ctas ? all : p.ctas;
    const int cta = blockIdx.x, rep = p.Hq / p.Hkv;
    Seg* seg = reinterpret_cast<Seg*>(p.segs) + (long long)cta * 2;
    seg[0].flags = seg[1].flags = -1;
    long long left = 0;
    int e = 0, k = 0, h = 0, part = 0;
    Entry en{};
    if (cta < runs) {
        const long long u0 = cta * all / runs;
        left = (cta + 1) * all / runs - u0;
        int lo = 0, hi = n_entries - 1;  // the last entry that begins at or before u0
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (before[mid] * vheads <= u0) lo = mid;
            else hi = mid - 1;
        }
        e = lo;
        en = entries[e];
        const long long at = u0 - before[e] * vheads;
        const int vh = (int)(at / (en.tiles + kEndUnits));
        k = (int)(at % (en.tiles + kEndUnits));
        h = vh / p.head_parts;
        part = vh % p.head_parts;
    }
    for (int n = 0;; ++n) {
        const int slot = n % kPieceRing;
        if (!mbar_wait_sleep(&sh.piece_empty[slot], ((uint32_t)(n / kPieceRing) & 1u) ^ 1u, p.wait_budget))
            return false;
        Piece q{};
        while (left > 0 && q.count == 0) {
            const int units = en.tiles + kEndUnits, n_units = (int)(left < units - k ? left : units - k);
            const int tiles = min(k + n_units, en.tiles) - k;  // the others are the row tile's end
            if (tiles > 0) {
                q.row0 = en.row0;
                q.toks = en.toks;
                q.p0 = en.p0;
                q.head0 = h * rep + part * p.part_heads;
                q.heads = min(p.part_heads, rep - part * p.part_heads);
                q.s = en.s;
                q.h = h;
                q.head_tiles = en.head_tiles;
                q.tail = en.tail;
                q.k0 = k;
                q.count = tiles;
                q.flags = (k == 0 ? kBegins : 0) | (k + tiles == en.tiles ? kEnds : 0);
                if (q.flags != (kBegins | kEnds)) {
                    Seg g;
                    g.row0 = q.row0;
                    g.toks = q.toks;
                    g.head0 = q.head0;
                    g.heads = q.heads;
                    g.flags = q.flags;
                    seg[(q.flags & kBegins) ? 1 : 0] = g;
                }
            }
            left -= n_units;
            k += n_units;
            if (k == units && left > 0) {
                k = 0;
                if (++part == p.head_parts) {
                    part = 0;
                    if (++h == p.Hkv) {
                        h = 0;
                        en = entries[++e];
                    }
                }
            }
        }
        sh.pieces[slot] = q;
        mbar_arrive(&sh.piece_full[slot]);
        if (q.count == 0) return true;
    }
}

// The same for the groups of a call over shared prefixes, by one lane.
template <int D, int G>
__device__ bool list_pieces(const KvSharedParams& p, Shared<D, G>& sh, SharedWalk& walk) {
    for (int n = 0;; ++n) {
        const int slot = n % kPieceRing;
        if (!mbar_wait_sleep(&sh.piece_empty[slot], ((uint32_t)(n / kPieceRing) & 1u) ^ 1u, p.wait_budget))
            return false;
        Piece q{};
        SharedPiece s;
        if (walk.next(p, &s)) {
            find_rows(p, s);
            q.heads = s.heads;
            q.head0 = s.head0;
            q.flat0 = s.flat0;
            q.toks = s.rows;
            q.row0 = s.it.row0;
            q.p0 = q.p1 = s.p1;
            q.s = s.item;
            q.h = s.h;
            q.k0 = s.k0;
            q.count = s.count;
            q.slot = s.tile + blockIdx.x;
        }
        sh.pieces[slot] = q;
        mbar_arrive(&sh.piece_full[slot]);
        if (q.count == 0) return true;
    }
}

// ---------------------------------------------------------------- codes -> operands

// Warp cw of eight converts 32 tokens of the keys (0 .. 3) or of the values of
// each unit.  Its loads run a unit ahead, the page numbers two.
template <int D, int G, class P>
struct Convert {
    using SH = Shape<D, G>;
    static constexpr int KB = SH::KB, NG = D / G, U = D / 32;
    const P& p;
    Shared<D, G>& sh;
    const int lane, part;
    const bool kv;
    // where the page numbers are looked up: unit at_k of piece at_n
    int at_n, at_k;
    bool at_end;
    // looked up: pages of the 32 tokens' halves; -2: not needed
    int id[2], look_t, look_p0, look_p1, look_h;
    // loaded
    uint32_t w[4][U], pr[NG];
    int t0, p0, p1, state;

    __device__ Convert(const P& p_, Shared<D, G>& sh_, int cw, int lane_)
        : p(p_), sh(sh_), lane(lane_), part(cw % kParts), kv(cw >= kParts), at_n(0), at_k(-1),
          at_end(false) {}

    __device__ bool look() {
        if (at_end) return true;
        ++at_k;
        if (at_k == 0 || at_k == sh.pieces[at_n % kPieceRing].count) {
            if (at_k) ++at_n;
            at_k = 0;
            if (!warp_wait_sleep(&sh.piece_full[at_n % kPieceRing], (uint32_t)(at_n / kPieceRing) & 1u,
                           p.wait_budget))
                return false;
        }
        const Piece& q = sh.pieces[at_n % kPieceRing];
        if (q.count == 0) {
            at_end = true;
            return true;
        }
        look_t = unit_token(q, q.k0 + at_k) + part * kPart;
        look_p0 = q.p0;
        look_p1 = last_position<P>(q);
        look_h = q.h;
        const int32_t* row = p.table + (long long)q.s * p.max_pages;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = look_t + 16 * i;
            id[i] = t <= look_p1 ? row[t >> p.page_shift] : -2;
        }
        return true;
    }
    __device__ void load() {
        t0 = look_t;
        p0 = look_p0;
        p1 = look_p1;
        state = 0;
        const int size = p.page_size;
        const int half = kv_block_bytes(D, G, size) / 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = t0 + 16 * i;
            if ((unsigned)id[i] < (unsigned)p.n_pages) {
                state |= 1 << i;
                const uint8_t* src = p.pages + ((long long)id[i] * p.Hkv + look_h) * (2LL * half) +
                                     (kv ? half : 0);
                const int skip = t & (size - 1);
                const uint8_t* codes = src + kv_code_bytes(D, skip) + lane * (D == 64 ? 8 : 16);
                load_words<U>(codes, w[2 * i]);
                load_words<U>(codes + 4 * D, w[2 * i + 1]);
                // lane i's pairs are those of token t0 + i
                if (lane / 16 == i)
                    load_pairs<NG>(src + kv_code_bytes(D, size) + (skip + lane % 16) * (NG * 4), pr);
            } else if (id[i] != -2 && !kv) {
                // a page that some row sees has to exist
                const int te = min(t + 15, p1);
                if (!p.window || te > p0 - p.window || t < p.sinks)
                    flag_status(p.status, MXQ_DEV_BAD_PAGE);
            }
        }
    }
    // The biased exponent e of a power of two above the unit's values: they are below
    // 2^(e - 126).
    __device__ int scale_bits() {
        const int t = t0 + lane;
        // what no row sees may hold anything
        if (!((state >> (lane / 16)) & 1) || t > p1 ||
            (p.window && t <= p0 - p.window && t >= p.sinks)) {
#pragma unroll
            for (int g = 0; g < NG; ++g) pr[g] = 0u;
        }
        uint32_t big = 0;
#pragma unroll
        for (int g = 0; g < NG; ++g) big = max_u16x2(big, pr[g] & 0x7FFF7FFFu);
        const int es = (int)(__reduce_max_sync(0xFFFFFFFFu, big & 0xFFFFu) >> 7) + 4;
        const int eb = (int)(__reduce_max_sync(0xFFFFFFFFu, big >> 16) >> 7);
        return min(max(max(es, eb) + 1, 30), 247);
    }
    // The loaded unit into operand buffer `out`.
    __device__ void store(uint32_t out, int e) {
        const int r = lane >> 2, i4 = lane & 3;
        // Values come out below 2^-5, so that 2^24 times a scale, which is at most 2^-5 of
        // the largest value, is an f16 number.
        const float dn = pow2_of(248 - e);  // 2^(121 - e)
        // each lane's own token as f16 pairs (scale, bias)
        uint32_t sb[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g)
            sb[g] = cvt_f16x2(__uint_as_float(pr[g] << 16) * dn * 0x1p24f,
                              __uint_as_float(pr[g] & 0xFFFF0000u) * dn);
        constexpr uint32_t sixteenth = 0x2C002C00u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // 8 tokens at a time
            if (!kv) {
                uint32_t s2[NG], t2[NG], b2[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint32_t x = __shfl_sync(0xFFFFFFFFu, sb[g], 8 * j + r);
                    s2[g] = prmt(x, x, 0x1010u);
                    t2[g] = hmul2_f16(s2[g], sixteenth);
                    b2[g] = prmt(x, x, 0x3232u);
                }
                const uint32_t row = out + (part * kPart + 8 * j + r) * 128;
                // odd tokens take the words of a pair in the other order: their
                // stores would meet the even ones' in the same banks
                const bool odd = r & 1;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint32_t word = odd ? w[j][u ^ 1] : w[j][u];
                    const int g0 = u * 32 / G, g1 = (u ^ 1) * 32 / G;
                    uint32_t x[4];
                    const bool other = g0 != g1 && odd;
                    dequant_word(word, other ? s2[g1] : s2[g0], other ? t2[g1] : t2[g0],
                                 other ? b2[g1] : b2[g0], x);
                    // values 32 u' + 8 i4 ..: 16 bytes of the token's row
                    const int chunk = (((u & 1) ^ (r & 1)) * 4 + i4) ^ r;
                    sts128(row + (u / 2) * (kTile * 128) + chunk * 16, x[0], x[1], x[2], x[3]);
                }
            } else {
                // values 32 u + r + 8 n of tokens 2 i4 and 2 i4 + 1
                const int tt = part * kPart + 8 * j;
                const uint32_t row = out + (tt / 64) * (D * 128) + r * 128 +
                                     ((((tt % 64) / 8) ^ r) * 16) + i4 * 4;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint32_t a = __shfl_sync(0xFFFFFFFFu, sb[g], 8 * j + 2 * i4);
                    const uint32_t c = __shfl_sync(0xFFFFFFFFu, sb[g], 8 * j + 2 * i4 + 1);
                    const uint32_t s2 = prmt(a, c, 0x5410u), b2 = prmt(a, c, 0x7632u);
                    const uint32_t t2 = hmul2_f16(s2, sixteenth);
#pragma unroll
                    for (int u = g * G / 32; u < (g + 1) * G / 32; ++u) {
                        uint32_t x[4];
                        dequant_word(w[j][u], s2, t2, b2, x);
#pragma unroll
                        for (int n = 0; n < 4; ++n) sts32(row + (32 * u + 8 * n) * 128, x[n]);
                    }
                }
            }
        }
    }
    __device__ bool run(uint32_t kbuf, uint32_t vbuf) {
        if (!look()) return false;
        if (!at_end) load();
        bool more = !at_end;
        if (!look()) return false;
        int n = 0, left = 0;  // piece of the loaded unit, its units left
        for (int jt = 0; more; ++jt) {
            if (left == 0) left = sh.pieces[n % kPieceRing].count;
            const int buf = jt % KB;
            const int e = scale_bits(), here = state;
            if (kv && lane == 0) {
                // the softmax warps need no more of the values
                sh.meta[jt % kMetaRing].v_exp[part] = (uint8_t)e;
                mbar_arrive(&sh.v_known[jt % kMetaRing]);
            }
            if (!warp_wait_sleep(kv ? &sh.v_empty[buf] : &sh.k_empty[buf], ((uint32_t)(jt / KB) & 1u) ^ 1u,
                           p.wait_budget))
                return false;
            store((kv ? vbuf : kbuf) + buf * SH::kOpBytes, e);
            if (!kv && lane == 0) {
                Meta& meta = sh.meta[jt % kMetaRing];
                meta.k_exp[part] = (uint8_t)e;
                meta.there[part] = (uint8_t)here;
            }
            fence_proxy_async_smem();  // the tensor cores read what was written
            __syncwarp();
            if (lane == 0) mbar_arrive(kv ? &sh.v_full[buf] : &sh.k_full[buf]);
            more = !at_end;
            if (more) load();
            if (--left == 0) {
                if (lane == 0) mbar_arrive(&sh.piece_empty[n % kPieceRing]);
                ++n;
            }
            if (more && !look()) return false;
        }
        return true;
    }
};

// ---------------------------------------------------------------- matrix instructions

// One warp issues the instructions of one half.
template <int D, int G, class P>
__device__ bool issue_products(const P& p, Shared<D, G>& sh, uint32_t qbuf, uint32_t kbuf,
                               uint32_t vbuf, uint32_t tmem, int m, int lane) {
    using SH = Shape<D, G>;
    constexpr int KB = SH::KB, kCols = SH::kCols, kSubs = SH::kSubs;
    constexpr uint32_t id_s = umma_idesc_f16(128, kCols), id_o = umma_idesc_f16(128, D);
    const uint32_t o_col = tmem + 256 + m * D, s_cols = tmem + m * kTile;
    Pieces<D, G> list(sh, p.wait_budget);
    int jt = 0;   // units so far: key and value buffers
    int at = 0;   // score tiles of this half so far
    int nq = 0;   // pieces of this half so far
    for (;;) {
        const Piece* q = list.next();
        if (!q) return false;
        const int count = q->count;
        if (count == 0) return true;
        // the units of this half: all of them, or every other one
        const bool narrow = is_narrow<D, G, P>(*q);
        const int k_first = narrow ? m : 0, k_step = narrow ? 2 : 1;
        // lets unit k's keys or values go without using them
        auto leave = [&](int k, uint64_t* full, uint64_t* empty) {
            const int j = jt + k, buf = j % KB;
            if (!warp_wait_sleep(&full[buf], (uint32_t)(j / KB) & 1u, p.wait_budget)) return false;
            if (lane == 0) mbar_arrive(&empty[buf]);
            return true;
        };
        auto leave_keys = [&](int k) { return leave(k, sh.k_full, sh.k_empty); };
        auto leave_values = [&](int k) { return leave(k, sh.v_full, sh.v_empty); };
        if (narrow ? k_first >= count : q->toks <= m * (P::kShared ? 128 : p.half_toks)) {
            // no rows in this half
            for (int k = 0; k < count; ++k)
                if (!leave_keys(k) || !leave_values(k)) return false;
            jt += count;
            list.done();
            continue;
        }
        if (!warp_wait_sleep(&sh.q_full[m], (uint32_t)nq & 1u, p.wait_budget)) return false;
        ++nq;
        // scores of tile i of the piece
        auto scores = [&](int i) {
            const int k = k_first + i / kSubs * k_step, j = jt + k, sub = i % kSubs, buf = j % KB, a = at + i;
            if (narrow && sub == 0 && k > 0 && !leave_keys(k - 1)) return false;
            if (!warp_wait_sleep(&sh.k_full[buf], (uint32_t)(j / KB) & 1u, p.wait_budget)) return false;
            // the buffer's earlier weights have been used
            if (i >= 2 && !warp_wait_sleep(&sh.pv_done[2 * m + (a & 1)], (uint32_t)((a >> 1) - 1) & 1u, p.wait_budget))
                return false;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t s_col = s_cols + (a & 1) * kCols;
#pragma unroll
                for (int kb = 0; kb < D / 64; ++kb) {
                    const uint64_t ad = umma_desc_sw128(qbuf + (m * (D / 64) + kb) * (128 * 128));
                    const uint64_t bd = umma_desc_sw128(kbuf + buf * SH::kOpBytes +
                                                        (kb * kTile + sub * kCols) * 128);
#pragma unroll
                    for (int j4 = 0; j4 < 4; ++j4)
                        umma_bf16(s_col, ad + 2 * j4, bd + 2 * j4, id_s, kb | j4 ? 1u : 0u);
                }
                umma_commit(&sh.s_full[2 * m + (a & 1)]);
                if (sub == kSubs - 1) umma_commit(&sh.k_empty[buf]);
            }
            __syncwarp();
            return true;
        };
        const int n_units = (count - k_first + k_step - 1) / k_step, n_tiles = n_units * kSubs;
        if (!scores(0)) return false;
        for (int i = 0; i < n_tiles; ++i) {
            if (i + 1 < n_tiles && !scores(i + 1)) return false;
            const int k = k_first + i / kSubs * k_step, j = jt + k, sub = i % kSubs, buf = j % KB, a = at + i;
            if (narrow && sub == 0 && k > 0 && !leave_values(k - 1)) return false;
            if (!warp_wait_sleep(&sh.v_full[buf], (uint32_t)(j / KB) & 1u, p.wait_budget) ||
                !warp_wait_sleep(&sh.p_full[2 * m + (a & 1)], (uint32_t)(a >> 1) & 1u, p.wait_budget))
                return false;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t p_col = s_cols + (a & 1) * kCols;
#pragma unroll
                for (int tb = 0; tb < kCols / 64; ++tb) {
                    const uint64_t bd = umma_desc_sw128(vbuf + buf * SH::kOpBytes +
                                                        (sub * (kCols / 64) + tb) * (D * 128));
#pragma unroll
                    for (int j4 = 0; j4 < 4; ++j4)
                        umma_bf16_tmem_a(o_col, p_col + (tb * 4 + j4) * 8, bd + 2 * j4, id_o,
                                         i | tb | j4 ? 1u : 0u);
                }
                if (sub == kSubs - 1) umma_commit(&sh.v_empty[buf]);
                umma_commit(&sh.pv_done[2 * m + (a & 1)]);
            }
            __syncwarp();
        }
        if (k_first + (n_units - 1) * k_step < count - 1 && (!leave_keys(count - 1) || !leave_values(count - 1)))
            return false;
        jt += count;
        at += n_tiles;
        list.done();
    }
}

// ---------------------------------------------------------------- softmax

template <int D, int G, class P>
__device__ bool softmax(const P& p, Shared<D, G>& sh, uint32_t qbuf, uint32_t tmem, int m,
                        int quarter, int lane) {
    using SH = Shape<D, G>;
    constexpr int KB = SH::KB, kCols = SH::kCols, kSubs = SH::kSubs;
    const int lr = quarter * 32 + lane;                 // row of the half
    const uint32_t t_lane = (uint32_t)(quarter * 32) << 16;
    const uint32_t o_at = tmem + t_lane + 256 + m * D;
    Pieces<D, G> list(sh, p.wait_budget);
    int jt = 0, at = 0;
    for (;;) {
        const Piece* q = list.next();
        if (!q) return false;
        const int count = q->count;
        if (count == 0) return true;
        const int heads = q->heads, tok0 = P::kShared ? 0 : m * p.half_toks;
        const bool narrow = is_narrow<D, G, P>(*q);
        const int half0 = P::kShared && !narrow ? m * 128 : 0;  // first row of a shared prefix's half
        const int k_first = narrow ? m : 0, k_step = narrow ? 2 : 1;
        const int toks = P::kShared ? q->toks - half0 : min(p.half_toks, q->toks - tok0);
        if (toks <= 0) {
            jt += count;
            list.done();
            continue;
        }
        // the half's rows, and where they begin among the sequence's or group's
        const int rows = P::kShared ? min(128, toks) : toks * heads;
        const int flat0 = P::kShared ? q->flat0 + half0 : 0;
        const bool in = lr < rows;
        const int tok = in ? (flat0 + lr) / heads : 0, hh = in ? (flat0 + lr) % heads : 0;
        const int row = q->row0 + tok0 + tok;
        if (narrow && k_first >= count) {
            // this half has no unit
            if (in)
                *reinterpret_cast<float2*>(p.partial + (long long)q->slot * SH::kPartialFloats + 2 * (m * 128 + lr)) =
                    make_float2(-INFINITY, 0.f);
            jt += count;
            list.done();
            continue;
        }
        // positions of the half (all of a shared prefix's rows see all of it)
        const int first = P::kShared ? q->p0 : q->p0 + tok0, last = P::kShared ? first : first + toks - 1;
        const int pos = in ? (P::kShared ? first : first + tok) : -1;
        // ---- the warp's 32 query rows, D / 8 lanes a row: f16, the largest value of each
        // row 2^13 .. 2^14
        float unit;
        {
            constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
            const int c = lane % kLanes;
            const uint32_t base = qbuf + m * (D / 64) * (128 * 128) + (c / 8) * (128 * 128);
            int my_ex = 16;
            constexpr int kBatch = 8;
#pragma unroll 1
            for (int i0 = 0; i0 < kLanes; i0 += kBatch) {
                uint4 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    // (rows past the last repeat it; their scores are not used)
                    const int at_row = min(quarter * 32 + (i0 + i) * kAtOnce + lane / kLanes, rows - 1);
                    v[i] = *(reinterpret_cast<const uint4*>(
                                     p.q + (long long)(q->row0 + tok0 + (flat0 + at_row) / heads) * p.q_row_stride +
                                     (long long)(q->head0 + (flat0 + at_row) % heads) * p.q_head_stride) +
                                 c);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int at_row = quarter * 32 + (i0 + i) * kAtOnce + lane / kLanes;
                    uint32_t big = max_u16x2(max_u16x2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                             max_u16x2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
                    big = max(big & 0xFFFFu, big >> 16);
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1)
                        big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
                    const int ex = max((int)(big >> 7), 16);
                    // the lane whose row this is keeps the exponent
                    const int mine = __shfl_sync(0xFFFFFFFFu, ex, lane % kAtOnce * kLanes);
                    if (lane / kAtOnce == i0 + i) my_ex = mine;
                    const float up = pow2_of(267 - ex);  // 2^(140 - ex)
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[2 * e] = __uint_as_float(w[e] << 16) * up;
                        x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u) * up;
                    }
                    // in the order of a code word's pairs
                    sts128(base + at_row * 128 + (((c % 8) ^ (at_row % 8)) * 16),
                           cvt_f16x2(x[0], x[4]), cvt_f16x2(x[1], x[5]), cvt_f16x2(x[2], x[6]),
                           cvt_f16x2(x[3], x[7]));
                }
            }
            unit = p.scale_log2 * pow2_of(my_ex - 13);
        }
        fence_proxy_async_smem();
        tc_fence_before();  // (the last piece's output has been read)
        mbar_arrive(&sh.q_full[m]);

        float mx = -INFINITY, mu = 0.f, l = 0.f;
        int e_o = 30;  // the output's sums are of values over 2^(e_o - 126)
        // The first scores come after the values of all units before this piece, of which
        // a half without rows has not waited for any: a parity does not tell a phase from
        // the next but one.
        if (!warp_wait_sleep(&sh.s_full[2 * m + (at & 1)], (uint32_t)(at >> 1) & 1u, p.wait_budget))
            return false;
        // (counted on where no half leaves units out: 284.1 us for 2048 tokens of 8192, worked out 285.0)
        const int jt0 = jt, at0 = at;
        for (int k = k_first; k < count; k += k_step, jt += P::kShared ? 0 : 1) {
            if constexpr (P::kShared) jt = jt0 + k;
            const volatile uint32_t* meta =
                reinterpret_cast<const volatile uint32_t*>(&sh.meta[jt % kMetaRing]);
            // the values' powers of two: one ring ahead at most, since the units before are done with
            if (!warp_wait_sleep(&sh.v_known[jt % kMetaRing], (uint32_t)(jt / kMetaRing) & 1u, p.wait_budget))
                return false;
            const uint32_t v_exps = meta[1];
            const uint32_t two = __vmaxu4(v_exps, v_exps >> 16);
            const int e_new = max(e_o, (int)max(two & 0xFFu, (two >> 8) & 0xFFu));
#pragma unroll 1
            for (int sub = 0; sub < kSubs; ++sub, ++at) {
                const uint32_t s_at = tmem + t_lane + m * kTile + (at & 1) * kCols;
                const int t0 = unit_token(*q, q->k0 + k) + sub * kCols;
                const bool inside = t0 + kCols - 1 <= first &&
                                    (!p.window || t0 > last - p.window || t0 + kCols <= p.sinks);
                if (!warp_wait_sleep(&sh.s_full[2 * m + (at & 1)], (uint32_t)(at >> 1) & 1u, p.wait_budget))
                    return false;
                tc_fence_after();
                uint32_t xa[16], xb[16];
                tmem_ld16(s_at, xa);
                // (the keys' part is complete now that there are scores)
                const uint32_t k_exp = meta[0] >> (sub * kCols / 4), v_exp = v_exps >> (sub * kCols / 4);
                uint32_t state = meta[2];
                state |= state >> 6;              // 2 bits of each byte, together
                state = ((state | state >> 12) & 0xFFu) >> (sub * kCols / 16);
                constexpr uint32_t kThere = (1u << (kCols / 16)) - 1u;
                const bool edge = (state & kThere) != kThere || !inside;
                // what this row sees of columns c .. c + 15, as bits
                auto sees = [&](int c) {
                    uint32_t bits = 0;
                    if (!((state >> (c / 16)) & 1)) return bits;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int t = t0 + c + i;
                        const bool s = t <= pos && (!p.window || t > pos - p.window || t < p.sinks);
                        bits |= (s ? 1u : 0u) << i;
                    }
                    return bits;
                };
                // Moves the maximum and the values' power of two: what has been summed, and
                // the weights of this unit's first `c` columns, follow.
                auto move = [&](float top, int c) {
                    const float mn = fmaxf(mx, top);
                    mu = mn == -INFINITY ? 0.f : mn;
                    const float a = exp2_approx(mx - mu);
                    mx = mn;
                    l *= a;
                    const float f = a * pow2_of(max(e_o - e_new + 127, 1));
                    e_o = e_new;
                    tmem_st_wait();
                    const uint32_t a2 = cvt_f16x2(f, f);
#pragma unroll 1
                    for (int i = 0; i < c / 2; i += 8) {
                        uint32_t y[8];
                        tmem_ld8(s_at + i, y);
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = hmul2_f16(y[j], a2);
                        tmem_st8(s_at + i, y);
                    }
                    bool ok = true;
                    if (P::kShared ? at != at0 : k + sub > 0) {
                        // the sums so far, once the last tile's products are in
                        ok = warp_wait_sleep(&sh.pv_done[2 * m + ((at - 1) & 1)], (uint32_t)((at - 1) >> 1) & 1u, p.wait_budget);
                        tc_fence_after();
#pragma unroll 1
                        for (int i = 0; i < D; i += 8) {
                            uint32_t y[8];
                            tmem_ld8(o_at + i, y);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
                            tmem_st8(o_at + i, y);
                        }
                    }
                    return ok;
                };
                // 16 columns: weights over the scores.  f: the scores' factor, off: what is
                // added to them (with the maximum), back: the factor of the weights' sum.
                auto weigh = [&](uint32_t (&x)[16], int c, float f, float shift, float back, auto masked) {
                    if constexpr (decltype(masked)::value) {
                        const uint32_t bits = sees(c);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (!((bits >> i) & 1u)) x[i] = 0xFF800000u;  // -inf
                    }
                    float t = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
                    for (int i = 2; i < 16; i += 2)
                        t = max3(t, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                    const bool over = __any_sync(0xFFFFFFFFu, t * f > mx + 8.f);
                    uint32_t y[8];
                    float sum;
                    auto weights = [&]() {
                        const float off = shift - mu;
                        const uint64_t f2 = pair_of(f, f), off2 = pair_of(off, off);
                        uint64_t s0 = 0, s1 = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float a, b;
                            parts_of(fma_pair(pair_of(__uint_as_float(x[2 * i]),
                                                      __uint_as_float(x[2 * i + 1])),
                                              f2, off2), &a, &b);
                            a = exp2_approx(a);
                            b = exp2_approx(b);
                            uint64_t& s = i & 1 ? s1 : s0;
                            s = i > 1 ? add_pair(s, pair_of(a, b)) : pair_of(a, b);
                            y[i] = cvt_f16x2(a, b);
                        }
                        float a, b;
                        parts_of(add_pair(s0, s1), &a, &b);
                        sum = a + b;
                    };
                    weights();  // most often the maximum stays, and this has not waited for the vote
                    if (over) {
                        if (!move(t * f, c)) return false;
                        weights();
                    }
                    l = fmaf(sum, back, l);
                    tmem_st8(s_at + c / 2, y);
                    return true;
                };
                bool ok = true;
                if (e_new > e_o) ok = move(-INFINITY, 0);
                auto all_columns = [&](auto masked) {
                    tmem_ld_wait_of(xa);
#pragma unroll 1
                    for (int c = 0; c < kCols; c += 32) {
                        tmem_ld16(s_at + c + 16, xb);
                        const int ek = (k_exp >> (c / 4)) & 0xFF, de = ((v_exp >> (c / 4)) & 0xFF) - e_o;
                        // (never zero: a query of zeros still has -inf where it sees nothing)
                        const float f = fmaxf(unit * pow2_of(ek + 6), 0x1p-126f);  // 2^(e - 121)
                        const float shift = (float)(7 + de);  // de <= 0
                        const float back = pow2_of(min(127 - de, 254));
                        ok = weigh(xa, c, f, shift, back, masked) && ok;
                        tmem_ld_wait_of(xb);
                        if (c + 32 < kCols) tmem_ld16(s_at + c + 32, xa);
                        ok = weigh(xb, c + 16, f, shift, back, masked) && ok;
                        tmem_ld_wait_of(xa);
                    }
                };
                if (edge) all_columns(std::true_type());
                else all_columns(std::false_type());
                if (!ok) return false;
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&sh.p_full[2 * m + (at & 1)]);
            }
        }
        if constexpr (P::kShared) jt = jt0 + count;
        // ---- the row's result, once the products of the last tile, and so of all, are in
        if (!warp_wait_sleep(&sh.pv_done[2 * m + ((at - 1) & 1)], (uint32_t)((at - 1) >> 1) & 1u, p.wait_budget))
            return false;
        tc_fence_after();
        const bool whole = !P::kShared && q->flags == (kBegins | kEnds);
        const float up = pow2_of(e_o + 1) * 32.f;  // 2^(e_o - 121)
        l *= 0x1p-7f;
        const float inv = whole ? (l > 0.f ? up * (0x1p-7f / l) : 0.f) : up * 0x1p-7f;
        const long long to = (long long)row * p.Hq + q->head0 + hh;
        float* part = p.partial + (P::kShared ? q->slot
                                              : (long long)blockIdx.x * 2 + ((q->flags & kBegins) ? 1 : 0)) *
                                      SH::kPartialFloats;
        const int dense = P::kShared ? m * 128 + lr : tok0 * heads + lr;
        // A finished row goes through this half's query buffer, which is not needed any
        // more, so that the warp writes whole rows at a time.
        const uint32_t stage = qbuf + m * (D / 64) * (128 * 128);
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
            uint32_t x[16];
            tmem_ld16(o_at + c, x);
            tmem_ld_wait_of(x);
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(x[i]) * inv;
            if (whole) {
                const uint32_t row_at = stage + (c / 64) * (128 * 128) + lr * 128;
                sts128(row_at + ((((c % 64) / 8) ^ (lr % 8)) * 16), cvt_bf16x2(v[0], v[1]),
                       cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
                sts128(row_at + ((((c % 64) / 8 + 1) ^ (lr % 8)) * 16), cvt_bf16x2(v[8], v[9]),
                       cvt_bf16x2(v[10], v[11]), cvt_bf16x2(v[12], v[13]),
                       cvt_bf16x2(v[14], v[15]));
            } else if (in) {
                float4* dst = reinterpret_cast<float4*>(part + 2 * SH::kRows + (long long)dense * D + c);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
            __syncwarp();
        }
        if (whole) {
            constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
            const int c = lane % kLanes;
#pragma unroll 4
            for (int i = 0; i < kLanes; ++i) {
                const int at_row = quarter * 32 + i * kAtOnce + lane / kLanes;
                const uint4 v = ld_shared_v4(stage + (c / 8) * (128 * 128) + at_row * 128 +
                                             (((c % 8) ^ (at_row % 8)) * 16));
                if (at_row < rows)
                    *(reinterpret_cast<uint4*>(
                          p.out + ((long long)(q->row0 + tok0 + at_row / heads) * p.Hq + q->head0 +
                                   at_row % heads) * D) + c) = v;
            }
            __syncwarp();
        }
        if (in) {
            if (whole) {
                if (p.lse) p.lse[to] = log_sum_of(mx, l);
            } else {
                part[2 * dense] = mx;
                part[2 * dense + 1] = l;
            }
        }
        list.done();
    }
}

// Of a call over shared prefixes `other` is the sequences' own part.
struct NoPart {};
template <int D, int G, class P, class Other>
__global__ void __launch_bounds__(kThreads, 1)
    kv_prefill_kernel(const __grid_constant__ P p, const __grid_constant__ Other other) {
    using SH = Shape<D, G>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared<D, G> sh;
    __shared__ std::conditional_t<P::kShared, Sums<kThreads>, NoPart> part_sums[2];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t qbuf = base, kbuf = qbuf + SH::kQBytes, vbuf = kbuf + SH::KB * SH::kOpBytes;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if constexpr (!P::kShared) pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPieceRing; ++i) {
            mbar_init(&sh.piece_full[i], 1);
            mbar_init(&sh.piece_empty[i], 5 * SH::MT + 8);
        }
        for (int i = 0; i < SH::KB; ++i) {
            mbar_init(&sh.k_full[i], 4);
            mbar_init(&sh.v_full[i], 4);
            mbar_init(&sh.k_empty[i], SH::MT);
            mbar_init(&sh.v_empty[i], SH::MT);
        }
        for (int i = 0; i < kMetaRing; ++i) mbar_init(&sh.v_known[i], 4);
        for (int i = 0; i < SH::MT; ++i) {
            mbar_init(&sh.q_full[i], 128);
            mbar_init(&sh.drained[i], 1);
        }
        for (int i = 0; i < 2 * SH::MT; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 128);  // (a warp may be a tile ahead of the others)
            mbar_init(&sh.pv_done[i], 1);
        }
        mbar_init_fence();
    }
    // what comes before the call is over, and holds no tensor memory any more
    if constexpr (P::kShared) pdl_wait();
    if (warp == 18) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    if constexpr (P::kShared) {
        // the sequences' own part may begin, once the last CTA has said on how many SMs this one is
        if (blockIdx.x != gridDim.x - 1) pdl_launch_dependents();
        sum_items(p, part_sums[0]);
        sum_items(other, part_sums[1]);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    SharedWalk walk;  // the listing warp's
    if constexpr (P::kShared) {
        if (warp == 18 || blockIdx.x == gridDim.x - 1) {
            Scan mine, theirs;
            scan_sums(part_sums[0], part_sums[1], mine, theirs);
            const long long all = all_units(p, mine);
            const int sms = share_of(all * p.unit_cost, all_units(other, theirs) * other.unit_cost, p.sms);
            const long long run = run_length(p, all, sms);
            if (blockIdx.x == gridDim.x - 1) {
                if (warp == 18) {
                    if (lane == 0) say_sms(p, sms);
                    __syncwarp();
                    pdl_launch_dependents();
                }
                write_before(p, part_sums[0], mine, run);
            }
            if (warp == 18) walk.start(p, part_sums[0], mine, run, blockIdx.x);
        }
    }

    bool ok = true;
    if (warp < 4 * SH::MT) {
        ok = softmax<D, G, P>(p, sh, qbuf, tmem, warp / 4, warp % 4, lane);
    } else if (warp >= 8 && warp < 16) {
        ok = Convert<D, G, P>(p, sh, warp - 8, lane).run(kbuf, vbuf);
    } else if (warp >= 16 && warp < 16 + SH::MT) {
        ok = issue_products<D, G, P>(p, sh, qbuf, kbuf, vbuf, tmem, warp - 16, lane);
        __syncwarp();
        // no instruction may still be running when the CTA lets its memory go
        if (elect_one()) umma_commit(&sh.drained[warp - 16]);
        __syncwarp();
        ok = warp_wait_sleep(&sh.drained[warp - 16], 0, kWaitBudgetCycles) && ok;
    } else if (warp == 18) {
        if constexpr (P::kShared) {
            if (lane == 0) ok = list_pieces<D, G>(p, sh, walk);
        } else if (lane == 0) {
            ok = list_pieces<D, G>(p, sh);
        }
    }
    if (!ok) flag_status(p.status, MXQ_DEV_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 18) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace
}  // namespace mxq
