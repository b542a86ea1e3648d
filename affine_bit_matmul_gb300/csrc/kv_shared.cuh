// Attention over shared prefixes: what the two parts of a call, the groups' rows over
// their prefixes and the sequences' rows over their own tokens, are made of, and how they are cut.
//
// A part is a list of items (groups or sequences).  For each key/value head an item's (token, query
// head) rows, in order, are cut into `planes` row tiles of equal size, all of which go over all of its
// tokens; the units of a part (row tile, tile of tokens) are cut into runs of equal length, one
// for each runner (a CTA on the tensor cores, else a warp), as in the calls without a prefix.  Row tiles
// are numbered in the order of the runs, so a runner's piece of row tile n has a place of its own at
// n + runner: both numbers never decrease along the units, and one of them grows from piece to
// piece.  The joining kernel finds a row's pieces from what comes before its item alone.
//   The parts run beside each other, and what each may have of the GPU goes by their costs, from
// the lengths, which only the device knows: every CTA works it out by itself, but for those beside the tensor
// cores' kernel, whose last CTA says so before they start.
#pragma once

#include "kv_attn_common.cuh"

namespace mxq {

// What the joining kernel has to know of an item (workspace).
struct Before {
    int units, planes;  // of one head, before it
    int row0, rows, len, item_planes;
    int group;          // a sequence's; -1: none
    int pad;
};

namespace {

// (What a call reads may be written while its first kernel's blocks are placed: plain loads, not those for what
// stays as it is.)
struct Item {
    int row0, rows;  // of q
    int len;         // tokens
    int planes;      // row tiles for one head; 0: nothing to do
    int bad;         // its arguments are out of range
};

__host__ __device__ __forceinline__ int items_of(const KvSharedParams& p) {
    return p.prefix ? p.groups_n : p.S;
}

// Sequences of group g, [*a, *b).
__host__ __device__ __forceinline__ void group_of(const KvGroupParams& p, int g, int* a, int* b) {
    if (p.groups) {
        *a = *(p.groups + g);
        *b = *(p.groups + g + 1);
    } else {
        const int each = p.S / p.groups_n;
        *a = g * each;
        *b = *a + each;
    }
}

// (`prefix`: a group, with its prefix in pages of a table of `width`, or a sequence)
__host__ __device__ __forceinline__ Item item_of(const KvGroupParams& p, int i, bool prefix, int width) {
    Item r;
    int a = i, b = i + 1, most = p.max_q, len;
    r.bad = 0;
    if (prefix) {
        group_of(p, i, &a, &b);
        if (a < 0 || b > p.S || a > b || b - a > p.max_group) {
            r.bad = 1;
            a = b = 0;
        }
        most = (int)min((long long)p.max_group * p.max_q, (long long)p.T);
        len = *(p.prefix_lens + i);
    } else {
        len = *(p.ctx_lens + i);
    }
    if (p.q_starts) {
        a = *(p.q_starts + a);
        b = *(p.q_starts + b);
    }
    if (a < 0 || b > p.T || a > b || b - a > most) {
        r.bad = 1;
        a = b = 0;  // none of its rows
    }
    const int room = width * p.page_size;
    if (len < 0 || len > room) {
        r.bad = 1;
        len = min(max(len, 0), room);
    }
    r.row0 = a;
    r.rows = b - a;
    r.len = len;
    r.planes = len > 0 ? (r.rows * p.part_heads + p.tile_rows - 1) / p.tile_rows : 0;
    return r;
}

__host__ __device__ __forceinline__ Item item_of(const KvSharedParams& p, int i) {
    return item_of(p, i, p.prefix, p.max_pages);
}
__host__ __device__ __forceinline__ Item item_of(const KvTwoParams& p, int g) {
    return item_of(p, g, true, p.max_prefix_pages);
}

__host__ __device__ __forceinline__ int tiles_of(const KvSharedParams& p, const Item& it) {
    return (it.len + (1 << p.tile_shift) - 1) >> p.tile_shift;
}
// Units of an item's row tiles for one head: their tiles, and what the end of each costs.
__host__ __device__ __forceinline__ int units_of(const KvSharedParams& p, const Item& it) {
    return it.planes * (tiles_of(p, it) + p.end_units);
}

// The group that sequence s belongs to, or -1.
__device__ __forceinline__ int group_with(const KvGroupParams& p, int s) {
    if (!p.groups) return s / (p.S / p.groups_n);
    int lo = 0, hi = p.groups_n - 1;  // the last group that starts at or before s
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (*(p.groups + mid) <= s) lo = mid;
        else hi = mid - 1;
    }
    return *(p.groups + lo) <= s && s < *(p.groups + lo + 1) ? lo : -1;
}

// The units of a part, summed up by a block of T threads: each thread's consecutive items.
template <int T>
struct Sums {
    int units[T], planes[T];
};

// Starts that decrease let items overlap: their row tiles may then be any number.  A thread's count stops at one more
// than there are places for, so that the sum of all, at most kKvListThreads times that (countable), tells; the units,
// which may have lost their highest bits, are not used then.
template <int T>
__device__ __forceinline__ void sum_items(const KvSharedParams& p, Sums<T>& s) {
    static_assert(T <= kKvListThreads);
    const int n = items_of(p), per = (n + T - 1) / T;
    unsigned units = 0;
    long long planes = 0;
#pragma unroll 4
    for (int i = threadIdx.x * per; i < min(((int)threadIdx.x + 1) * per, n); ++i) {
        const Item it = item_of(p, i);
        units += (unsigned)units_of(p, it);
        planes += it.planes;
        if (it.bad && blockIdx.x == 0) flag_status(p.status, MXQ_DEV_BAD_SEQUENCE);
    }
    s.units[threadIdx.x] = (int)units;
    s.planes[threadIdx.x] = (int)min(planes, p.max_planes + 1LL);
}

// The same for a warp, each lane with T / 32 threads' items: up to and with its own, and all.  Units in the
// high word, row tiles in the low one (both fit 31 bits).
struct Scan {
    long long mine, upto, all;
    __device__ int units() const { return (int)(all >> 32); }
    __device__ int planes() const { return (int)all; }
    __device__ int units_before() const { return (int)((upto - mine) >> 32); }
    __device__ int units_upto() const { return (int)(upto >> 32); }
    __device__ int planes_before() const { return (int)(upto - mine); }
};

template <int T>
__device__ __forceinline__ void scan_sums(const Sums<T>& s, const Sums<T>& t, Scan& x, Scan& y) {
    const int lane = threadIdx.x & 31;
    x.mine = y.mine = 0;
#pragma unroll 4
    for (int i = 0; i < T / 32; ++i) {
        x.mine += (long long)s.units[lane * (T / 32) + i] << 32 | (unsigned)s.planes[lane * (T / 32) + i];
        y.mine += (long long)t.units[lane * (T / 32) + i] << 32 | (unsigned)t.planes[lane * (T / 32) + i];
    }
    x.upto = x.mine;
    y.upto = y.mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, x.upto, o), v = __shfl_up_sync(0xFFFFFFFFu, y.upto, o);
        if (lane >= o) {
            x.upto += u;
            y.upto += v;
        }
    }
    x.all = __shfl_sync(0xFFFFFFFFu, x.upto, 31);
    y.all = __shfl_sync(0xFFFFFFFFu, y.upto, 31);
}

// Items that overlap can make more row tiles than there are places for: nothing is done, and the joining kernel finds
// all items without rows.
__device__ __forceinline__ bool too_many(const KvSharedParams& p, const Scan& s) { return s.planes() > p.max_planes; }

__device__ __forceinline__ long long all_units(const KvSharedParams& p, const Scan& s) {
    return too_many(p, s) ? 0 : (long long)s.units() * (p.Hkv * p.head_parts);
}

// On how many SMs the tensor cores' part is: said by one thread of that kernel with the call's number (SMs are
// fewer than 256), in one word, so that who finds the number has the SMs, and with a fence (heard) all that was there when
// they were said, the call's arguments among it.  The joining kernel takes the word back: a graph's next replay has
// the same number.
__device__ __forceinline__ void say_sms(const KvSharedParams& p, int sms) {
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p.totals + 1), "l"(p.call | (unsigned)sms) : "memory");
}
// The same, read in the kernel beside it; where the number is another's, once that kernel is over.
__device__ __forceinline__ int said_sms(const KvSharedParams& p) {
    unsigned long long x;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(x) : "l"(p.totals + 1) : "memory");
    if ((x ^ p.call) >> 8) {
        pdl_wait();
        x = (unsigned long long)__ldcg(p.totals + 1);
    }
    return (int)(x & 255u);
}
__device__ __forceinline__ void heard() { __threadfence(); }

// How many of `all` runners (or SMs) the first of two parts gets, by their costs.
__device__ __forceinline__ int share_of(long long cost1, long long cost2, int all) {
    if (cost1 == 0) return 0;
    if (cost2 == 0) return all;
    const int n = (int)(__fdividef((float)cost1, (float)cost1 + (float)cost2) * all + 0.5f);
    return min(max(n, 1), all - 1);
}

// Units of a run of `runners`, at least the part's least.
__device__ __forceinline__ long long run_length(const KvSharedParams& p, long long all, int runners) {
    if (all == 0 || runners <= 0) return 0;
    // (most often it fits 32 bits, and the division is short)
    const long long up = all + runners - 1;
    const long long n = up >> 32 ? up / runners : (long long)((unsigned)up / (unsigned)runners);
    return n > p.least_run ? n : p.least_run;
}

// What the joining kernel needs, by one block.
template <int T>
__device__ void write_before(const KvSharedParams& p, const Sums<T>& s, const Scan& scan, long long run) {
    const int n = items_of(p), per = (n + T - 1) / T, from = threadIdx.x / (T / 32);
    const bool left_out = too_many(p, scan);
    if (threadIdx.x == 0) {
        p.totals[0] = run;
        if (left_out) flag_status(p.status, MXQ_DEV_BAD_SEQUENCE);
    }
    // (every warp holds the whole scan)
    int u = __shfl_sync(0xFFFFFFFFu, scan.units_before(), from);
    int t = __shfl_sync(0xFFFFFFFFu, scan.planes_before(), from);
    for (int i = from * (T / 32); i < (int)threadIdx.x; ++i) {
        u += s.units[i];
        t += s.planes[i];
    }
    for (int i = threadIdx.x * per; i < min(((int)threadIdx.x + 1) * per, n); ++i) {
        const Item it = item_of(p, i);
        Before b;
        b.units = u;
        b.planes = t;
        b.row0 = it.row0;
        b.rows = left_out ? 0 : it.rows;
        b.len = it.len;
        b.item_planes = left_out ? 0 : it.planes;
        b.group = p.prefix ? i : group_with(p, i);
        b.pad = 0;
        p.before[i] = b;
        u += units_of(p, it);
        t += it.planes;
    }
}

// A run's pieces: units k0 .. k0 + count - 1 of row tile (item, vh, plane), number `tile`.
struct SharedPiece {
    int item, vh, plane, k0, count, tile;
    Item it;
    // find_rows: its key/value head, query heads, rows (one at least) and the first of them in the item, position of
    // the last row, which sees most
    int h, head0, heads, flat0, rows, p1;
};

// The query heads of head part vh.
__host__ __device__ __forceinline__ int heads_of(const KvSharedParams& p, int vh) {
    return min(p.part_heads, p.Hq / p.Hkv - vh % p.head_parts * p.part_heads);
}

// What follows from a piece's numbers.
__host__ __device__ __forceinline__ void find_rows(const KvSharedParams& p, SharedPiece& q) {
    const int rep = p.Hq / p.Hkv, part = q.vh % p.head_parts;
    q.h = q.vh / p.head_parts;
    q.heads = heads_of(p, q.vh);
    q.head0 = q.h * rep + part * p.part_heads;
    q.flat0 = q.plane * p.tile_rows;
    q.rows = min(p.tile_rows, q.it.rows * q.heads - q.flat0);
    q.p1 = p.prefix ? q.it.len - 1 : q.it.len - q.it.rows + (q.flat0 + q.rows - 1) / q.heads;
}

struct SharedWalk {
    int i, vh, plane, k, tile, tiles;
    long long left;
    Item it;

    __host__ __device__ void load(const KvSharedParams& p, int item) {
        i = item;
        it = item_of(p, i);
        tiles = tiles_of(p, it);
    }
    // Run `runner` of length `run`, by a whole warp.
    template <int T>
    __device__ void start(const KvSharedParams& p, const Sums<T>& s, const Scan& scan, long long run, int runner) {
        const int vheads = p.Hkv * p.head_parts;
        const long long all = all_units(p, scan), u0 = runner * run;
        left = run == 0 || u0 >= all ? 0 : (all - u0 < run ? all - u0 : run);
        if (left == 0) return;
        const uint32_t here = __ballot_sync(0xFFFFFFFFu, u0 >= (long long)scan.units_before() * vheads &&
                                                             u0 < (long long)scan.units_upto() * vheads);
        const int owner = __ffs(here) - 1;
        long long at = u0 - (long long)__shfl_sync(0xFFFFFFFFu, scan.units_before(), owner) * vheads;
        tile = __shfl_sync(0xFFFFFFFFu, scan.planes_before(), owner) * vheads;
        int t = owner * (T / 32);  // the thread whose items the run starts in
        while (at >= (long long)s.units[t] * vheads) {
            tile += s.planes[t] * vheads;
            at -= (long long)s.units[t++] * vheads;
        }
        load(p, t * ((items_of(p) + T - 1) / T));
        while (at >= (long long)units_of(p, it) * vheads) {
            at -= (long long)units_of(p, it) * vheads;
            tile += it.planes * vheads;
            load(p, i + 1);
        }
        // (an item's units of one head fit 32 bits, those of all heads may not)
        const int each = tiles + p.end_units;
        const int n = at >> 32 ? (int)(at / each) : (int)((unsigned)at / (unsigned)each);
        k = (int)(at - (long long)n * each);
        vh = n / it.planes;
        plane = n - vh * it.planes;
        tile += n;
    }
    // An item has the planes that its largest head part fills: where the heads do not divide evenly, the last ones
    // of a smaller part may have no rows.  They count (units, numbers), but are no pieces.  False, and a count of 0, when
    // the run is over.
    __host__ __device__ bool next(const KvSharedParams& p, SharedPiece* out) {
        while (left > 0) {
            while (it.planes == 0) load(p, i + 1);
            const int all = tiles + p.end_units, n = (int)(left < all - k ? left : all - k);
            const int here = min(k + n, tiles) - k;  // the others are the row tile's end
            if (here > 0) {
                out->item = i;
                out->vh = vh;
                out->plane = plane;
                out->k0 = k;
                out->count = here;
                out->tile = tile;
                out->it = it;
            }
            left -= n;
            k += n;
            if (k == all && left > 0) {
                k = 0;
                ++tile;
                if (++plane == it.planes) {
                    plane = 0;
                    if (++vh == p.Hkv * p.head_parts) {
                        vh = 0;
                        load(p, i + 1);
                    }
                }
            }
            if (here > 0 && out->plane * p.tile_rows < out->it.rows * heads_of(p, out->vh)) return true;
        }
        out->count = 0;
        return false;
    }
};

}  // namespace
}  // namespace mxq
