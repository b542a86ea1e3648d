// Attention over shared prefixes: what the two parts of a call, the groups' rows over
// their prefixes and the sequences' rows over their own tokens, are made of.
//
// A part is a list of items (groups or sequences).  An item's rows are cut into `planes` row
// tiles for each key/value head, all of which go over all of its tokens; the units of a
// part (row tile, tile of tokens) are cut into runs of equal length, one for each CTA, as in
// the calls without a prefix.  Row tiles are numbered in the order of the runs, so a CTA's
// piece of row tile n has a place of its own at n + CTA: both numbers never decrease along
// the units, and one of them grows from piece to piece.  The joining kernel finds a row's
// pieces from the numbers of units and row tiles before its item alone.
#pragma once

#include "kv_attn_common.cuh"

namespace mxq {
namespace {

struct Item {
    int row0, rows;  // of q
    int len;         // tokens
    int planes;      // row tiles for one head; 0: nothing to do
    int bad;         // its arguments are out of range
};

__device__ __forceinline__ int items_of(const KvAttnParams&) { return 0; }
__device__ __forceinline__ int items_of(const KvSharedParams& p) {
    return p.prefix ? p.groups_n : p.S;
}

// Units of a run: equal runs for all CTAs, the last of them shorter.
__device__ __forceinline__ long long run_length(long long all, int ctas) {
    return (all + ctas - 1) / ctas;
}

// Sequences of group g, [*a, *b).
__device__ __forceinline__ void group_of(const KvSharedParams& p, int g, int* a, int* b) {
    if (p.groups) {
        *a = __ldg(p.groups + g);
        *b = __ldg(p.groups + g + 1);
    } else {
        const int each = p.S / p.groups_n;
        *a = g * each;
        *b = *a + each;
    }
}

__device__ __forceinline__ Item item_of(const KvSharedParams& p, int i) {
    Item r;
    int a = i, b = i + 1, most = p.max_q, len;
    r.bad = 0;
    if (p.prefix) {
        group_of(p, i, &a, &b);
        if (a < 0 || b > p.S || a > b || b - a > p.max_group) {
            r.bad = 1;
            a = b = 0;
        }
        most = (int)min((long long)p.max_group * p.max_q, (long long)p.T);
        len = __ldg(p.prefix_lens + i);
    } else {
        len = __ldg(p.ctx_lens + i);
    }
    if (p.q_starts) {
        a = __ldg(p.q_starts + a);
        b = __ldg(p.q_starts + b);
    }
    if (a < 0 || b > p.T || a > b || b - a > most) {
        r.bad = 1;
        a = b = 0;  // none of its rows
    }
    const int room = p.max_pages * p.page_size;
    if (len < 0 || len > room) {
        r.bad = 1;
        len = min(max(len, 0), room);
    }
    r.row0 = a;
    r.rows = b - a;
    r.len = len;
    r.planes = len > 0 ? (r.rows + p.tile_toks - 1) / p.tile_toks : 0;
    return r;
}

}  // namespace
}  // namespace mxq
