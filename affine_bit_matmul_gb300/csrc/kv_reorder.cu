// Reordering of a paged cache after a selection of beams: sequence i of a group goes on from
// sequence parents[i] of it.
//
// Every column of the page table has as many pages as the group has sequences, its home
// pages.  A page that is full is shared by all who go on from it; the one that is being written
// and those after it stay with the lowest of them, and each other one takes the lowest home page
// of the column that nobody keeps, into which the tokens so far are copied.  There always is
// one: a column's pages that are kept are no more than those who keep one.  Pages that are
// copied to are read by nobody, so nothing has to wait for anything.
//   The first kernel takes a group: a warp a column, a lane a sequence, the home pages' use
// in a bit mask.  It writes the table, the lengths and a list of copies; a second kernel does
// those, for all layers and heads: whole slabs of 8 tokens, the four regions of a block (K
// codes, K pairs, V codes, V pairs) from their beginnings.
#include <cstdint>
#include <cuda_runtime.h>

#include "kv_format.cuh"
#include "mxq_internal.h"
#include "tc_common.cuh"

namespace mxq {
namespace {

constexpr int kTableThreads = 256;
constexpr int kCopyThreads = 128;

// A sequence's copy; tokens 0: none.
struct Move {
    int from, to, tokens, pad;
};

// NW: words of the masks of a group's sequences.
template <int NW>
__global__ void __launch_bounds__(kTableThreads) kv_table_kernel(const KvReorderParams p) {
    __shared__ int parent_of[32 * NW], len_of[32 * NW];
    __shared__ int bad;
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int W = p.W, C = p.max_pages, seq0 = blockIdx.x * W;
    const long long at0 = (long long)seq0 * C;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    if (threadIdx.x < W) {
        const int parent = __ldg(p.parents + seq0 + threadIdx.x);
        const bool in = (unsigned)parent < (unsigned)W;
        const int len = in ? p.lens[seq0 + parent] : 0;
        if (!in || len < 0 || len > C * p.page_size) bad = 1;
        parent_of[threadIdx.x] = parent;
        len_of[threadIdx.x] = len;
    }
    __syncthreads();
    Move* moves = static_cast<Move*>(p.moves) + seq0;
    if (bad) {
        // the group stays as it is
        if (threadIdx.x == 0) flag_status(p.status, MXQ_DEV_BAD_SEQUENCE);
        for (int i = threadIdx.x; i < W; i += kTableThreads) {
            moves[i].tokens = 0;
            p.lens_out[seq0 + i] = p.lens[seq0 + i];
        }
        for (long long i = threadIdx.x; i < (long long)W * C; i += kTableThreads)
            p.table_out[at0 + i] = p.table[at0 + i];
        return;
    }
    // this lane's sequences
    int parent[NW], len[NW];
    bool in[NW], lowest[NW];
#pragma unroll
    for (int u = 0; u < NW; ++u) {
        const int i = 32 * u + lane;
        in[u] = i < W;
        parent[u] = in[u] ? parent_of[i] : 0;
        len[u] = in[u] ? len_of[i] : 0;
        lowest[u] = in[u];
        for (int j = 0; j < W; ++j)
            if (j < i && parent_of[j] == parent[u]) lowest[u] = false;
    }
    for (int c = warp; c < C; c += kTableThreads / 32) {
        int home[NW], theirs[NW], mine[NW];
        bool full[NW], keeps[NW];
        uint32_t taken[NW] = {}, rest[NW];
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const long long row = at0 + (long long)(32 * u + lane) * C + c;
            home[u] = in[u] ? __ldg(p.home + row) : -1;
            theirs[u] = in[u] ? p.table[at0 + (long long)parent[u] * C + c] : -2;
            mine[u] = in[u] ? p.table[row] : -2;
            full[u] = in[u] && len[u] / p.page_size > c;
            keeps[u] = full[u] || lowest[u];
        }
        bool ok = true, given = false, used = false;
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            given = given || __any_sync(0xFFFFFFFFu, in[u] && home[u] >= 0);
            used = used || __any_sync(0xFFFFFFFFu, in[u] && len[u] > c * p.page_size);
        }
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, keeps[u]);
            for (uint32_t left = who; left; left &= left - 1) {
                const int page = __shfl_sync(0xFFFFFFFFu, theirs[u], __ffs(left) - 1);
                int found = 0;
#pragma unroll
                for (int h = 0; h < NW; ++h) {
                    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, in[h] && home[h] == page);
                    taken[h] |= hit;
                    found += __popc(hit);
                }
                ok = ok && found == 1;
            }
            rest[u] = __ballot_sync(0xFFFFFFFFu, in[u] && !keeps[u]);
        }
        // the n-th of those without a page takes the n-th page that nobody keeps
        int before = 0, free_pages = 0;
        int to[NW];
#pragma unroll
        for (int h = 0; h < NW; ++h) {
            const uint32_t all = W >= 32 * (h + 1) ? ~0u : W > 32 * h ? (1u << (W - 32 * h)) - 1u : 0u;
            taken[h] = ~taken[h] & all;  // free ones from here on
            free_pages += __popc(taken[h]);
        }
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            to[u] = theirs[u];
            int n = before + __popc(rest[u] & ((1u << lane) - 1u));
            before += __popc(rest[u]);
#pragma unroll
            for (int h = 0; h < NW; ++h) {
                const int here = __popc(taken[h]);
                const int pos = n >= 0 && n < here ? (int)__fns(taken[h], 0, n + 1) : 0;
                const int page = __shfl_sync(0xFFFFFFFFu, home[h], pos & 31);
                if (in[u] && !keeps[u] && n >= 0 && n < here) to[u] = page;
                n = n < here ? -1 : n - here;
            }
        }
        ok = ok && given && before <= free_pages;
        // (pages that nobody has been given yet and that hold no tokens are no fault)
        if (!ok && (given || used) && lane == 0) flag_status(p.status, MXQ_DEV_BAD_PAGE);
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            if (!in[u]) continue;
            // a column with other pages than the group's own stays as it is
            const int page = ok ? to[u] : mine[u];
            p.table_out[at0 + (long long)(32 * u + lane) * C + c] = page;
            const int at = min(len[u] / p.page_size, C - 1);  // (with C pages full nothing is copied)
            if (at != c) continue;
            Move m;
            m.from = theirs[u];
            m.to = page;
            m.pad = 0;
            const bool copy = ok && !keeps[u] && (unsigned)m.from < (unsigned)p.n_pages &&
                              (unsigned)m.to < (unsigned)p.n_pages;
            m.tokens = copy ? (len[u] % p.page_size + 7) / 8 * 8 : 0;
            if (ok && !keeps[u] && !copy) flag_status(p.status, MXQ_DEV_BAD_PAGE);
            moves[32 * u + lane] = m;
        }
    }
#pragma unroll
    for (int u = 0; u < NW; ++u)
        if (warp == 0 && in[u]) p.lens_out[seq0 + 32 * u + lane] = len[u];
}

// blockIdx.x: the sequence; blockIdx.y: its share of the layers' and heads' blocks.
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const KvReorderParams p, int D, int G) {
    pdl_wait();
    const int4 move = __ldcg(reinterpret_cast<const int4*>(p.moves) + blockIdx.x);
    const Move m{move.x, move.y, move.z, 0};
    if (m.tokens == 0) return;
    const int codes = kv_code_bytes(D, m.tokens) / 16, pairs = kv_pair_bytes(D, G, m.tokens) / 16;
    const int half = codes + pairs, all = 2 * half;
    const int codes_room = kv_code_bytes(D, p.page_size) / 16;
    const long long block = kv_block_bytes(D, G, p.page_size) / 16;
    uint4* pages = reinterpret_cast<uint4*>(p.pages);
    const int blocks = p.layers * p.H;
    for (int b = blockIdx.y; b < blocks; b += gridDim.y) {
        const long long page0 = (long long)(b / p.H) * p.n_pages;
        const uint4* from = pages + ((page0 + m.from) * p.H + b % p.H) * block;
        uint4* to = pages + ((page0 + m.to) * p.H + b % p.H) * block;
        for (int i = threadIdx.x; i < all; i += kCopyThreads) {
            const int j = i < half ? i : i - half;
            const long long at = (i < half ? 0 : block / 2) + (j < codes ? j : codes_room + j - codes);
            to[at] = from[at];
        }
    }
}

}  // namespace

size_t kv_reorder_move_bytes() { return sizeof(Move); }

cudaError_t launch_kv_reorder(const KvReorderParams& p, int D, int G, cudaStream_t stream) {
    if (p.W <= 32)
        kv_table_kernel<1><<<(unsigned)(p.S / p.W), kTableThreads, 0, stream>>>(p);
    else
        kv_table_kernel<2><<<(unsigned)(p.S / p.W), kTableThreads, 0, stream>>>(p);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    // the second kernel's blocks are placed while the first one finishes
    cudaLaunchConfig_t cfg = {};
    const long long blocks = (long long)p.layers * p.H;
    cfg.gridDim = dim3((unsigned)p.S, (unsigned)(blocks < 65535 ? blocks : 65535));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_copy_kernel, p, D, G);
}

}  // namespace mxq
