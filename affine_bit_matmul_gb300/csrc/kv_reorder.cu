// Reordering of a paged cache after a selection of beams: sequence i of a group goes on from
// sequence parents[i] of it.
//
// Every column of the page table has as many pages as the group has sequences, its home
// pages.  A page that is full is shared by all who go on from it; the one that is being written
// and those after it stay with the lowest of them, and each other one takes the lowest home page
// of the column that nobody keeps, into which the tokens so far are copied.  There always is
// one: a column's pages that are kept are no more than those who keep one.  Pages that are
// copied to are read by nobody, so nothing has to wait for anything.
//   A block takes a group's table: a warp a column, a lane a sequence, the home pages' use in a bit
// mask.  Other blocks take the copies of one sequence, for some of the layers and heads: whole
// slabs of 8 tokens, the four regions of a block (K codes, K pairs, V codes, V pairs) from their
// beginnings.  They work out the one column that they need by themselves, unless the table is
// written in place: then they run after it, from a list.
//   Copies are bound by the memory, small calls by a chain of loads (parents, lengths, table, pages).
//   16 groups of 8 over 16 layers, 26 MB read and as many written: 19.8 us with 4 pieces of 16 bytes of a thread in
// flight (20.7 with 2, 22.5 with 8; 22.9 in blocks of 512 threads, 20.8 of 128), 3 of them the chain; 1 group of 4: 4.1 us.
#include <cstdint>
#include <cuda_runtime.h>

#include "kv_format.cuh"
#include "mxq_internal.h"
#include "tc_common.cuh"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kSms = 152;
constexpr long long kMostBlocks = 500000;  // of a share: up to 2560 pieces of 16 bytes each, 32 bits

// A sequence's copy; tokens 0: none.
struct Move {
    int from, to, tokens, pad;
};

// NW: words of the masks of a group's sequences.
template <int NW>
struct Group {
    int parent[32 * NW], len[32 * NW];
    int bad;
};

// The group's parents and its sequences' lengths as they go on; the whole block.  False if
// something is out of range.
template <int NW>
__device__ __forceinline__ bool load_group(const KvReorderParams& p, int seq0, Group<NW>& g) {
    const int i = threadIdx.x;
    if (i == 0) g.bad = 0;
    __syncthreads();
    if (i < p.W) {
        const int parent = __ldg(p.parents + seq0 + i);
        const bool in = (unsigned)parent < (unsigned)p.W;
        const int len = in ? p.lens[seq0 + parent] : 0;
        if (!in || len < 0 || len > p.max_pages * p.page_size) g.bad = 1;
        g.parent[i] = parent;
        g.len[i] = len;
    }
    __syncthreads();
    return !g.bad;
}

// A lane's sequences (32 u + lane), and what a column of the table comes to be for them.
template <int NW>
struct Column {
    int theirs[NW], mine[NW], to[NW];  // the parent's page, the present one, the new one
    bool in[NW], lowest[NW], keeps[NW];
    bool ok, given, used;  // the pages are the group's own; it has pages there; tokens are there

    // the lowest of those who go on from the same sequence
    __device__ __forceinline__ void start(const KvReorderParams& p, const Group<NW>& g) {
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const int i = 32 * u + (threadIdx.x & 31);
            in[u] = lowest[u] = i < p.W;
            for (int j = 0; j < p.W; ++j)
                if (in[u] && j < i && g.parent[j] == g.parent[i]) lowest[u] = false;
        }
    }
    __device__ __forceinline__ void work_out(const KvReorderParams& p, const Group<NW>& g, long long at0, int c) {
        const int lane = threadIdx.x & 31, C = p.max_pages;
        int home[NW];
        uint32_t taken[NW] = {}, rest[NW];
        ok = true;
        given = used = false;
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const int i = 32 * u + lane;
            const long long row = at0 + (long long)i * C + c;
            const int len = in[u] ? g.len[i] : 0;
            home[u] = in[u] ? __ldg(p.home + row) : -1;
            theirs[u] = in[u] ? p.table[at0 + (long long)g.parent[i] * C + c] : -2;
            mine[u] = in[u] ? p.table[row] : -2;
            keeps[u] = in[u] && (len / p.page_size > c || lowest[u]);
            given = given || __any_sync(0xFFFFFFFFu, in[u] && home[u] >= 0);
            used = used || __any_sync(0xFFFFFFFFu, in[u] && len > c * p.page_size);
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
#pragma unroll
        for (int h = 0; h < NW; ++h) {
            const uint32_t all = p.W >= 32 * (h + 1) ? ~0u : p.W > 32 * h ? (1u << (p.W - 32 * h)) - 1u : 0u;
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
    }
    // what is copied for sequence 32 u + lane in this column
    __device__ __forceinline__ Move move(const KvReorderParams& p, int u, int len) const {
        Move m{theirs[u], to[u], 0, 0};
        if (ok && in[u] && !keeps[u] && (unsigned)m.from < (unsigned)p.n_pages && (unsigned)m.to < (unsigned)p.n_pages)
            m.tokens = (len % p.page_size + 7) / 8 * 8;
        return m;
    }
};

template <int NW>
__device__ __forceinline__ void write_table(const KvReorderParams& p, int group, Group<NW>& g) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int W = p.W, C = p.max_pages, seq0 = group * W;
    const long long at0 = (long long)seq0 * C;
    Move* moves = p.moves ? static_cast<Move*>(p.moves) + seq0 : nullptr;
    if (!load_group(p, seq0, g)) {
        // the group stays as it is
        if (threadIdx.x == 0) flag_status(p.status, MXQ_DEV_BAD_SEQUENCE);
        for (int i = threadIdx.x; i < W; i += kThreads) {
            if (moves) moves[i].tokens = 0;
            p.lens_out[seq0 + i] = p.lens[seq0 + i];
        }
        for (long long i = threadIdx.x; i < (long long)W * C; i += kThreads)
            p.table_out[at0 + i] = p.table[at0 + i];
        return;
    }
    Column<NW> col;
    col.start(p, g);
    for (int c = warp; c < C; c += kThreads / 32) {
        col.work_out(p, g, at0, c);
        // (pages that nobody has been given yet and that hold no tokens are no fault)
        if (!col.ok && (col.given || col.used) && lane == 0) flag_status(p.status, MXQ_DEV_BAD_PAGE);
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            if (!col.in[u]) continue;
            const int i = 32 * u + lane, len = g.len[i];
            // a column with other pages than the group's own stays as it is
            p.table_out[at0 + (long long)i * C + c] = col.ok ? col.to[u] : col.mine[u];
            if (min(len / p.page_size, C - 1) != c) continue;  // (with C pages full nothing is copied)
            const Move m = col.move(p, u, len);
            if (col.ok && !col.keeps[u] && m.tokens == 0 && len % p.page_size) flag_status(p.status, MXQ_DEV_BAD_PAGE);
            if (moves) moves[i] = m;
        }
    }
    for (int i = threadIdx.x; i < W; i += kThreads) p.lens_out[seq0 + i] = g.len[i];
}

// A share (of `shares`) of a move's blocks, four 16-byte pieces of a thread at a time.
__device__ __forceinline__ void copy_tokens(const KvReorderParams& p, int D, int G, const Move& m, int share, int shares) {
    const int codes = kv_code_bytes(D, m.tokens) / 16, half = codes + kv_pair_bytes(D, G, m.tokens) / 16;
    const int codes_room = kv_code_bytes(D, p.page_size) / 16;
    const long long block = kv_block_bytes(D, G, p.page_size) / 16;
    uint4* pages = reinterpret_cast<uint4*>(p.pages);
    const int blocks = p.layers * p.H, b0 = (int)((long long)blocks * share / shares);
    const int b1 = (int)((long long)blocks * (share + 1) / shares);
    const unsigned all = (unsigned)(b1 - b0) * (2u * half);  // (kMostBlocks)
    constexpr int kAtOnce = 4;
    for (unsigned i0 = threadIdx.x; i0 < all; i0 += kThreads * kAtOnce) {
        uint4 x[kAtOnce];
        uint4* to[kAtOnce];
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n) {
            const unsigned i = i0 + n * kThreads;
            to[n] = nullptr;
            if (i >= all) continue;
            const unsigned q = i / (2u * half);
            const int k = (int)(i - q * (2u * half)), j = k < half ? k : k - half;
            const unsigned b = b0 + q, layer = b / (unsigned)p.H, h = b - layer * p.H;
            const long long at = (k < half ? 0 : block / 2) + (j < codes ? j : codes_room + j - codes);
            uint4* src = pages + (((long long)layer * p.n_pages + m.from) * p.H + h) * block + at;
            x[n] = *src;
            to[n] = src + (long long)(m.to - m.from) * p.H * block;
        }
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n)
            if (to[n]) *to[n] = x[n];
    }
}

// The first blocks take the groups' tables; without a list (p.moves) the others take a sequence's
// copies each, `shares` of them a sequence.
template <int NW>
__global__ void __launch_bounds__(kThreads) kv_reorder_kernel(const KvReorderParams p, int D, int G, int shares) {
    __shared__ Group<NW> g;
    __shared__ Move move;
    if (p.moves) pdl_launch_dependents();
    const int groups = p.S / p.W;
    if ((int)blockIdx.x < groups) {
        write_table(p, blockIdx.x, g);
        return;
    }
    const int n = blockIdx.x - groups, s = n / shares, seq0 = s / p.W * p.W, i = s - seq0;
    if (!load_group(p, seq0, g)) return;
    const int c = g.len[i] / p.page_size;
    // the lowest of those who go on from the same sequence keeps the page
    bool lowest = true;
    for (int j = 0; j < i; ++j) lowest = lowest && g.parent[j] != g.parent[i];
    if (lowest || g.len[i] % p.page_size == 0) return;
    if (threadIdx.x < 32) {
        Column<NW> col;
        col.start(p, g);
        col.work_out(p, g, (long long)seq0 * p.max_pages, c);
#pragma unroll
        for (int u = 0; u < NW; ++u)
            if (32 * u + (int)threadIdx.x == i) move = col.move(p, u, g.len[i]);
    }
    __syncthreads();
    if (move.tokens) copy_tokens(p, D, G, move, n - s * shares, shares);
}

// blockIdx.x: the sequence; blockIdx.y: its share of the layers' and heads' blocks.
__global__ void __launch_bounds__(kThreads) kv_copy_kernel(const KvReorderParams p, int D, int G) {
    pdl_wait();
    const int4 x = __ldcg(reinterpret_cast<const int4*>(p.moves) + blockIdx.x);
    const Move m{x.x, x.y, x.z, 0};
    if (m.tokens) copy_tokens(p, D, G, m, blockIdx.y, gridDim.y);
}

}  // namespace

size_t kv_reorder_move_bytes() { return sizeof(Move); }

cudaError_t launch_kv_reorder(KvReorderParams p, int D, int G, cudaStream_t stream) {
    // Blocks for a sequence's copies: with a third of the sequences copied as where parents are drawn
    // at random, some for each SM.
    const long long blocks = (long long)p.layers * p.H;
    long long shares = (12LL * kSms - 1) / p.S + 1;
    if (shares > blocks) shares = blocks;
    if (shares < blocks / kMostBlocks + 1) shares = blocks / kMostBlocks + 1;
    const int groups = p.S / p.W;
    const bool in_place = p.table_out == p.table || p.lens_out == p.lens;
    if (!in_place) p.moves = nullptr;
    const long long grid = in_place ? groups : groups + p.S * shares;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (p.W <= 32)
        kv_reorder_kernel<1><<<(unsigned)grid, kThreads, 0, stream>>>(p, D, G, (int)shares);
    else
        kv_reorder_kernel<2><<<(unsigned)grid, kThreads, 0, stream>>>(p, D, G, (int)shares);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !in_place) return err;
    // the second kernel's blocks are placed while the first one finishes
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.S, (unsigned)shares);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_copy_kernel, p, D, G);
}

}  // namespace mxq
