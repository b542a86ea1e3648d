// Attention of a few query rows over a paged 4-bit key/value cache by warps on their own, for
// the parts of a call over shared prefixes: a run of a warp (kv_shared.cuh) is a few hundred tokens.
//
// The mathematics is kv_attention.cu's: codes as f16 subnormals in m16n8k16, scales and biases in
// fp32, the running maximum moved only when a score exceeds it by 2^8, sums centred every 512
// tokens.  What differs is where the codes come from and where the result goes: a lane's operands of 8
// tokens are 16 bytes of the page, so they are loaded from memory into registers, the values'
// while the scores are made, the next tile's keys while the values are added up, and a piece of a row
// tile leaves its (largest score, sum, weighted sum) in the workspace as it is.  No warp waits for
// another, and nothing is shared but the list of items.  Where contexts are short, the ends of row
// tiles are most of the work, and they cost a few stores here.
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

// Row tiles of 4 KT rows.
template <int D, int G, int KT>
struct Lone {
    static constexpr int kRows = 4 * KT;
    static constexpr int kColumns = (KT + 1) / 2;  // tiles of 8 columns
    static constexpr int kSub = KT == 4 || D == 256 ? 1 : 2;  // 16 tokens, so many times a tile
    static constexpr int kTile = 16 * kSub;
    static constexpr int kShift = kSub == 1 ? 4 : 5;
    // the queries lie in shared memory where they would take 32 registers or more
    static constexpr bool kQueryShared = D * kColumns >= 256;
    static constexpr int kQueryBytes = kQueryShared ? kColumns * D * 16 : 0;  // of a warp
    // CTAs of an SM, by the registers of a thread: 168, 255
    static constexpr int kCtas = D == 256 && KT == 4 ? 2 : 3;
};

// 16 tokens' codes and pairs of the keys or of the values, as a lane has them: tokens r and r + 8.
template <int D, int G>
struct Codes {
    uint32_t w0[D / 32], w1[D / 32], pr0[D / G], pr1[D / G];

    __device__ __forceinline__ void none() {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w0[i] = w1[i] = 0u;
#pragma unroll
        for (int i = 0; i < D / G; ++i) pr0[i] = pr1[i] = 0u;
    }
    // from a page's keys or values at `src`, from token `skip` of the page on
    __device__ __forceinline__ void load(const uint8_t* src, int page, int skip, int lane) {
        const uint8_t* codes = src + kv_code_bytes(D, skip) + lane * (D == 64 ? 8 : 16);
        load_words<D / 32>(codes, w0);
        load_words<D / 32>(codes + 4 * D, w1);
        const uint8_t* pairs = src + kv_code_bytes(D, page) + (skip + (lane >> 2)) * (D / G * 4);
        load_pairs<D / G>(pairs, pr0);
        load_pairs<D / G>(pairs + 8 * (D / G * 4), pr1);
    }
};

// A warp's pieces of the run.
template <int D, int G, int KT>
__device__ __forceinline__ void lone_run(const KvSharedParams& p, SharedWalk& walk, int runner, uint4* queries) {
    using LN = Lone<D, G, KT>;
    constexpr int NG = D / G, U = D / 32, MT = D / 16, VT = LN::kColumns, SUB = LN::kSub, TILE = LN::kTile;
    const int lane = threadIdx.x & 31, r = lane >> 2, i4 = lane & 3;
    const int rep = p.Hq / p.Hkv;
    const long long block = kv_block_bytes(D, G, p.page_size);
    SharedPiece pc;
    while (walk.next(p, &pc)) {
        const int h = pc.vh / p.head_parts, part = pc.vh - h * p.head_parts;
        const int head0 = h * rep + part * p.part_heads, heads = min(p.part_heads, rep - part * p.part_heads);
        const int flat0 = pc.plane * LN::kRows, rows = min(LN::kRows, pc.it.rows * heads - flat0);
        if (rows <= 0) continue;  // (a part with fewer heads than the first)
        // positions of the first and of the last row: the tokens that they see
        const int p0 = p.prefix ? pc.it.len - 1 : pc.it.len - pc.it.rows + flat0 / heads;
        const int p1 = p.prefix ? pc.it.len - 1 : pc.it.len - pc.it.rows + (flat0 + rows - 1) / heads;
        auto position = [&](int kt) {
            const int row = kt * 4 + i4;
            return row < rows ? (p.prefix ? p0 : pc.it.len - pc.it.rows + (flat0 + row) / heads) : -1;
        };
        const int32_t* table = p.table + (long long)pc.item * p.max_pages;
        const uint8_t* pages = p.pages + (long long)h * block;
        const int end = pc.k0 + pc.count;

        // ---- pages of a tile's halves, and their loads
        auto look = [&](int (&id)[SUB], int k) {
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
                const int t = k * TILE + 16 * b;
                id[b] = k < end && t <= p1 ? __ldg(table + (t >> p.page_shift)) : -2;  // -2: not needed
            }
        };
        auto exists = [&](int id) { return (unsigned)id < (unsigned)p.n_pages; };
        Codes<D, G> kc[SUB], vc[SUB];
        auto load = [&](Codes<D, G>& c, int id, int t, long long half) {
            if (exists(id))
                c.load(pages + (long long)id * p.Hkv * block + half, p.page_size, t & (p.page_size - 1), lane);
            else
                c.none();
        };
        int id[SUB], next_id[SUB];
        look(id, pc.k0);
#pragma unroll
        for (int b = 0; b < SUB; ++b) load(kc[b], id[b], pc.k0 * TILE + 16 * b, 0);

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
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
            const int rr = vt * 8 + (r >> 1) + (r & 1) * 4;
            const bool in = rr < rows && (KT > 1 || !(r & 1));
            const int flat = flat0 + (in ? rr : 0), j = flat / heads;
            const __nv_bfloat16* src = p.q + (long long)(pc.it.row0 + j) * p.q_row_stride +
                                       (long long)(head0 + flat - j * heads) * p.q_head_stride + 8 * i4;
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
        if (LN::kQueryShared) __syncwarp();

        for (int k = pc.k0, n = 0; k < end; ++k, ++n) {
            const int t0 = k * TILE;
            bool all = t0 + TILE - 1 <= p0;  // every row sees every token
            look(next_id, k + 1);
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
                load(vc[b], id[b], t0 + 16 * b, block / 2);
                all = all && exists(id[b]);
                if (!exists(id[b]) && id[b] != -2 && lane == 0) flag_status(p.status, MXQ_DEV_BAD_PAGE);
            }
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
            // ---- sums q . c of 16 tokens at a time, tokens r and r + 8 in a lane
            float sc[SUB][KT][2];
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float a[VT][4];
#pragma unroll
                    for (int u = g * G / 32; u < (g + 1) * G / 32; ++u) {
                        uint32_t x[4], y[4];
                        codes_of(kc[b].w0[u], x);
                        codes_of(kc[b].w1[u], y);
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
                    const float s0 = __uint_as_float(kc[b].pr0[g] << 16);
                    const float s1 = __uint_as_float(kc[b].pr1[g] << 16);
                    const float b0 = __uint_as_float(kc[b].pr0[g] & 0xFFFF0000u);
                    const float b1 = __uint_as_float(kc[b].pr1[g] & 0xFFFF0000u);
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
            if (!all) {
                // some row does not see some token; what no row sees may hold anything
#pragma unroll
                for (int b = 0; b < SUB; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = t0 + 16 * b + r + 8 * i;
                        const bool is = exists(id[b]) && t <= p1;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            if (!is && i == 0) vc[b].pr0[g] = 0u;
                            if (!is && i == 1) vc[b].pr1[g] = 0u;
                        }
#pragma unroll
                        for (int kt = 0; kt < KT; ++kt)
                            if (!(is && t <= position(kt))) sc[b][kt][i] = -INFINITY;
                    }
            }
            // ---- running maximum: moved only when a score is far above it, and the
            // values' power of two, when a scale is above it
            uint32_t scales = 0;  // the low half word
#pragma unroll
            for (int b = 0; b < SUB; ++b)
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    scales = max_u16x2(scales, max_u16x2(vc[b].pr0[g], vc[b].pr1[g]));
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
#pragma unroll
                    for (int b = 0; b < SUB; ++b)
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            size = max(size, max(vc[b].pr0[g] & 0x7FFFu, vc[b].pr1[g] & 0x7FFFu));
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
            // ---- the next tile's keys, then the weighted sum of the values
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
                load(kc[b], next_id[b], t0 + TILE + 16 * b, 0);
                id[b] = next_id[b];
            }
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
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
                    const float s0 = __uint_as_float(vc[b].pr0[g] << 16);
                    const float s1 = __uint_as_float(vc[b].pr1[g] << 16);
                    const float b0 = __uint_as_float(vc[b].pr0[g] & 0xFFFF0000u);
                    const float b1 = __uint_as_float(vc[b].pr1[g] & 0xFFFF0000u);
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
                        codes_of(vc[b].w0[u], x);
                        codes_of(vc[b].w1[u], y);
#pragma unroll
                        for (int vt = 0; vt < VT; ++vt) {
                            mma_f16(acc[vt][2 * u], x[0], x[1], y[0], y[1], f0[vt], f1[vt]);
                            mma_f16(acc[vt][2 * u + 1], x[2], x[3], y[2], y[3], f0[vt], f1[vt]);
                        }
                    }
                }
            }
        }

        // ---- the piece's result
        const float v_down = pow2_of(max(v_exp - 6, 1));  // 1 / v_up
        float* to = p.partial + (long long)(pc.tile + runner) * (LN::kRows * (D + 2));
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
__global__ void __launch_bounds__(kLoneThreads,
                                  Lone<D, G, KT1>::kCtas < Lone<D, G, KT2>::kCtas ? Lone<D, G, KT1>::kCtas
                                                                                 : Lone<D, G, KT2>::kCtas)
    kv_lone_kernel(const __grid_constant__ KvSharedParams a, const __grid_constant__ KvSharedParams b) {
    constexpr int kQuery = Lone<D, G, KT1>::kQueryBytes > Lone<D, G, KT2>::kQueryBytes ? Lone<D, G, KT1>::kQueryBytes
                                                                                      : Lone<D, G, KT2>::kQueryBytes;
    __shared__ Sums<kLoneThreads> prefix_sums, own_sums;
    __shared__ uint4 queries[kQuery ? kLoneWarps * kQuery / 16 : 1];
    pdl_launch_dependents();
    sum_items(a, prefix_sums);
    sum_items(b, own_sums);
    __syncthreads();
    const int warp = threadIdx.x / 32;
    const Scan prefix = scan_sums(a, prefix_sums), own = scan_sums(b, own_sums);
    const long long prefix_cost = all_units(a, prefix) * a.unit_cost, own_cost = all_units(b, own) * b.unit_cost;
    // Runners of the two parts.  Beside the other kernel they are the first CTAs, which are on the SMs
    // that it leaves; else consecutive ones are on different SMs.
    const int all = gridDim.x * kLoneWarps;
    const int runner = a.on_tensor_cores ? blockIdx.x * kLoneWarps + warp : warp * gridDim.x + blockIdx.x;
    int first = 0, second = all;
    if (a.on_tensor_cores) {
        // the SMs that the other kernel leaves; it needs them all for itself if there is nothing else
        const int sms = share_of(prefix_cost, own_cost, a.sms);
        if (sms < a.sms) second = (int)((long long)all * (a.sms - sms) / a.sms);
    } else {
        first = share_of(prefix_cost, own_cost, all);
        second = all - first;
    }
    const long long own_run = run_length(b, all_units(b, own), second);
    const long long prefix_run = a.on_tensor_cores ? 0 : run_length(a, all_units(a, prefix), first);
    if (blockIdx.x == 0) {
        write_before(b, own_sums, own, own_run);
        if (!a.on_tensor_cores) write_before(a, prefix_sums, prefix, prefix_run);
    }
    SharedWalk walk;
    uint4* mine = queries + (kQuery ? warp * (kQuery / 16) : 0);
    if (!a.on_tensor_cores && runner < first) {
        walk.start(a, prefix_sums, prefix, prefix_run, runner);
        lone_run<D, G, KT1>(a, walk, runner, mine);
    } else if (runner - first < second) {
        walk.start(b, own_sums, own, own_run, runner - first);
        lone_run<D, G, KT2>(b, walk, runner - first, mine);
    }
    // The tensor cores' kernel may still run; the joining kernel waits for this one only.
    if (a.on_tensor_cores) pdl_wait();
}

}  // namespace
}  // namespace mxq
