// C ABI of the key/value cache operators: argument checks, planning, launches.
#include <atomic>
#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>

#include "../../include/mxq.h"
#include "kv_format.cuh"
#include "mxq_internal.h"

namespace {

constexpr int kMaxSms = 160;          // workspace sizes do not depend on the device
constexpr int kMaxInt = 1 << 30;      // windows and sinks beyond this are all of it

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool cache_shape(int D, int G, int page_size) {
    if (D != 64 && D != 128 && D != 256) return false;
    if ((G != 32 && G != 64 && G != 128) || G > D) return false;
    return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128;
}

int page_shift_of(int page_size) {
    return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
}

bool stride_ok(long long s) { return s >= 0 && s % 8 == 0; }

// How an attention call is cut into row tiles and CTAs.  Sequences whose rows
// times query heads of a key/value head are at most 16 go through the kernel for
// few rows (bound by the cache's bytes), the others through the tensor cores'
// (bound by their products).  32 sequences of 8192 tokens, 8 key/value heads of 128
// values: the first takes 117 us for 16 rows, the second 262 for 20 rows and 270 for
// 128; of 64 values 87 and 243, of 256 272 and 409.  Two row tiles of the first took
// 226 for 17 to 32 rows; they are not used: a prompt's first rows, which see few tokens,
// would then have weights times scales of 11 bits, rounded against a group's range, as rows
// of up to 16 have, and not weights and values of 11 bits each, which is what rows of this
// number are held to.
struct AttnPlan {
    int head_parts, part_heads, tile_rows, tile_toks, ctas;  // few rows
    int many, many_parts, many_heads, half_toks, many_toks, many_ctas;
    long long max_entries;
    size_t seg_bytes, few_bytes;
    size_t many_seg_bytes, many_partial_bytes, seq_bytes, entry_bytes, before_bytes, many_bytes;
    size_t bytes;
};

AttnPlan plan_attn(int T, int S, int Hq, int Hkv, int D, int max_q, int sms) {
    AttnPlan a;
    const int rep = Hq / Hkv;
    a.head_parts = (rep + 15) / 16;
    a.part_heads = (rep + a.head_parts - 1) / a.head_parts;
    const long long rows = (long long)max_q * a.part_heads;
    a.tile_rows = rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
    a.tile_toks = a.tile_rows / a.part_heads;
    a.ctas = sms * mxq::kv_attn_ctas_per_sm();
    a.seg_bytes = align_up(mxq::kv_attn_seg_bytes(a.ctas), 256);
    a.few_bytes = a.seg_bytes + align_up(mxq::kv_attn_partial_bytes(a.ctas, a.tile_rows, D), 256);
    a.bytes = a.few_bytes;
    a.many = max_q > a.tile_toks;
    if (a.many) {
        a.many_parts = (rep + 127) / 128;
        a.many_heads = (rep + a.many_parts - 1) / a.many_parts;
        a.half_toks = 128 / a.many_heads;
        const int tile_rows = mxq::kv_prefill_rows(D);
        a.many_toks = a.half_toks * (tile_rows / 128);
        a.many_ctas = sms;
        a.max_entries = (long long)T / a.many_toks + S;
        a.many_seg_bytes = align_up(mxq::kv_attn_seg_bytes(a.many_ctas), 256);
        a.many_partial_bytes =
            align_up(mxq::kv_attn_partial_bytes(a.many_ctas, tile_rows, D), 256);
        a.seq_bytes = align_up((size_t)S * sizeof(int), 256);
        a.entry_bytes = align_up((size_t)a.max_entries * mxq::kv_prefill_entry_bytes(), 256);
        a.before_bytes = align_up((size_t)a.max_entries * sizeof(int), 256);
        a.many_bytes = a.many_seg_bytes + a.many_partial_bytes + a.seq_bytes + a.entry_bytes +
                       a.before_bytes + 256;
        a.bytes += a.many_bytes;
    }
    return a;
}

// The kernels count units (a row tile and a tile of the tokens that it sees) in 32 bits: of a few
// rows' sequences in a thread and in a CTA's run, of all prompts' row tiles for one head.  True
// where the counts fit for any lengths in pages of `tokens` tokens.
bool countable(const AttnPlan& a, int S, int Hkv, long long tokens) {
    constexpr long long kMost = (1LL << 30) - 64;
    const long long vheads = (long long)Hkv * a.head_parts, few = tokens / 32 + 32;
    if ((S / 128 + 1) * few > kMost || few * vheads > kMost || S * few > kMost / vheads * a.ctas)
        return false;
    if (!a.many) return true;
    const long long many_vheads = (long long)Hkv * a.many_parts, units = tokens / 128 + 16;
    if (a.max_entries > 2 * kMost || a.max_entries * units > 2 * kMost) return false;
    return a.max_entries * units <= kMost / many_vheads * a.many_ctas;
}

// How one part of a call over shared prefixes is cut (KvSharedParams): row tiles, runners (warps, or
// CTAs on the tensor cores), and its share of the workspace.
struct SharedPart {
    int head_parts, part_heads, tile_rows, tensor_cores;
    long long runners;
    // row tiles of one head: those that there are places for, as many as items can have between them whose rows do
    // not overlap; and with starts that decrease, so that they do
    long long planes, most_planes;
    size_t before_bytes, bytes;
};

SharedPart shared_part(long long items, long long rows, int rep, int sms) {
    SharedPart a;
    a.head_parts = (rep + 15) / 16;
    a.part_heads = (rep + a.head_parts - 1) / a.head_parts;
    const long long all = rows * a.part_heads;
    a.tile_rows = all <= 4 ? 4 : all <= 8 ? 8 : 16;
    a.tensor_cores = 0;
    a.runners = 16LL * sms;  // warps
    a.most_planes = items * ((all + a.tile_rows - 1) / a.tile_rows);
    return a;
}

struct SharedPlan {
    SharedPart prefix, own;
    size_t bytes;
};

// The groups' rows are taken by warps on their own up to kFewPrefixRows, above by the tensor cores.  32 groups of
// 8 and 12 sequences (32 and 48 rows) over 4096 tokens, 8 heads of 128 values: 158 and 220 us by warps, 172 and 176 on
// the tensor cores; 8 such groups: 52.8 and 68.8, 54.6 and 57.6.
constexpr int kFewPrefixRows = 32;

SharedPlan plan_shared(int T, int S, int N, int Hq, int Hkv, int D, int max_q, int max_group, int sms) {
    SharedPlan a;
    const int rep = Hq / Hkv;
    a.own = shared_part(S, max_q, rep, sms);
    const long long all = (long long)max_group * max_q, rows = all < T ? all : T;
    SharedPart& p = a.prefix;
    p = shared_part(N, rows, rep, sms);
    if (rows * p.part_heads > kFewPrefixRows) {
        p.tensor_cores = 1;
        p.head_parts = (rep + 127) / 128;
        p.part_heads = (rep + p.head_parts - 1) / p.head_parts;
        p.tile_rows = mxq::kv_prefill_rows(D);
        p.runners = sms;
        p.most_planes = N * ((rows * p.part_heads + p.tile_rows - 1) / p.tile_rows);
    } else if (p.tile_rows != a.own.tile_rows) {
        p.tile_rows = 16;  // (there is no kernel of 8 rows beside 4)
        p.most_planes = N * ((rows * p.part_heads + 15) / 16);
    }
    a.bytes = 0;
    for (SharedPart* x : {&a.prefix, &a.own}) {
        const int items = x == &a.own ? S : N;
        x->planes = (long long)T * x->part_heads / x->tile_rows + items;
        if (x->planes > x->most_planes) x->planes = x->most_planes;
        x->before_bytes = align_up((size_t)items * mxq::kv_shared_before_bytes(), 256) + 256;
        const size_t places = (size_t)x->planes * Hkv * x->head_parts + x->runners;
        x->bytes = x->before_bytes + align_up(places * x->tile_rows * (D + 2) * sizeof(float), 256);
        a.bytes += x->bytes;
    }
    return a;
}

// As for AttnPlan: units of one head and of a run, places, and the rows times query heads fit 32 bits, for rows that do
// not overlap; and the row tiles that a block's threads count where they do, each one more than there are places at most.
bool countable(const SharedPart& a, int T, int Hkv, long long tokens) {
    constexpr long long kMost = (1LL << 30) - 64;
    const long long units = tokens / (a.tensor_cores ? 128 : 16) + 32, vheads = (long long)Hkv * a.head_parts;
    return a.planes <= kMost / units && a.planes <= kMost / vheads - a.runners && (long long)T * a.part_heads <= kMost &&
           (a.most_planes <= 2 * kMost || a.planes < 2 * kMost / mxq::kKvListThreads);
}

// Calls over shared prefixes in which each sequence may go over its prefix for itself, in one kernel
// and for short calls in one launch: where that takes no longer.  Times are of 152 SMs, in us: a row
// tile and token of 128 values takes 30, 35 and 53 ps of the whole GPU for 4, 8 and 16 rows (32
// sequences of 8192 tokens, 8 heads: 62, 73, 111 us), on the tensor cores 123 for a tile of up to 128
// rows and 160 above.  What the calls take beside it: 8, and 22 in two parts with their joining.  The
// lengths are not known here, only how many pages they may be in.  4 sequences after 573 tokens: 8.2 us, in
// two parts 21.8.
bool each_for_itself(const AttnPlan& each, const SharedPlan& a, int S, int N, int Hkv, int D, int max_q,
                     int max_group, const long long (&tokens)[2]) {
    if (max_q > each.tile_toks) return false;
    if (max_group == 1) return true;
    const double size = D / 128.0 * 1e-6;
    auto few = [](int rows) { return rows == 4 ? 30.0 : rows == 8 ? 35.0 : 53.0; };
    const double own = few(each.tile_rows) * S * Hkv * each.head_parts * size;
    const SharedPart& p = a.prefix;
    const double shared = (p.tensor_cores ? (p.most_planes > N || max_group * (long long)max_q * p.part_heads > 128 ? 160.0 : 123.0)
                                          : few(p.tile_rows)) * p.most_planes * Hkv * p.head_parts * size;
    return 8 + own * (double)(tokens[0] + tokens[1]) <= 22 + shared * (double)tokens[0] + own * (double)tokens[1];
}

}  // namespace

extern "C" {

size_t mxq_kv_block_bytes(int D, int page_size, int group_size) {
    if (!cache_shape(D, group_size, page_size)) return 0;
    return (size_t)mxq::kv_block_bytes(D, group_size, page_size);
}

mxq_status mxq_qk_norm_rope(const void* q, long long q_row_stride, long long q_head_stride,
                            const void* k, long long k_row_stride, long long k_head_stride,
                            const int32_t* positions, const float* inv_freq, const void* q_weight,
                            const void* k_weight, void* q_out, long long q_out_row_stride,
                            long long q_out_head_stride, void* k_out,
                            long long k_out_row_stride, long long k_out_head_stride, int T,
                            int Hq, int Hk, int D, int rot_dim, int interleaved, float eps,
                            float weight_offset, float rope_scale, void* stream) {
    if (T < 0 || Hq < 0 || Hk < 0 || Hq + (long long)Hk <= 0 || Hq > 65535 || Hk > 65535)
        return MXQ_ERR_INVALID_ARG;
    if (D <= 0 || D > 256 || D % 8 != 0) return MXQ_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0) return MXQ_ERR_INVALID_ARG;
    if (rot_dim == 0 && !q_weight && !k_weight) return MXQ_ERR_INVALID_ARG;
    if (T > 0 && ((rot_dim && (!positions || !inv_freq)) || (Hq && (!q || !q_out)) ||
                  (Hk && (!k || !k_out))))
        return MXQ_ERR_INVALID_ARG;
    if (!stride_ok(q_row_stride) || !stride_ok(q_head_stride) || !stride_ok(k_row_stride) ||
        !stride_ok(k_head_stride) || !stride_ok(q_out_row_stride) ||
        !stride_ok(q_out_head_stride) || !stride_ok(k_out_row_stride) ||
        !stride_ok(k_out_head_stride))
        return MXQ_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
        !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(positions, 4) ||
        !aligned(inv_freq, 4))
        return MXQ_ERR_MISALIGNED;
    int sms = 0;
    const mxq_status st = mxq::check_current_device(&sms);
    if (st != MXQ_OK) return st;
    if (T == 0) return MXQ_OK;
    mxq::NormRopeParams p;
    p.q = {static_cast<const __nv_bfloat16*>(q), q_row_stride, q_head_stride,
           static_cast<const __nv_bfloat16*>(q_weight), static_cast<__nv_bfloat16*>(q_out),
           q_out_row_stride, q_out_head_stride};
    p.k = {static_cast<const __nv_bfloat16*>(k), k_row_stride, k_head_stride,
           static_cast<const __nv_bfloat16*>(k_weight), static_cast<__nv_bfloat16*>(k_out),
           k_out_row_stride, k_out_head_stride};
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.T = T;
    p.Hq = Hq;
    p.Hk = Hk;
    p.D = D;
    p.rot = rot_dim;
    p.interleaved = interleaved ? 1 : 0;
    p.eps = eps;
    p.weight_offset = weight_offset;
    p.rope_scale = rope_scale;
    const cudaError_t err = mxq::launch_qk_norm_rope(p, sms, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

mxq_status mxq_kv_append(const void* k, long long k_row_stride, long long k_head_stride,
                         const void* v, long long v_row_stride, long long v_head_stride,
                         void* pages, const int32_t* slots, int T, int Hkv, int D, int n_pages,
                         int page_size, int group_size, int32_t* dev_status, void* stream) {
    if (T < 0 || Hkv <= 0 || n_pages <= 0 || !cache_shape(D, group_size, page_size))
        return MXQ_ERR_INVALID_ARG;
    if (!pages || (T > 0 && (!k || !v || !slots))) return MXQ_ERR_INVALID_ARG;
    if (!stride_ok(k_row_stride) || !stride_ok(k_head_stride) || !stride_ok(v_row_stride) ||
        !stride_ok(v_head_stride))
        return MXQ_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pages, 16) || !aligned(slots, 4) ||
        !aligned(dev_status, 4))
        return MXQ_ERR_MISALIGNED;
    int sms = 0;
    const mxq_status st = mxq::check_current_device(&sms);
    if (st != MXQ_OK) return st;
    if (2LL * T * Hkv > (long long)kMaxInt * 4) return MXQ_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dev_status && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess)
        return MXQ_ERR_CUDA;
    if (T == 0) return MXQ_OK;
    mxq::KvRowsParams p;
    std::memset(&p, 0, sizeof p);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.k_row_stride = k_row_stride;
    p.k_head_stride = k_head_stride;
    p.v_row_stride = v_row_stride;
    p.v_head_stride = v_head_stride;
    p.pages = static_cast<uint8_t*>(pages);
    p.slots = slots;
    p.T = T;
    p.H = Hkv;
    p.n_pages = n_pages;
    p.page_size = page_size;
    p.page_shift = page_shift_of(page_size);
    p.status = dev_status;
    const cudaError_t err = mxq::launch_kv_append(p, D, group_size, sms, s);
    return err == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

mxq_status mxq_kv_read(const void* pages, const int32_t* slots, void* k_out, void* v_out, int T,
                       int Hkv, int D, int n_pages, int page_size, int group_size,
                       int32_t* dev_status, void* stream) {
    if (T < 0 || Hkv <= 0 || n_pages <= 0 || !cache_shape(D, group_size, page_size))
        return MXQ_ERR_INVALID_ARG;
    if (!pages || (T > 0 && (!slots || !k_out || !v_out))) return MXQ_ERR_INVALID_ARG;
    if (!aligned(pages, 16) || !aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
        !aligned(dev_status, 4))
        return MXQ_ERR_MISALIGNED;
    int sms = 0;
    const mxq_status st = mxq::check_current_device(&sms);
    if (st != MXQ_OK) return st;
    if (2LL * T * Hkv > (long long)kMaxInt * 4) return MXQ_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dev_status && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess)
        return MXQ_ERR_CUDA;
    if (T == 0) return MXQ_OK;
    mxq::KvRowsParams p;
    std::memset(&p, 0, sizeof p);
    p.k_out = static_cast<__nv_bfloat16*>(k_out);
    p.v_out = static_cast<__nv_bfloat16*>(v_out);
    p.pages = static_cast<uint8_t*>(const_cast<void*>(pages));
    p.slots = slots;
    p.T = T;
    p.H = Hkv;
    p.n_pages = n_pages;
    p.page_size = page_size;
    p.page_shift = page_shift_of(page_size);
    p.status = dev_status;
    const cudaError_t err = mxq::launch_kv_read(p, D, group_size, sms, s);
    return err == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

size_t mxq_kv_attention_workspace_bytes(int T, int S, int Hq, int Hkv, int D, int max_q_len) {
    if (T < 0 || S < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0 || max_q_len <= 0)
        return 0;
    if (max_q_len > T) max_q_len = T > 0 ? T : 1;
    // more SMs never need less
    return plan_attn(T, S, Hq, Hkv, D, max_q_len, kMaxSms).bytes;
}

mxq_status mxq_kv_attention(const void* q, long long q_row_stride, long long q_head_stride,
                            const void* pages, const int32_t* page_table, const int32_t* ctx_lens,
                            const int32_t* q_starts, void* out, float* lse, int T, int S, int Hq,
                            int Hkv, int D, int n_pages, int max_pages, int page_size,
                            int group_size, int max_q_len, float scale, int window, int sinks,
                            void* workspace, size_t workspace_bytes, int32_t* dev_status,
                            void* stream) {
    if (T < 0 || S < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || n_pages <= 0 || max_pages <= 0 ||
        !cache_shape(D, group_size, page_size))
        return MXQ_ERR_INVALID_ARG;
    if (max_q_len <= 0 || window < 0 || sinks < 0 || !(scale > 0.f) || scale - scale != 0.f)
        return MXQ_ERR_INVALID_ARG;
    if (!q_starts && (T != S || max_q_len != 1)) return MXQ_ERR_INVALID_ARG;
    if (!pages || (T > 0 && S > 0 && (!q || !page_table || !ctx_lens || !out)))
        return MXQ_ERR_INVALID_ARG;
    if (!stride_ok(q_row_stride) || !stride_ok(q_head_stride)) return MXQ_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size > kMaxInt || T > kMaxInt || S > kMaxInt)
        return MXQ_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(pages, 16) || !aligned(out, 16) || !aligned(page_table, 4) ||
        !aligned(ctx_lens, 4) || !aligned(q_starts, 4) || !aligned(lse, 4) ||
        !aligned(dev_status, 4) || !aligned(workspace, 256))
        return MXQ_ERR_MISALIGNED;
    if (max_q_len > T && T > 0) max_q_len = T;  // no sequence has more rows than there are
    const long long tokens = (long long)max_pages * page_size;
    if (!countable(plan_attn(T, S, Hq, Hkv, D, max_q_len, kMaxSms), S, Hkv, tokens))
        return MXQ_ERR_UNSUPPORTED;
    if (T > 0 && S > 0 &&
        (!workspace ||
         workspace_bytes < mxq_kv_attention_workspace_bytes(T, S, Hq, Hkv, D, max_q_len)))
        return MXQ_ERR_WORKSPACE;
    int sms = 0;
    const mxq_status st = mxq::check_current_device(&sms);
    if (st != MXQ_OK) return st;
    const AttnPlan a = plan_attn(T, S, Hq, Hkv, D, max_q_len, sms < kMaxSms ? sms : kMaxSms);
    if (!countable(a, S, Hkv, tokens)) return MXQ_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dev_status && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess)
        return MXQ_ERR_CUDA;
    if (T == 0 || S == 0) return MXQ_OK;
    mxq::KvAttnParams p;
    std::memset(&p, 0, sizeof p);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.q_row_stride = q_row_stride;
    p.q_head_stride = q_head_stride;
    p.pages = static_cast<const uint8_t*>(pages);
    p.table = page_table;
    p.ctx_lens = ctx_lens;
    p.q_starts = q_starts;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.T = T;
    p.S = S;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.page_size = page_size;
    p.max_q = max_q_len;
    p.window = window < kMaxInt ? window : kMaxInt;
    p.sinks = sinks < kMaxInt ? sinks : kMaxInt;
    p.scale_log2 = (float)(scale * 1.4426950408889634);
    p.page_shift = page_shift_of(page_size);
    p.status = dev_status;
    p.wait_budget = mxq::wait_budget_cycles();
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.head_parts = a.head_parts;
    p.part_heads = a.part_heads;
    p.tile_toks = a.tile_toks;
    p.min_rows = 0;
    p.max_rows = a.tile_toks;
    p.ctas = a.ctas;
    p.segs = reinterpret_cast<int*>(ws);
    p.partial = reinterpret_cast<float*>(ws + a.seg_bytes);
    // where the others' rows cannot make up the total, every sequence has many
    const bool all_many = T - (long long)(S - 1) * max_q_len > a.tile_toks;
    if (!all_many && mxq::launch_kv_attn(p, D, group_size, a.tile_rows, s) != cudaSuccess)
        return MXQ_ERR_CUDA;
    if (!a.many) return MXQ_OK;
    ws += a.few_bytes;
    p.head_parts = a.many_parts;
    p.part_heads = a.many_heads;
    p.tile_toks = a.many_toks;
    p.half_toks = a.half_toks;
    p.min_rows = all_many ? 0 : a.tile_toks + 1;
    p.max_rows = kMaxInt;
    p.ctas = a.many_ctas;
    p.max_entries = (int)a.max_entries;
    p.segs = reinterpret_cast<int*>(ws);
    ws += a.many_seg_bytes;
    p.partial = reinterpret_cast<float*>(ws);
    ws += a.many_partial_bytes;
    p.seq_tiles = reinterpret_cast<int*>(ws);
    ws += a.seq_bytes;
    p.entries = ws;
    ws += a.entry_bytes;
    p.before = reinterpret_cast<int*>(ws);
    ws += a.before_bytes;
    p.counts = reinterpret_cast<int*>(ws);
    const cudaError_t err = mxq::launch_kv_prefill(p, D, group_size, s);
    return err == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

size_t mxq_kv_attention_shared_workspace_bytes(int T, int S, int N, int Hq, int Hkv, int D,
                                               int max_q_len, int max_group) {
    if (T < 0 || S < 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0 || max_q_len <= 0 ||
        max_group <= 0)
        return 0;
    if (max_q_len > T) max_q_len = T > 0 ? T : 1;
    if (max_group > S) max_group = S > 0 ? S : 1;
    const size_t parts = plan_shared(T, S, N, Hq, Hkv, D, max_q_len, max_group, kMaxSms).bytes;
    const size_t each = plan_attn(T, S, Hq, Hkv, D, max_q_len, kMaxSms).few_bytes;
    return parts > each ? parts : each;
}

mxq_status mxq_kv_attention_shared(const void* q, long long q_row_stride, long long q_head_stride,
                                   const void* pages, const int32_t* prefix_table,
                                   const int32_t* prefix_lens, const int32_t* group_starts,
                                   const int32_t* page_table, const int32_t* ctx_lens,
                                   const int32_t* q_starts, void* out, float* lse, int T, int S, int N,
                                   int Hq, int Hkv, int D, int n_pages, int max_prefix_pages,
                                   int max_pages, int page_size, int group_size, int max_q_len,
                                   int max_group, float scale, void* workspace, size_t workspace_bytes,
                                   int32_t* dev_status, void* stream) {
    if (T < 0 || S < 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || n_pages <= 0 ||
        max_pages <= 0 || max_prefix_pages <= 0 || !cache_shape(D, group_size, page_size))
        return MXQ_ERR_INVALID_ARG;
    if (max_q_len <= 0 || max_group <= 0 || !(scale > 0.f) || scale - scale != 0.f)
        return MXQ_ERR_INVALID_ARG;
    if (!q_starts && (T != S || max_q_len != 1)) return MXQ_ERR_INVALID_ARG;
    if (!group_starts && (S % N != 0 || S / N > max_group)) return MXQ_ERR_INVALID_ARG;
    if (!pages || (T > 0 && S > 0 &&
                   (!q || !prefix_table || !prefix_lens || !page_table || !ctx_lens || !out)))
        return MXQ_ERR_INVALID_ARG;
    if (!stride_ok(q_row_stride) || !stride_ok(q_head_stride)) return MXQ_ERR_INVALID_ARG;
    const long long tokens[2] = {(long long)max_prefix_pages * page_size, (long long)max_pages * page_size};
    if (tokens[0] > kMaxInt || tokens[1] > kMaxInt || T > kMaxInt || S > kMaxInt || N > kMaxInt ||
        Hq > 65535 * 8)
        return MXQ_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(pages, 16) || !aligned(out, 16) || !aligned(prefix_table, 4) ||
        !aligned(prefix_lens, 4) || !aligned(group_starts, 4) || !aligned(page_table, 4) ||
        !aligned(ctx_lens, 4) || !aligned(q_starts, 4) || !aligned(lse, 4) ||
        !aligned(dev_status, 4) || !aligned(workspace, 256))
        return MXQ_ERR_MISALIGNED;
    if (max_q_len > T && T > 0) max_q_len = T;
    if (max_group > S && S > 0) max_group = S;
    const SharedPlan most = plan_shared(T, S, N, Hq, Hkv, D, max_q_len, max_group, kMaxSms);
    if (!countable(most.prefix, T, Hkv, tokens[0]) || !countable(most.own, T, Hkv, tokens[1]))
        return MXQ_ERR_UNSUPPORTED;
    if (T > 0 && S > 0 &&
        (!workspace || workspace_bytes < mxq_kv_attention_shared_workspace_bytes(T, S, N, Hq, Hkv, D, max_q_len, max_group)))
        return MXQ_ERR_WORKSPACE;
    int sms = 0;
    const mxq_status st = mxq::check_current_device(&sms);
    if (st != MXQ_OK) return st;
    const SharedPlan a =
        plan_shared(T, S, N, Hq, Hkv, D, max_q_len, max_group, sms < kMaxSms ? sms : kMaxSms);
    if (!countable(a.prefix, T, Hkv, tokens[0]) || !countable(a.own, T, Hkv, tokens[1]))
        return MXQ_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dev_status && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess)
        return MXQ_ERR_CUDA;
    if (T == 0 || S == 0) return MXQ_OK;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    auto set = [&](mxq::KvGroupParams& x) {
        x.q = static_cast<const __nv_bfloat16*>(q);
        x.q_row_stride = q_row_stride;
        x.q_head_stride = q_head_stride;
        x.pages = static_cast<const uint8_t*>(pages);
        x.table = page_table;
        x.max_pages = max_pages;
        x.ctx_lens = ctx_lens;
        x.q_starts = q_starts;
        x.out = static_cast<__nv_bfloat16*>(out);
        x.lse = lse;
        x.T = T;
        x.S = S;
        x.n_pages = n_pages;
        x.Hq = Hq;
        x.Hkv = Hkv;
        x.page_size = page_size;
        x.page_shift = page_shift_of(page_size);
        x.max_q = max_q_len;
        x.scale_log2 = (float)(scale * 1.4426950408889634);
        x.status = dev_status;
        x.wait_budget = mxq::wait_budget_cycles();
        x.groups_n = N;
        x.max_group = max_group;
        x.groups = group_starts;
        x.prefix_lens = prefix_lens;
    };
    const AttnPlan each = plan_attn(T, S, Hq, Hkv, D, max_q_len, sms < kMaxSms ? sms : kMaxSms);
    if (each_for_itself(each, a, S, N, Hkv, D, max_q_len, max_group, tokens) &&
        countable(each, S, Hkv, tokens[0] + tokens[1])) {
        mxq::KvTwoParams x = mxq::KvTwoParams();
        set(x);
        x.prefix_table = prefix_table;
        x.max_prefix_pages = max_prefix_pages;
        x.head_parts = each.head_parts;
        x.part_heads = each.part_heads;
        x.tile_rows = each.tile_rows;
        x.tile_toks = each.tile_toks;
        x.max_rows = each.tile_toks;
        x.ctas = each.ctas;
        x.segs = reinterpret_cast<int*>(ws);
        x.partial = reinterpret_cast<float*>(ws + each.seg_bytes);
        return mxq::launch_kv_two(x, D, group_size, each.tile_rows, s) == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
    }
    // spread over all bits, so that what lies in a workspace is no call's
    static std::atomic<uint64_t> calls{0};
    const uint64_t call = (++calls * 0x9E3779B97F4A7C15u) & ~255ull;
    mxq::KvSharedParams p[2] = {};
    for (int i = 0; i < 2; ++i) {
        mxq::KvSharedParams& x = p[i];
        const SharedPart& part = i ? a.own : a.prefix;
        set(x);
        if (!i) {
            x.table = prefix_table;
            x.max_pages = max_prefix_pages;
        }
        x.prefix = !i;
        x.head_parts = part.head_parts;
        x.part_heads = part.part_heads;
        x.max_planes = (int)part.planes;
        x.tile_rows = part.tile_rows;
        x.on_tensor_cores = part.tensor_cores;
        x.sms = sms < kMaxSms ? sms : kMaxSms;
        mxq::kv_shared_shape(x, D);
        x.totals = reinterpret_cast<long long*>(ws);
        x.call = call;
        x.before = reinterpret_cast<mxq::Before*>(ws + 256);
        x.partial = reinterpret_cast<float*>(ws + part.before_bytes);
        ws += part.bytes;
    }
    cudaError_t err = cudaSuccess;
    if (p[0].on_tensor_cores) err = mxq::launch_kv_shared_many(p[0], p[1], D, group_size, s);
    if (err == cudaSuccess) err = mxq::launch_kv_shared_lone(p[0], p[1], D, group_size, s);
    if (err == cudaSuccess) err = mxq::launch_kv_shared_join(p[0], p[1], D, s);
    return err == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

size_t mxq_kv_reorder_workspace_bytes(int S) {
    return S < 0 ? 0 : align_up((size_t)S * mxq::kv_reorder_move_bytes(), 256);
}

mxq_status mxq_kv_reorder(void* pages, const int32_t* page_table, const int32_t* home_table,
                          const int32_t* ctx_lens, const int32_t* parents, int32_t* table_out,
                          int32_t* lens_out, int S, int W, int layers, int n_pages, int Hkv, int D,
                          int max_pages, int page_size, int group_size, void* workspace,
                          size_t workspace_bytes, int32_t* dev_status, void* stream) {
    if (S < 0 || W <= 0 || W > 64 || S % W != 0 || layers <= 0 || n_pages <= 0 || Hkv <= 0 ||
        max_pages <= 0 || !cache_shape(D, group_size, page_size))
        return MXQ_ERR_INVALID_ARG;
    if (!pages || (S > 0 && (!page_table || !home_table || !ctx_lens || !parents || !table_out || !lens_out)))
        return MXQ_ERR_INVALID_ARG;
    if (S > 0 && (table_out == home_table || lens_out == parents)) return MXQ_ERR_INVALID_ARG;
    if (!aligned(pages, 16) || !aligned(page_table, 4) || !aligned(home_table, 4) || !aligned(ctx_lens, 4) ||
        !aligned(parents, 4) || !aligned(table_out, 4) || !aligned(lens_out, 4) || !aligned(dev_status, 4) ||
        !aligned(workspace, 256))
        return MXQ_ERR_MISALIGNED;
    if ((long long)max_pages * page_size > kMaxInt || S > kMaxInt || (long long)layers * Hkv > kMaxInt)
        return MXQ_ERR_UNSUPPORTED;
    if (S > 0 && (!workspace || workspace_bytes < mxq_kv_reorder_workspace_bytes(S)))
        return MXQ_ERR_WORKSPACE;
    const mxq_status st = mxq::check_current_device(nullptr);
    if (st != MXQ_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dev_status && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess)
        return MXQ_ERR_CUDA;
    if (S == 0) return MXQ_OK;
    mxq::KvReorderParams p;
    p.pages = static_cast<uint8_t*>(pages);
    p.table = page_table;
    p.home = home_table;
    p.lens = ctx_lens;
    p.parents = parents;
    p.table_out = table_out;
    p.lens_out = lens_out;
    p.moves = workspace;
    p.S = S;
    p.W = W;
    p.layers = layers;
    p.n_pages = n_pages;
    p.H = Hkv;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.status = dev_status;
    const cudaError_t err = mxq::launch_kv_reorder(p, D, group_size, s);
    return err == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

}  // extern "C"
