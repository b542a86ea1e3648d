// C ABI of the key/value cache operators: argument checks, planning, launches.
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

}  // extern "C"
