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

bool stride_ok(long long s) { return s >= 0 && s % 8 == 0; }

// How an attention call is cut into row tiles and CTAs.
struct AttnPlan {
    int head_parts, part_heads, tile_rows, tile_toks, planes, ctas;
    size_t seg_bytes, bytes;
};

AttnPlan plan_attn(int Hq, int Hkv, int D, int max_q, int sms) {
    AttnPlan a;
    const int rep = Hq / Hkv;
    a.head_parts = (rep + 15) / 16;
    a.part_heads = (rep + a.head_parts - 1) / a.head_parts;
    const long long rows = (long long)max_q * a.part_heads;
    a.tile_rows = rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
    a.tile_toks = a.tile_rows / a.part_heads;
    a.planes = (max_q + a.tile_toks - 1) / a.tile_toks;
    const int all = sms * mxq::kv_attn_ctas_per_sm();
    a.ctas = a.planes == 1 ? all : (2 * all + a.planes - 1) / a.planes;
    a.seg_bytes = 0;
    a.bytes = 0;
    if (a.ctas > 1) {  // otherwise no row tile is cut
        a.seg_bytes = align_up(mxq::kv_attn_seg_bytes(a.planes, a.ctas), 256);
        a.bytes = a.seg_bytes +
                  align_up(mxq::kv_attn_partial_bytes(a.planes, a.ctas, a.tile_rows, D), 256);
    }
    return a;
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
    const mxq_status st = mxq::check_current_device(nullptr);
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
    p.status = dev_status;
    const cudaError_t err = mxq::launch_kv_append(p, D, group_size, s);
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
    const mxq_status st = mxq::check_current_device(nullptr);
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
    p.status = dev_status;
    const cudaError_t err = mxq::launch_kv_read(p, D, group_size, s);
    return err == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

size_t mxq_kv_attention_workspace_bytes(int Hq, int Hkv, int D, int max_q_len) {
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0 || max_q_len <= 0) return 0;
    // more SMs never need less, and the longest of shorter rows may need more than
    // many: the largest need over the numbers of rows up to max_q_len
    size_t most = 256;
    for (int n = 1;; n = n < max_q_len / 2 ? 2 * n : max_q_len) {
        const size_t b = plan_attn(Hq, Hkv, D, n, kMaxSms).bytes;
        if (b > most) most = b;
        if (n == max_q_len) return most;
    }
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
    if (T > 0 && S > 0 &&
        (!workspace ||
         workspace_bytes < mxq_kv_attention_workspace_bytes(Hq, Hkv, D, max_q_len)))
        return MXQ_ERR_WORKSPACE;
    int sms = 0;
    const mxq_status st = mxq::check_current_device(&sms);
    if (st != MXQ_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dev_status && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess)
        return MXQ_ERR_CUDA;
    if (T == 0 || S == 0) return MXQ_OK;
    const AttnPlan a = plan_attn(Hq, Hkv, D, max_q_len, sms < kMaxSms ? sms : kMaxSms);
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
    p.head_parts = a.head_parts;
    p.part_heads = a.part_heads;
    p.tile_toks = a.tile_toks;
    p.planes = a.planes;
    p.ctas = a.ctas;
    p.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    p.segs = a.ctas > 1 ? static_cast<int*>(workspace) : nullptr;
    p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + a.seg_bytes);
    p.status = dev_status;
    p.wait_budget = mxq::wait_budget_cycles();
    const cudaError_t err = mxq::launch_kv_attn(p, D, group_size, a.tile_rows, s);
    return err == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

}  // extern "C"
