// One part of an attention call over shared prefixes by the kernel for few rows.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_few.cuh"

namespace mxq {
namespace {

template <int D, int G, int KT>
cudaError_t launch(KvSharedParams& p, bool dependent, cudaStream_t stream) {
    using SH = Shape<D, G, KT>;
    static std::atomic<uint64_t> asked{0};  // devices on which the kernel may take its memory
    cudaError_t err = allow_shared(kv_attn_kernel<D, G, KT, KvSharedParams>, SH::kSmem, asked);
    if (err != cudaSuccess) return err;
    p.tile_tokens = SH::kTile;
    p.end_units = kEndTokens / SH::kTile;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.ctas);
    cfg.blockDim = dim3(SH::kThreads);
    cfg.dynamicSmemBytes = SH::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kv_attn_kernel<D, G, KT, KvSharedParams>, p);
}

}  // namespace

cudaError_t launch_kv_shared_part(KvSharedParams& p, int D, int G, bool dependent,
                                  cudaStream_t stream) {
    if (p.tile_rows > 16) return launch_kv_shared_many(p, D, G, stream);
#define MXQ_KV_SHARED(d, g)                                                 \
    if (D == d && G == g)                                                   \
        return p.tile_rows <= 4   ? launch<d, g, 1>(p, dependent, stream)   \
               : p.tile_rows <= 8 ? launch<d, g, 2>(p, dependent, stream)   \
                                  : launch<d, g, 4>(p, dependent, stream);
    MXQ_KV_SHARED(64, 32)
    MXQ_KV_SHARED(64, 64)
    MXQ_KV_SHARED(128, 32)
    MXQ_KV_SHARED(128, 64)
    MXQ_KV_SHARED(128, 128)
    MXQ_KV_SHARED(256, 32)
    MXQ_KV_SHARED(256, 64)
    MXQ_KV_SHARED(256, 128)
#undef MXQ_KV_SHARED
    return cudaErrorInvalidValue;
}

}  // namespace mxq
