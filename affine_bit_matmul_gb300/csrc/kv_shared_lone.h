// The launch of kv_lone.cuh's kernel for one shape of the cache.
#pragma once

#include "kv_lone.cuh"

namespace mxq {
namespace {

template <int D, int G, int KT1, int KT2>
cudaError_t launch_lone_tiles(const KvSharedParams& prefix, const KvSharedParams& own, cudaStream_t stream) {
    using LB = LoneBoth<D, G, KT1, KT2>;
    static std::atomic<uint64_t> asked{0};  // devices on which the kernel may take its memory
    constexpr auto kernel = kv_lone_kernel<D, G, KT1, KT2>;
    const cudaError_t err = allow_shared(kernel, LB::kSmem, asked);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(own.sms * LB::kCtas));
    cfg.dynamicSmemBytes = LB::kSmem;
    cfg.blockDim = dim3(kLoneThreads);
    cfg.stream = stream;
    // beside the tensor cores' kernel, if there is one; else its blocks are placed while what comes
    // before finishes
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, prefix, own);
}

template <int D, int G>
cudaError_t launch_lone(const KvSharedParams& prefix, const KvSharedParams& own, cudaStream_t stream) {
    const int own_rows = own.tile_rows, rows = prefix.on_tensor_cores ? own_rows : prefix.tile_rows;
    if (rows == own_rows)
        return own_rows == 4   ? launch_lone_tiles<D, G, 1, 1>(prefix, own, stream)
               : own_rows == 8 ? launch_lone_tiles<D, G, 2, 2>(prefix, own, stream)
                               : launch_lone_tiles<D, G, 4, 4>(prefix, own, stream);
    return own_rows == 4 ? launch_lone_tiles<D, G, 4, 1>(prefix, own, stream)
                         : launch_lone_tiles<D, G, 4, 2>(prefix, own, stream);
}

}  // namespace
}  // namespace mxq
