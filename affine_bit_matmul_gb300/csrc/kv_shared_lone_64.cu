// Both parts of an attention call over shared prefixes, or the sequences' own tokens, by warps on
// their own: heads of 64 values.
#include "kv_lone.cuh"
#include "kv_shared_lone.h"

namespace mxq {

cudaError_t launch_kv_shared_lone_64(const KvSharedParams& prefix, const KvSharedParams& own, int G,
                                     cudaStream_t stream) {
    if (G == 32) return launch_lone<64, 32>(prefix, own, stream);
    if (G == 64) return launch_lone<64, 64>(prefix, own, stream);
    return cudaErrorInvalidValue;
}

}  // namespace mxq
