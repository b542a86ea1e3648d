// Both parts of an attention call over shared prefixes, or the sequences' own tokens, by warps on
// their own: heads of 128 values.
#include "kv_lone.cuh"
#include "kv_shared_lone.h"

namespace mxq {

cudaError_t launch_kv_shared_lone_128(const KvSharedParams& prefix, const KvSharedParams& own, int G,
                                     cudaStream_t stream) {
    if (G == 32) return launch_lone<128, 32>(prefix, own, stream);
    if (G == 64) return launch_lone<128, 64>(prefix, own, stream);
    if (G == 128) return launch_lone<128, 128>(prefix, own, stream);
    return cudaErrorInvalidValue;
}

}  // namespace mxq
