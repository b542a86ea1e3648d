// The choice of kv_lone.cuh's kernel by the size of the heads, and the shapes of both parts.
#include "kv_many.cuh"
#include "mxq_internal.h"

namespace mxq {

cudaError_t launch_kv_shared_lone_64(const KvSharedParams&, const KvSharedParams&, int, cudaStream_t);
cudaError_t launch_kv_shared_lone_128(const KvSharedParams&, const KvSharedParams&, int, cudaStream_t);
cudaError_t launch_kv_shared_lone_256(const KvSharedParams&, const KvSharedParams&, int, cudaStream_t);

cudaError_t launch_kv_shared_lone(const KvSharedParams& prefix, const KvSharedParams& own, int D, int G,
                                  cudaStream_t stream) {
    return D == 64    ? launch_kv_shared_lone_64(prefix, own, G, stream)
           : D == 128 ? launch_kv_shared_lone_128(prefix, own, G, stream)
                      : launch_kv_shared_lone_256(prefix, own, G, stream);
}

// Costs are ns of one SM: the tensor cores' kernel takes some 2600 for a unit of 256 rows and 128
// tokens of 128 values, 1700 where 128 rows are shared between its halves; warps on their own, for
// 32 tokens, are bound by the memory with few rows, 110, and by their instructions with 16, 260.
void kv_shared_shape(KvSharedParams& p, int D) {
    if (p.prefix && p.on_tensor_cores) {
        p.tile_shift = 7;
        p.end_units = kEndUnits;
        p.unit_cost = (long long)p.max_group * p.max_q * p.part_heads <= 128 ? 1700 : 2600;
        p.least_run = 1;
        return;
    }
    // (tiles of 16 tokens for heads of 256)
    p.tile_shift = D == 256 ? 4 : 5;
    p.end_units = D == 256 ? 4 : p.tile_rows == 16 ? 2 : 3;
    p.unit_cost = p.tile_rows == 16 ? 260 : p.tile_rows == 8 ? 150 : 130;
    p.least_run = D == 256 ? 4 : 2;
}

}  // namespace mxq
