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

// Costs, in ns of one SM, by which the parts share the GPU: the tensor cores' kernel takes 2650 for a unit of 256 rows
// and 128 tokens of 128 values, 2400 where 128 rows are shared between its halves (64 rows 2000; of 64 values 2450 and
// 1500, of 256, where a tile is 128 rows, 2800 to 3500); warps on their own, with the GPU for themselves, take 105 for 32 tokens
// of up to 8 rows and 214 of 16, and are reckoned a quarter higher beside the others.  5 prefixes of 5000
// tokens with 20 sequences each of 600 of their own, 16 heads over 4 of 256 values: 53.7 us with 2400, 57.9 with 1700; with 105
// and 214, 57.6, and 256 sequences of 512 tokens after 32768, 40 heads over 8 of 128, 317 instead of 246.
void kv_shared_shape(KvSharedParams& p, int D) {
    if (p.prefix && p.on_tensor_cores) {
        p.tile_shift = 7;
        p.end_units = kEndUnits;
        p.unit_cost = (long long)p.max_group * p.max_q * p.part_heads <= 128 ? 2400 : 2600;
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
