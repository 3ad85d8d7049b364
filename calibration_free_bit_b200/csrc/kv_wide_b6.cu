// kv_wide_b6.cu -- the cache's attention for many rows over 6-bit codes (kv_wide.cuh).
#include "kv_wide.cuh"

namespace oq {

cudaError_t launch_kv_wide_b6(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                              cudaStream_t st) {
    return dtype == OQ_BF16 ? attend::launch_wide<__nv_bfloat16, 6>(p, ws, st)
                            : attend::launch_wide<__half, 6>(p, ws, st);
}

}  // namespace oq
