// kv_wide_b3.cu -- the cache's attention for many rows over 3-bit codes (kv_wide.cuh).
#include "kv_wide.cuh"

namespace oq {

cudaError_t launch_kv_wide_b3(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                              cudaStream_t st) {
    return dtype == OQ_BF16 ? attend::launch_wide<__nv_bfloat16, 3>(p, ws, st)
                            : attend::launch_wide<__half, 3>(p, ws, st);
}

}  // namespace oq
