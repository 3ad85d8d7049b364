// kv_wide_b6.cu -- the cache's attention for many rows over 6-bit codes (kv_wide.cuh).
#include "kv_wide.cuh"

namespace oq {

cudaError_t launch_kv_wide_b6(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st) {
    return attend::launch_wide<6>(p, ws, st);
}

}  // namespace oq
