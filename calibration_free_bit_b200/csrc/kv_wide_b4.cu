// kv_wide_b4.cu -- the cache's attention for many rows over 4-bit codes (kv_wide.cuh).
#include "kv_wide.cuh"

namespace oq {

cudaError_t launch_kv_wide_b4(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st) {
    return attend::launch_wide<4>(p, ws, st);
}

}  // namespace oq
