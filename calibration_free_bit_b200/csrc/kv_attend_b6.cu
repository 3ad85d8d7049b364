// kv_attend_b6.cu -- the cache's attention over 6-bit codes (kv_attend.cuh).
#include "kv_attend.cuh"

namespace oq {

cudaError_t launch_kv_attend_b6(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                                int splits, cudaStream_t st) {
    return attend::launch_bits<6>(p, ws, dtype, splits, st);
}

int kv_attend_workers_b6(const KvAttendParams &p, int sms) {
    return attend::workers_bits<6>(p, sms);
}

}  // namespace oq
