// kv_attend_b3.cu -- the cache's attention over 3-bit codes (kv_attend.cuh).
#include "kv_attend.cuh"

namespace oq {

cudaError_t launch_kv_attend_b3(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                                int splits, cudaStream_t st) {
    return attend::launch_bits<3>(p, ws, dtype, splits, st);
}

int kv_attend_workers_b3(const KvAttendParams &p, int sms) {
    return attend::workers_bits<3>(p, sms);
}

}  // namespace oq
