// kv_attend_b2.cu -- the cache's attention over 2-bit codes (kv_attend.cuh).
#include "kv_attend.cuh"

namespace oq {

cudaError_t launch_kv_attend_b2(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                                int splits, cudaStream_t st) {
    return attend::launch_bits<2>(p, ws, dtype, splits, st);
}

int kv_attend_workers_b2(const KvAttendParams &p, int sms) {
    return attend::workers_bits<2>(p, sms);
}

}  // namespace oq
