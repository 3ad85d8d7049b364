// kv_attend_b4.cu -- the cache's attention over 4-bit codes (kv_attend.cuh).
#include "kv_attend.cuh"

namespace oq {

cudaError_t launch_kv_attend_b4(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                                int splits, cudaStream_t st) {
    return attend::launch_bits<4>(p, ws, dtype, splits, st);
}

int kv_attend_workers_b4(const KvAttendParams &p, int sms) {
    return attend::workers_bits<4>(p, sms);
}

}  // namespace oq
