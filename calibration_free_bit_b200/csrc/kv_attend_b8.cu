// kv_attend_b8.cu -- the cache's attention over 8-bit codes (kv_attend.cuh).
#include "kv_attend.cuh"

namespace oq {

cudaError_t launch_kv_attend_b8(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                                int splits, cudaStream_t st) {
    return attend::launch_bits<8>(p, ws, dtype, splits, st);
}

int kv_attend_workers_b8(const KvAttendParams &p, int sms) {
    return attend::workers_bits<8>(p, sms);
}

}  // namespace oq
