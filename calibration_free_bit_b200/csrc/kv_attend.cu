// kv_attend.cu -- launch of the attention over the quantised cache (kernels: kv_attend.cuh, one
// object a bit width) and its device error word.
#include "kv_internal.h"

namespace oq {
namespace {

__device__ unsigned int g_attend_err;

// CTAs that share a row tile's tokens: a cluster.  Enough of them to give every SM a few, but none
// with less than a step for each of its four warps at the longest context the table can hold.
int split_count(const KvAttendParams &p, int num_sms) {
    const int rows = p.max_nodes * p.group, tile = rows <= 8 ? 8 : 16;
    const long long ctas = (long long)p.c.kv_heads * ((rows + tile - 1) / tile) * p.B;
    const long long tokens = (long long)p.table_width << p.c.page_log2;
    int s = 1;
    while (s < 16 && ctas * s < 4ll * num_sms && tokens >= 128ll * s)
        s *= 2;
    return s;
}

}  // namespace

cudaError_t launch_kv_attend(const KvAttendParams &params, int dtype, cudaStream_t st, int num_sms,
                             std::string *why) {
    *why = "oq_kv_attend: launch";
    KvAttendParams p = params;
    static PerDevice known;
    static void *word[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = known.once([&] { return cudaGetSymbolAddress(&word[dev], g_attend_err); });
    if (e != cudaSuccess)
        return e;
    p.err = static_cast<unsigned *>(word[dev]);
    const int s = split_count(p, num_sms);
    switch (p.c.bits) {
    case 2:
        return launch_kv_attend_b2(p, dtype, s, st);
    case 3:
        return launch_kv_attend_b3(p, dtype, s, st);
    case 4:
        return launch_kv_attend_b4(p, dtype, s, st);
    case 6:
        return launch_kv_attend_b6(p, dtype, s, st);
    default:
        return launch_kv_attend_b8(p, dtype, s, st);
    }
}

cudaError_t read_and_clear_attend_error(unsigned *out, cudaStream_t st) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_attend_err, sizeof(unsigned), 0,
                                              cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbolAsync(g_attend_err, &zero, sizeof(unsigned), 0,
                                    cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    return e;
}

}  // namespace oq
