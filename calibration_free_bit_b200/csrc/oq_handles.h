// oq_handles.h -- the handle types behind the C ABI and the host helpers its source files share
// (oq_host.cpp: rotations, codebooks, the linear layer; oq_cache.cpp: rotary positions and the
// quantised cache).  Not part of the public ABI (include/oq.h is).
#pragma once

#include <mutex>
#include <string>
#include <vector>

#include "oq_internal.h"

// ---------------------------------------------------------------------------------------
// Handles.
// ---------------------------------------------------------------------------------------
struct oq_rpbh {
    int d = 0, h = 0;
    uint64_t seed = 0;
    std::vector<int32_t> perm;
    std::vector<int8_t> sign;
    std::vector<uint32_t> ent_img[2];             // K1 gather-entry images: [0] bf16, [1] fp32
    std::vector<uint16_t> ent16;                  // tensor-core K1: perm[i] | sign bit << 15
    std::mutex mu;
    uint32_t *dev_ent[2][oq::kMaxDevices] = {};
    uint32_t *dev_ent16[oq::kMaxDevices] = {};
    // d <= 256: the rotation times sqrt(h) as a dense operand of the tensor cores (oq_cache.cpp,
    // rotation_matrix): [0] bf16, [1] fp16, [2] fp16 transposed
    std::vector<uint16_t> rmat[3];
    uint32_t *dev_rmat[3][oq::kMaxDevices] = {};
};

struct oq_codebook {
    int d = 0, bits = 0, marginal = OQ_MARGINAL_GAUSSIAN;
    std::vector<double> c, t;                     // unit centroids / boundaries
    uint16_t lut[256] = {};                       // unit centroids, fp16 bits
    int G = 0, F = 0;
    double delta = 0.0;
    std::vector<uint32_t> grid;                   // G + 1 words
    std::vector<uint32_t> tbl_img;                // K1 shared-memory image of the table
    std::vector<uint32_t> dec_img;                // K1 fp16 output: byte -> centroids (b 2,4,8)
    std::mutex mu;
    uint32_t *dev_tbl[oq::kMaxDevices] = {};
    uint32_t *dev_dec[oq::kMaxDevices] = {};
    std::vector<float> cent32;                    // the cache: unit centroids, boundaries, and
                                                  // what fp32 leaves of those
    uint32_t *dev_cent32[oq::kMaxDevices] = {};
    // the cache's fp16 decode table (oq_cache.cpp, decode_table: made at its first use): centroids
    // times kv_alpha
    double kv_alpha = 1.0;
    std::vector<uint32_t> kv_lut;
    uint32_t *dev_kv_lut[oq::kMaxDevices] = {};
};

// Rotary positions: frequencies in radians a position, and what both coordinates are multiplied by.
struct oq_rope {
    int rot = 0, layout = OQ_ROPE_HALF;
    double amplitude = 1.0;
    std::vector<double> freq;                     // rot / 2
    std::vector<double> turns;                    // freq / (2 pi), as the kernel reads it
    std::mutex mu;
    uint32_t *dev_turns[oq::kMaxDevices] = {};
};

namespace oq {
namespace host {

// Set the calling thread's oq_last_error text and return `code`.
int fail(int code, const char *fmt, ...);
int fail_cuda(cudaError_t e, const char *what);

struct DeviceInfo {
    int checked = 0;       // 0 unknown, 1 ok, -1 unsupported
    int sms = 0;
    cudaMemPool_t pool = nullptr;
    cudaStream_t side = nullptr;      // oq_quantized_linear: weight decode beside K1
    cudaEvent_t fork = nullptr, join = nullptr;
    uint32_t *gelu_tab = nullptr;     // the fused GELU's table (oq::gelu_table_image)
};
uint16_t to_half_bits(double x);        // IEEE binary16, to nearest even

// The current device, checked once to be sm_100.
int current_device(int *dev_out, DeviceInfo **info_out);

// The device's stream-ordered memory pool (created once; nullptr and *rc set on failure).
cudaMemPool_t device_pool(int dev, DeviceInfo *di, int *rc);

// A handle's table on the current device, copied there at its first use.
template <class T>
int upload(std::mutex &mu, uint32_t **slot, const std::vector<T> &host, const char *what) {
    std::lock_guard<std::mutex> lk(mu);
    if (*slot)
        return OQ_OK;
    void *p = nullptr;
    cudaError_t e = cudaMalloc(&p, host.size() * sizeof(T));
    if (e != cudaSuccess)
        return fail_cuda(e, what);
    e = cudaMemcpy(p, host.data(), host.size() * sizeof(T), cudaMemcpyHostToDevice);
    // a copy from pageable memory may return before it lands, and the caller's stream need not
    // wait for the legacy stream
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(cudaStreamLegacy);
    if (e != cudaSuccess) {
        cudaFree(p);
        return fail_cuda(e, what);
    }
    *slot = static_cast<uint32_t *>(p);
    return OQ_OK;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Optional per-kernel timing (oq_timing_enable / oq_timing_collect): events recorded on the
// caller's stream around every kernel this thread launches through the C ABI.
struct TimedLaunch {
    int kernel;
    cudaEvent_t start, stop;
};
bool timing_on();
cudaEvent_t take_event();
void keep_timed(const TimedLaunch &t);

// Run `launch` (returning cudaError_t), bracketed by events when timing is on.  While the
// stream is being captured into a CUDA graph the events are recorded as external event nodes,
// so each replay of the graph re-records them and they stay readable afterwards.
template <class F>
cudaError_t timed(int kernel, cudaStream_t st, F &&launch) {
    if (!timing_on())
        return launch();
    TimedLaunch t{kernel, take_event(), take_event()};
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    cudaStreamIsCapturing(st, &cs);
    const unsigned flags =
        cs == cudaStreamCaptureStatusActive ? cudaEventRecordExternal : cudaEventRecordDefault;
    if (t.start)
        cudaEventRecordWithFlags(t.start, st, flags);
    cudaError_t e = launch();
    if (t.stop)
        cudaEventRecordWithFlags(t.stop, st, flags);
    if (t.start && t.stop)
        keep_timed(t);
    return e;
}

}  // namespace host
}  // namespace oq
