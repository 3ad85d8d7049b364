// kv_internal.h -- parameters of the rotary-position and quantised-cache kernels (rope.cu,
// kv_cache.cu, kv_attend.cu) and their launchers, called by oq_cache.cpp.
#pragma once

#include "oq_internal.h"

namespace oq {

// A kernel's set-up, made once on each device (function attributes belong to a device).
struct PerDevice {
    std::mutex mu;
    bool done[kMaxDevices] = {};
    template <class F> cudaError_t once(F &&f) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess)
            return e;
        if (dev < 0 || dev >= kMaxDevices)
            return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lk(mu);
        if (done[dev])
            return cudaSuccess;
        e = f();
        done[dev] = e == cudaSuccess;
        return e;
    }
};

// Rotary positions of up to two tensors (queries and keys) of the same tokens.
struct RopeParams {
    const void *x[2];
    void *y[2];
    int heads[2];                 // heads[1] = 0: one tensor
    long long x_stride[2], y_stride[2];   // elements between tokens
    const long long *pos;         // [T]
    const double *turns;          // [rot / 2] turns a position
    float amplitude;
    int T, d, rot;
    int inverse;
};
cudaError_t launch_rope(const RopeParams &p, int dtype, int layout, cudaStream_t st, int num_sms,
                        std::string *why);

// The paged cache as the kernels see it: codes [pages, kv_heads, page, row_bytes], norms
// [pages, kv_heads, page]; slot = page index * page + offset.
struct KvView {
    uint8_t *codes[2];            // keys, values
    float *norms[2];
    long long pages;
    int page_log2;
    int kv_heads, d, bits, row_bytes;
};

struct KvWriteParams {
    KvView c;
    const void *x[2];             // keys, values: [T, kv_heads, d]
    long long x_stride[2];
    const long long *slots;       // [T], -1: skip
    int T, h;
    const uint16_t *ent;          // [d] perm | sign bit << 15
    const uint32_t *tbl;          // quantizer grid words (each `tbl_copies` times)
    int tbl_copies, tbl_words;
    const float *bounds;          // the codes' 2^bits - 1 boundaries as fp32, and (2^bits on) the rests
    double unit;                  // sqrt(d / h)
    const void *r_img;            // R' as the tensor cores' operand in x's type (16-bit x)
    int wide;                     // code rows keep 32-byte stores aligned
    unsigned *err;                // device error word (set by launch_kv_write)
    float eps, K;                 // as K1Params
    int G, F;
};
cudaError_t launch_kv_write(const KvWriteParams &p, int dtype, cudaStream_t st, int num_sms,
                            std::string *why);

struct KvReadParams {
    KvView c;
    void *y[2];
    long long y_stride[2];
    const long long *slots;
    int T, h;
    const uint16_t *ent;
    const float *cent;            // fp32 unit centroids (rows kernel)
    float scale;                  // 1 / sqrt(d h): norms times this, on the unnormalised transform
    const void *r_img;            // R'^T as the tensor cores' fp16 operand (16-bit y)
    const uint32_t *lut;          // fp16 decode table (tensor cores)
    float alpha_inv;              // what its centroids are multiplied by, inverted
    unsigned *err;                // device error word (set by launch_kv_read)
};
// The tensor-core forms (kv_tc.cu); p.scale of the read includes alpha_inv.
cudaError_t launch_kv_write_tc(const KvWriteParams &p, const void *r_img, int tbl_words, bool bf16,
                               cudaStream_t st, int num_sms);
cudaError_t launch_kv_read_tc(const KvReadParams &p, const void *r_img, bool bf16, cudaStream_t st,
                              int num_sms);
cudaError_t launch_kv_read(const KvReadParams &p, int dtype, cudaStream_t st, int num_sms,
                           std::string *why);

struct KvAttendParams {
    KvView c;
    const void *q;
    void *out;
    long long q_stride, out_stride;
    int q_heads, group;           // group = q_heads / kv_heads
    long long q_rows;             // rows of q and out
    const int *q_start;           // [B + 1]
    const int *prefix;            // [B]
    const int *table;             // [B, table_width]
    const long long *mask;        // [q_rows] or null
    int B, table_width, max_nodes;
    const uint16_t *ent;
    const uint32_t *lut;          // fp16 decode table (oq_cache.cpp, build_kv_lut)
    int h;
    float qk_scale;               // scale * log2(e) / (sqrt(d h) alpha)
    float o_scale;                // 1 / (sqrt(d h) alpha)
    const void *r_img;            // R' as the tensor cores' operand in bf16 (kv_wide.cuh)
    unsigned *err;                // device error word (set by launch_kv_attend)
};
// Workspace and work list of the forms that share out all tokens evenly (kv_attend_ops.cuh).
struct KvAttendSpace {
    float *part;                  // [slots][rows][d] sums of a piece's rows
    float *stat;                  // [slots][2][rows] references and weights' sums
    long long *first;             // [B + 1] units before each sequence
    uint2 *queries;               // few rows: [segments of all][rows of a tile][d] rotated, as the
                                  // lanes take them (kv_attend.cu, rotate_queries)
    float *factors;               // [segments of all][rows of a tile] of their scores
    int rows;                     // rows of a slot: the tile's, or all a sequence can have
    int segments;                 // segments of a sequence with the most rows
    int most, least;              // workers, and units that one has at least
};
// Many rows a key head, heads of 128, bf16 (kv_wide.cuh).
cudaError_t launch_kv_wide_b2(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st);
cudaError_t launch_kv_wide_b3(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st);
cudaError_t launch_kv_wide_b4(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st);
cudaError_t launch_kv_wide_b6(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st);
cudaError_t launch_kv_wide_b8(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st);
// Few rows a key head, or heads of 256 (kv_attend.cuh): in one launch, a cluster of `splits` CTAs a
// segment, or with splits = 0 by workers (their number on `sms` SMs) with a workspace.
cudaError_t launch_kv_attend_b2(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, int splits, cudaStream_t st);
int kv_attend_workers_b2(const KvAttendParams &p, int sms);
cudaError_t launch_kv_attend_b3(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, int splits, cudaStream_t st);
int kv_attend_workers_b3(const KvAttendParams &p, int sms);
cudaError_t launch_kv_attend_b4(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, int splits, cudaStream_t st);
int kv_attend_workers_b4(const KvAttendParams &p, int sms);
cudaError_t launch_kv_attend_b6(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, int splits, cudaStream_t st);
int kv_attend_workers_b6(const KvAttendParams &p, int sms);
cudaError_t launch_kv_attend_b8(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, int splits, cudaStream_t st);
int kv_attend_workers_b8(const KvAttendParams &p, int sms);
// Device memory that launch_kv_attend needs for a call, 0 for none (given to it as `space`).
size_t kv_attend_space(const KvAttendParams &p, int dtype, int num_sms);
cudaError_t launch_kv_attend(const KvAttendParams &p, void *space, int dtype, cudaStream_t st,
                             int num_sms, std::string *why);

cudaError_t read_and_clear_kv_error(unsigned *out, cudaStream_t st);
cudaError_t read_and_clear_attend_error(unsigned *out, cudaStream_t st);

}  // namespace oq
