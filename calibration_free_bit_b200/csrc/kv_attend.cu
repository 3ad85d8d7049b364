// kv_attend.cu -- attention of drafted tokens over the quantised cache.
//
// o = sum_t p_t v_hat_t, p = softmax_t(scale * q . k_hat_t), over the visible cached tokens t of
// the row's sequence: its prefix, and those of its drafted tokens that the row's mask names (bit
// j: node j; without a mask, nodes up to its own).  R is orthogonal, so q . k_hat = (R q) .
// centroid[code] s / sqrt(d), and R^T is applied once, to the finished row.
//
// One warp a row (drafted token, query head), one cached token at a time.
#include <math_constants.h>

#include "kv_internal.h"
#include "kv_ops.cuh"

namespace oq {
namespace {

using namespace kvops;

__device__ unsigned int g_attend_err;

enum : unsigned {
    AT_ERR_ROWS = 1u << 0,      // q_start: decreasing, past the rows given, or over max_nodes
    AT_ERR_LEN = 1u << 1,       // prefix negative, or past the page table
    AT_ERR_PAGE = 1u << 2,      // a page index outside the cache
    AT_ERR_WAIT = 1u << 3,      // a bounded wait gave up
};

// One sequence's rows and lengths; false (with the error recorded) if they are not usable.
struct Seq {
    int row0, nodes, prefix;
};
__device__ __forceinline__ bool load_seq(const KvAttendParams &p, int b, Seq *s, bool tell) {
    const int r0 = p.q_start[b], r1 = p.q_start[b + 1];
    const int prefix = p.prefix[b];
    unsigned err = 0;
    if (r0 < 0 || r1 < r0 || (long long)r1 > p.q_rows || r1 - r0 > p.max_nodes)
        err = AT_ERR_ROWS;
    else if (prefix < 0 || (long long)prefix + (r1 - r0) > ((long long)p.table_width << p.c.page_log2))
        err = AT_ERR_LEN;
    if (err) {
        if (tell)
            atomicOr(&g_attend_err, err);
        return false;
    }
    s->row0 = r0;
    s->nodes = r1 - r0;
    s->prefix = prefix;
    return true;
}

constexpr int kWarps = 4;

template <class E, int D>
__global__ void __launch_bounds__(32 * kWarps) attend_rows(const KvAttendParams p) {
    constexpr int N = D / 32;
    __shared__ float xs[kWarps][D];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ent[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        ent[i] = p.ent[lane * N + i];
    pdl_wait();
    const int b = blockIdx.y;
    const int item = blockIdx.x * kWarps + warp;          // node * q_heads + head
    const int node = item / p.q_heads, head = item - node * p.q_heads;
    Seq s;
    if (!load_seq(p, b, &s, blockIdx.x == 0 && threadIdx.x == 0) || node >= s.nodes)
        return;
    const long long row = s.row0 + node;
    const int kvh = head / p.group;
    const E *q = static_cast<const E *>(p.q) + row * p.q_stride + head * D;
#pragma unroll
    for (int i = 0; i < N; ++i)
        xs[warp][i * 32 + lane] = to_f32(q[i * 32 + lane]);
    __syncwarp();
    float z[N], o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float v = xs[warp][ent[i] & 0x7fffu];
        z[i] = ((ent[i] & 0x8000u) ? -v : v);
        o[i] = 0.f;
    }
    warp_wht<D>(z, p.h, lane);
    const unsigned long long mask =
        p.mask ? (unsigned long long)p.mask[row] : (2ull << node) - 1ull;
    float m = -CUDART_INF_F, l = 0.f;
    for (int t = 0; t < s.prefix + s.nodes; ++t) {
        if (t >= s.prefix && !((mask >> (t - s.prefix)) & 1ull))
            continue;
        const int page = p.table[(long long)b * p.table_width + (t >> p.c.page_log2)];
        if (page < 0 || page >= p.c.pages) {
            if (lane == 0)
                atomicOr(&g_attend_err, AT_ERR_PAGE);
            continue;
        }
        const long long at = (((long long)page * p.c.kv_heads + kvh) << p.c.page_log2) +
                             (t & ((1 << p.c.page_log2) - 1));
        const uint8_t *kr = p.c.codes[0] + at * p.c.row_bytes;
        const uint8_t *vr = p.c.codes[1] + at * p.c.row_bytes;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            dot += z[i] * p.cent[code_at(kr, lane * N + i, p.c.bits)];
#pragma unroll
        for (int k = 16; k; k >>= 1)
            dot += __shfl_xor_sync(0xffffffffu, dot, k);
        const float x = dot * p.c.norms[0][at] * p.qk_scale;
        const float mn = fmaxf(m, x);
        const float c = exp2f(m - mn), e = exp2f(x - mn);
        m = mn;
        l = l * c + e;
        const float ev = e * p.c.norms[1][at];
#pragma unroll
        for (int i = 0; i < N; ++i)
            o[i] = o[i] * c + ev * p.cent[code_at(vr, lane * N + i, p.c.bits)];
    }
    warp_wht<D>(o, p.h, lane);
    const float inv = l > 0.f ? p.o_scale / l : 0.f;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i)
        xs[warp][ent[i] & 0x7fffu] = inv * ((ent[i] & 0x8000u) ? -o[i] : o[i]);
    __syncwarp();
    E *y = static_cast<E *>(p.out) + row * p.out_stride + head * D;
#pragma unroll
    for (int i = 0; i < N; ++i)
        y[i * 32 + lane] = from_f32<E>(xs[warp][i * 32 + lane]);
}

template <class E>
cudaError_t run(const KvAttendParams &p, cudaStream_t st) {
    const dim3 grid((p.max_nodes * p.q_heads + kWarps - 1) / kWarps, p.B), block(32 * kWarps);
    if (p.c.d == 128)
        return launch_pdl(attend_rows<E, 128>, grid, block, 0, st, p);
    return launch_pdl(attend_rows<E, 256>, grid, block, 0, st, p);
}

}  // namespace

cudaError_t launch_kv_attend(const KvAttendParams &p, int dtype, cudaStream_t st, int num_sms,
                             std::string *why) {
    *why = "oq_kv_attend: launch";
    if (dtype == OQ_BF16)
        return run<__nv_bfloat16>(p, st);
    return run<__half>(p, st);
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
