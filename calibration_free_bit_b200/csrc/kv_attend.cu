// kv_attend.cu -- launch of the attention over the quantised cache: which form a call takes
// (kv_attend.cuh, kv_wide.cuh; an object for each bit width), the kernel that joins a segment's
// pieces, and the device error word.
#include "kv_attend_ops.cuh"
#include "kv_internal.h"

namespace oq {
namespace attend {
namespace {

__device__ unsigned int g_attend_err;

constexpr int kJoinWarps = 4;

// One warp a row: o = R^T (sum of its pieces) over the sum of their weights.
template <class E, int D, int TOKENS, int ROWS>
__global__ void __launch_bounds__(32 * kJoinWarps)
join_pieces(const KvAttendParams p, const KvAttendSpace ws) {
    constexpr int N = D / 32;
    __shared__ float xs[kJoinWarps][D];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
    uint32_t ent[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        ent[i] = p.ent[lane * N + i];
    pdl_wait();
    Seq s;
    const Units un = units_of<TOKENS, ROWS>(p, b, &s, false);
    const int row = blockIdx.x * kJoinWarps + warp;          // node * q_heads + head
    const int node = row / p.q_heads, head = row - node * p.q_heads;
    if (un.segments == 0 || node >= s.nodes)
        return;
    const int kvh = head / p.group, at = node * p.group + head - kvh * p.group;
    const int seg = kvh * (un.segments / p.c.kv_heads) + at / ROWS, r = at % ROWS;
    const long long U = ws.first[p.B], W = workers_for(U, ws.most, ws.least);
    const long long start = ws.first[b] + (long long)seg * un.tiles;
    // the workers that have its first and its last unit
    const int w0 = (int)(((start + 1) * W - 1) / U);
    const int w1 = (int)(((start + un.tiles) * W - 1) / U);
    const long long slot0 = (long long)b * ws.segments + seg;
    float mx = kNone;
    for (int w = w0 + lane; w <= w1; w += 32)
        mx = fmaxf(mx, ws.stat[(slot0 + w) * 2 * ws.rows + r]);
#pragma unroll
    for (int k = 16; k; k >>= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    float o[N], sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        o[i] = 0.f;
#pragma unroll 4
    for (int w = w0; w <= w1; ++w) {
        const float *st = ws.stat + (slot0 + w) * 2 * ws.rows + r;
        const float f = ex2(st[0] - mx);
        sum += f * st[ws.rows];
        const float4 *src = reinterpret_cast<const float4 *>(
            ws.part + ((slot0 + w) * ws.rows + r) * D + lane * N);
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = src[i / 4];
            o[i] += f * v.x, o[i + 1] += f * v.y, o[i + 2] += f * v.z, o[i + 3] += f * v.w;
        }
    }
    warp_wht<D>(o, p.h, lane);
    const float inv = sum == 0.f ? 0.f : p.o_scale / sum;    // nothing seen: zeros
#pragma unroll
    for (int i = 0; i < N; ++i)
        xs[warp][ent[i] & 0x7fffu] = inv * ((ent[i] & 0x8000u) ? -o[i] : o[i]);
    __syncwarp();
    E *y = static_cast<E *>(p.out) + (s.row0 + node) * p.out_stride + head * D;
#pragma unroll
    for (int i = 0; i < N; ++i)
        y[i * 32 + lane] = from_f32<E>(xs[warp][i * 32 + lane]);
}

template <int D, int TOKENS, int ROWS>
cudaError_t join(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, cudaStream_t st) {
    const dim3 grid((p.max_nodes * p.q_heads + kJoinWarps - 1) / kJoinWarps, p.B);
    if (dtype == OQ_BF16)
        return launch_pdl(join_pieces<__nv_bfloat16, D, TOKENS, ROWS>, grid, dim3(32 * kJoinWarps),
                          0, st, p, ws);
    return launch_pdl(join_pieces<__half, D, TOKENS, ROWS>, grid, dim3(32 * kJoinWarps), 0, st, p,
                      ws);
}

#define OQ_BY_BITS(bits, call)  \
    switch (bits) {             \
    case 2:                     \
        return call(2);         \
    case 3:                     \
        return call(3);         \
    case 4:                     \
        return call(4);         \
    case 6:                     \
        return call(6);         \
    default:                    \
        return call(8);         \
    }

int narrow_workers(const KvAttendParams &p, int dtype, int sms) {
#define OQ_CALL(B) kv_attend_workers_b##B(p, dtype, sms)
    OQ_BY_BITS(p.c.bits, OQ_CALL)
#undef OQ_CALL
}
cudaError_t launch_narrow(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                          cudaStream_t st) {
#define OQ_CALL(B) launch_kv_attend_b##B(p, ws, dtype, st)
    OQ_BY_BITS(p.c.bits, OQ_CALL)
#undef OQ_CALL
}
cudaError_t launch_wide(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                        cudaStream_t st) {
#define OQ_CALL(B) launch_kv_wide_b##B(p, ws, dtype, st)
    OQ_BY_BITS(p.c.bits, OQ_CALL)
#undef OQ_CALL
}

// How a call runs: tiles of 128 rows (kv_wide.cuh) for more than 16 rows a key head of 128, else
// of 8 or 16 (kv_attend.cuh).
struct Plan {
    bool wide;
    int tile;                     // rows of a tile
    long long slots;              // of the workspace
    KvAttendSpace ws;
};

Plan plan_for(const KvAttendParams &p, int dtype, int num_sms) {
    Plan a = {};
    const int rows = p.max_nodes * p.group;
    a.wide = p.c.d == 128 && rows > 16;
    a.tile = a.wide ? 128 : rows <= 8 ? 8 : 16;
    a.ws.rows = rows < a.tile ? rows : a.tile;
    a.ws.segments = p.c.kv_heads * ((rows + a.tile - 1) / a.tile);
    a.ws.most = a.wide ? num_sms : narrow_workers(p, dtype, num_sms);
    // a wide worker is an SM, a narrow one a warp, which should not be set up for less than this
    a.ws.least = a.wide ? 1 : 4;
    a.slots = (long long)p.B * a.ws.segments + a.ws.most;
    return a;
}

}  // namespace
}  // namespace attend

size_t kv_attend_space(const KvAttendParams &p, int dtype, int num_sms) {
    const attend::Plan a = attend::plan_for(p, dtype, num_sms);
    return KvAttendSpace::first_at(a.slots, a.ws.rows, p.c.d) + (size_t)(p.B + 1) * 8;
}

cudaError_t launch_kv_attend(const KvAttendParams &params, void *space, int dtype, cudaStream_t st,
                             int num_sms, std::string *why) {
    *why = "oq_kv_attend: launch";
    KvAttendParams p = params;
    static PerDevice known;
    static void *word[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = known.once([&] { return cudaGetSymbolAddress(&word[dev], attend::g_attend_err); });
    if (e != cudaSuccess)
        return e;
    p.err = static_cast<unsigned *>(word[dev]);
    attend::Plan a = attend::plan_for(p, dtype, num_sms);
    char *w = static_cast<char *>(space);
    a.ws.part = reinterpret_cast<float *>(w);
    a.ws.stat = reinterpret_cast<float *>(w + KvAttendSpace::stat_at(a.slots, a.ws.rows, p.c.d));
    a.ws.first =
        reinterpret_cast<long long *>(w + KvAttendSpace::first_at(a.slots, a.ws.rows, p.c.d));
    if (a.wide) {
        e = attend::launch_wide(p, a.ws, dtype, st);
        return e != cudaSuccess ? e : attend::join<128, 128, 128>(p, a.ws, dtype, st);
    }
    if ((e = attend::launch_narrow(p, a.ws, dtype, st)) != cudaSuccess)
        return e;
    if (p.c.d == 128)
        return a.tile == 8 ? attend::join<128, 16, 8>(p, a.ws, dtype, st)
                           : attend::join<128, 16, 16>(p, a.ws, dtype, st);
    return a.tile == 8 ? attend::join<256, 16, 8>(p, a.ws, dtype, st)
                       : attend::join<256, 16, 16>(p, a.ws, dtype, st);
}

cudaError_t read_and_clear_attend_error(unsigned *out, cudaStream_t st) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, attend::g_attend_err, sizeof(unsigned), 0,
                                              cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbolAsync(attend::g_attend_err, &zero, sizeof(unsigned), 0,
                                    cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    return e;
}

}  // namespace oq
