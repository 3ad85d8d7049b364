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

// Before the other two kernels of a call: its work list and, for tiles of few rows, the rotated
// queries, one warp a row of a tile (rows that no query fills are zeros).  A query is kept as fp16
// over the power of two below its largest element; with SPLIT also what that leaves, as fp16.
template <class E, int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(32 * kJoinWarps)
rotate_queries(const KvAttendParams p, const KvAttendSpace ws) {
    constexpr int N = D / 32, KS = D / 16, R = 8 * NT;
    __shared__ float xs[kJoinWarps][D];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
    uint32_t ent[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        ent[i] = p.ent[lane * N + i];
    pdl_wait();
    if (blockIdx.x == 0 && b == 0 && warp == 0)
        list_units<NarrowForm<NT>>(p, ws);
    const int at = blockIdx.x * kJoinWarps + warp, seg = at / R, r = at % R;
    Seq s;
    const Units un = units_of<NarrowForm<NT>>(p, b, &s, false);
    if (seg >= un.segments)
        return;
    const int row_tiles = un.segments / p.c.kv_heads, kvh = seg / row_tiles;
    const int i0 = (seg - kvh * row_tiles) * R + r;          // of the key head's rows
    float z[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        z[i] = 0.f;
    if (i0 < s.nodes * p.group) {
        const int node = i0 / p.group, e = i0 - node * p.group;
        const E *q = static_cast<const E *>(p.q) + (long long)(s.row0 + node) * p.q_stride +
                     (kvh * p.group + e) * D;
#pragma unroll
        for (int i = 0; i < N; ++i)
            xs[warp][i * 32 + lane] = to_f32(q[i * 32 + lane]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float v = xs[warp][ent[i] & 0x7fffu];
            z[i] = (ent[i] & 0x8000u) ? -v : v;
        }
        warp_wht<D>(z, p.h, lane);
    }
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        big = fmaxf(big, fabsf(z[i]));
#pragma unroll
    for (int k = 16; k; k >>= 1)
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, k));
    // 2^e <= big < 2^(e+1); values over 2^e stay below 2 (2^e and its inverse are normal)
    uint32_t ex = (__float_as_uint(big) >> 23) & 255u;
    ex = ex < 1u ? 1u : (ex > 253u ? 253u : ex);
    const float up = __uint_as_float(ex << 23), down = __uint_as_float((254u - ex) << 23);
    const long long sigma = (long long)b * ws.segments + seg;
    __half *to = reinterpret_cast<__half *>(ws.queries) + sigma * R * D * (SPLIT ? 2 : 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float v = z[i] * down;
        const __half hi = __float2half_rn(v);
        // [row / 8][step][lane][4], lane = 4 (row % 8) + quarter of the row
        const int x = lane * N + i, y = x % (D / 4);
        const int o = (((r >> 3) * KS + (y >> 2)) * 32 + (r & 7) * 4 + x / (D / 4)) * 4 + (y & 3);
        to[o] = hi;
        if constexpr (SPLIT)
            to[R * D + o] = __float2half_rn(v - __half2float(hi));
    }
    if (lane == 0)
        ws.factors[sigma * R + r] = up * p.qk_scale;
}

template <class Form>
__global__ void __launch_bounds__(32) list_work(const KvAttendParams p, const KvAttendSpace ws) {
    pdl_trigger();
    pdl_wait();
    list_units<Form>(p, ws);
}

// One warp a row: o = R^T (sum of its pieces) over the sum of their weights.
template <class E, int D, class Form>
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
    const Units un = units_of<Form>(p, b, &s, false);
    const int row = blockIdx.x * kJoinWarps + warp;          // node * q_heads + head
    const int node = row / p.q_heads, head = row - node * p.q_heads;
    if (un.segments == 0 || node >= s.nodes)
        return;
    const int kvh = head / p.group, at = node * p.group + head - kvh * p.group;
    const int seg = kvh * (un.segments / p.c.kv_heads) + at / Form::rows, r = at % Form::rows;
    const long long U = ws.first[p.B], W = workers_for(U, ws.most, ws.least);
    const long long start = ws.first[b] + (long long)seg * (un.tiles + Form::extra) + Form::extra;
    // the workers that have its first and its last tile
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
    // 32 pieces' factors at a time, a lane each; then their rows, eight under way
    for (int w = w0; w <= w1; w += 32) {
        float f = 0.f;
        if (w + lane <= w1) {
            const float *st = ws.stat + (slot0 + w + lane) * 2 * ws.rows + r;
            f = ex2(st[0] - mx);
            sum += f * st[ws.rows];
        }
        const int n = min(32, w1 - w + 1);
        const float *src = ws.part + ((slot0 + w) * ws.rows + r) * D + lane * N;
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, k);
            const float4 *v4 = reinterpret_cast<const float4 *>(src + (long long)k * ws.rows * D);
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 v = v4[i / 4];
                o[i] += fk * v.x, o[i + 1] += fk * v.y, o[i + 2] += fk * v.z, o[i + 3] += fk * v.w;
            }
        }
    }
#pragma unroll
    for (int k = 16; k; k >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, k);
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

template <int D, class Form>
cudaError_t join(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, cudaStream_t st) {
    const dim3 grid((p.max_nodes * p.q_heads + kJoinWarps - 1) / kJoinWarps, p.B);
    if (dtype == OQ_BF16)
        return launch_pdl(join_pieces<__nv_bfloat16, D, Form>, grid, dim3(32 * kJoinWarps), 0, st,
                          p, ws);
    return launch_pdl(join_pieces<__half, D, Form>, grid, dim3(32 * kJoinWarps), 0, st, p, ws);
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

// A call for tiles of 8 NT rows.
template <int D, int NT>
cudaError_t run_narrow(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                       cudaStream_t st) {
    const dim3 grid(ws.segments * 8 * NT / kJoinWarps, p.B), block(32 * kJoinWarps);
    cudaError_t e =
        dtype == OQ_BF16
            ? launch_pdl(rotate_queries<__nv_bfloat16, D, NT, false>, grid, block, 0, st, p, ws)
            : launch_pdl(rotate_queries<__half, D, NT, true>, grid, block, 0, st, p, ws);
    if (e == cudaSuccess)
        e = launch_narrow(p, ws, dtype, st);
    return e == cudaSuccess ? join<D, NarrowForm<NT>>(p, ws, dtype, st) : e;
}

cudaError_t run_wide(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, cudaStream_t st) {
    cudaError_t e = launch_pdl(list_work<WideForm>, dim3(1), dim3(32), 0, st, p, ws);
    if (e == cudaSuccess)
        e = launch_wide(p, ws, dtype, st);
    return e == cudaSuccess ? join<128, WideForm>(p, ws, dtype, st) : e;
}

// How a call runs: tiles of 128 rows (kv_wide.cuh) for more than 16 rows a key head of 128, else
// of 8 or 16 (kv_attend.cuh); and where its workspace's arrays lie.
struct Plan {
    bool wide;
    int tile;                     // rows of a tile
    size_t stat_at, first_at, queries_at, factors_at, bytes;
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
    const size_t all = (size_t)p.B * a.ws.segments, slots = all + a.ws.most;
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    a.stat_at = up(slots * a.ws.rows * p.c.d * 4);
    a.first_at = a.stat_at + up(slots * a.ws.rows * 8);
    a.queries_at = a.first_at + up((size_t)(p.B + 1) * 8);
    a.factors_at =
        a.queries_at + (a.wide ? 0 : up(all * a.tile * p.c.d * (dtype == OQ_BF16 ? 2 : 4)));
    a.bytes = a.factors_at + (a.wide ? 0 : up(all * a.tile * 4));
    return a;
}

}  // namespace
}  // namespace attend

size_t kv_attend_space(const KvAttendParams &p, int dtype, int num_sms) {
    return attend::plan_for(p, dtype, num_sms).bytes;
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
    a.ws.stat = reinterpret_cast<float *>(w + a.stat_at);
    a.ws.first = reinterpret_cast<long long *>(w + a.first_at);
    a.ws.queries = reinterpret_cast<uint2 *>(w + a.queries_at);
    a.ws.factors = reinterpret_cast<float *>(w + a.factors_at);
    if (a.wide)
        return attend::run_wide(p, a.ws, dtype, st);
    if (p.c.d == 128)
        return a.tile == 8 ? attend::run_narrow<128, 1>(p, a.ws, dtype, st)
                           : attend::run_narrow<128, 2>(p, a.ws, dtype, st);
    return a.tile == 8 ? attend::run_narrow<256, 1>(p, a.ws, dtype, st)
                       : attend::run_narrow<256, 2>(p, a.ws, dtype, st);
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
