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

// How a call runs.
struct Plan {
    bool wide = false;            // kv_wide.cuh and a join; else kv_attend.cuh
    int splits = 1;               // kv_attend.cuh: CTAs that share a row tile's tokens
    long long slots = 0;          // wide: the workspace's
    KvAttendSpace ws = {};
};

Plan plan_for(const KvAttendParams &p, int num_sms) {
    Plan a;
    const int rows = p.max_nodes * p.group;
    const long long tokens = (long long)p.table_width << p.c.page_log2;
    if (p.c.d == 128 && rows > 16) {
        a.ws.rows = rows < 128 ? rows : 128;
        a.ws.segments = p.c.kv_heads * ((rows + 127) / 128);
        a.ws.most = num_sms;
        a.ws.least = 1;
        a.slots = (long long)p.B * a.ws.segments + a.ws.most;
        // a workspace of this size at most (its slots go with the sequences, used or not)
        a.wide = a.slots * a.ws.rows * 128 * 4 <= (1ll << 30);
        if (a.wide)
            return a;
    }
    // Enough CTAs to give every SM a few, but none with less than two steps for each of its
    // warps at the longest context the table can hold.
    const int tile = rows <= 8 ? 8 : 16;
    const long long ctas = (long long)p.c.kv_heads * ((rows + tile - 1) / tile) * p.B;
    while (a.splits < 16 && ctas * a.splits < 4ll * num_sms && tokens >= 128ll * a.splits)
        a.splits *= 2;
    return a;
}

}  // namespace
}  // namespace attend

cudaError_t launch_kv_wide(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                           cudaStream_t st) {
    switch (p.c.bits) {
    case 2:
        return launch_kv_wide_b2(p, ws, dtype, st);
    case 3:
        return launch_kv_wide_b3(p, ws, dtype, st);
    case 4:
        return launch_kv_wide_b4(p, ws, dtype, st);
    case 6:
        return launch_kv_wide_b6(p, ws, dtype, st);
    default:
        return launch_kv_wide_b8(p, ws, dtype, st);
    }
}

size_t kv_attend_space(const KvAttendParams &p, int num_sms) {
    const attend::Plan a = attend::plan_for(p, num_sms);
    if (!a.wide)
        return 0;
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
    attend::Plan a = attend::plan_for(p, num_sms);
    if (a.wide) {
        char *w = static_cast<char *>(space);
        a.ws.part = reinterpret_cast<float *>(w);
        a.ws.stat = reinterpret_cast<float *>(w + KvAttendSpace::stat_at(a.slots, a.ws.rows, 128));
        a.ws.first =
            reinterpret_cast<long long *>(w + KvAttendSpace::first_at(a.slots, a.ws.rows, 128));
        e = launch_kv_wide(p, a.ws, dtype, st);
        return e != cudaSuccess ? e : attend::join<128, 128, 128>(p, a.ws, dtype, st);
    }
    switch (p.c.bits) {
    case 2:
        return launch_kv_attend_b2(p, dtype, a.splits, st);
    case 3:
        return launch_kv_attend_b3(p, dtype, a.splits, st);
    case 4:
        return launch_kv_attend_b4(p, dtype, a.splits, st);
    case 6:
        return launch_kv_attend_b6(p, dtype, a.splits, st);
    default:
        return launch_kv_attend_b8(p, dtype, a.splits, st);
    }
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
