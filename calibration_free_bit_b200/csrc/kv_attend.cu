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
// Rows of a call from which a joining warp takes four rows.  It and four warps a row, us: 64 sequences of
// 2000 tokens, 2048 rows 58 and 54, 128 sequences 91 and 92, 512 of 500 tokens 113 and 131; 16 sequences
// with 31 nodes, 15872 rows 63 and 84.
constexpr int kManyRows = 4096;
// Tiles of 16 tokens, over all segments, up to which clusters take a call: tiles of 8 rows of 128 (two
// CTAs an SM), others.  They are counted by what the page tables can hold, since lengths are on the
// device: the figures are of tables as wide as the lengths, and a sequence of 4096 tokens in a table for
// 131072 is a call for workers (18.9 us).  Clusters and workers, us, bf16: 8 key heads, a sequence of 4096 tokens 11 and
// 19, 32768 30 and 46, 65536 51 and 55, 131072 93 and 74, 16 of 4000 tokens 29 and 33; with 16 rows
// 16000 tokens 27 and 32, 32000 44 and 37, 4 sequences of 4000 27 and 25.
constexpr long long kNearTiles = 32768, kNearOther = 8192;
// Rows of a key head from which a call is the tensor memory's (kv_wide.cuh).  It and the tiles of 16
// rows, us, 8 key heads, 4 bits: 32 rows, 32 sequences of 4000 tokens 147 and 120, one of 4000 22 and
// 19; 48 rows 149 and 169, and 23 and 20; 64 rows, 8 sequences 56 and 72; 128 rows 61 and 120.
constexpr int kWideRows = 33;

// Before the other two kernels of a call with few rows: its work list and the rotated queries, one
// warp a row of a tile (rows that no query fills are zeros).
template <class E, int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(32 * kJoinWarps)
rotate_queries(const KvAttendParams p, const KvAttendSpace ws) {
    constexpr int N = D / 32, R = 8 * NT;
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
    const int i = (seg - kvh * row_tiles) * R + r;           // of the key head's rows
    const long long sigma = (long long)b * ws.segments + seg;
    const float f = rotate_row<E, D, SPLIT>(
        p, s, kvh, i, i < s.nodes * p.group, ent, xs[warp], r, NT,
        reinterpret_cast<__half *>(ws.queries) + sigma * R * D * (SPLIT ? 2 : 1));
    if (lane == 0)
        ws.factors[sigma * R + r] = f;
}

template <class Form>
__global__ void __launch_bounds__(32) list_work(const KvAttendParams p, const KvAttendSpace ws) {
    pdl_trigger();
    pdl_wait();
    list_units<Form>(p, ws);
}

// The sum of a row's pieces, and of their weights, in a fixed order.  Where there are few rows, each has
// many pieces: four warps a row take every fourth.  Where there are many, a warp takes ROWS rows of one
// tile in turn, for which the search for their pieces is the same.
template <class E, int D, class Form, int WARPS, int ROWS>
__global__ void __launch_bounds__(32 * kJoinWarps)
join_pieces(const KvAttendParams p, const KvAttendSpace ws) {
    static_assert(Form::rows % ROWS == 0, "a warp's rows are in one tile");
    constexpr int N = D / 32, per = kJoinWarps / WARPS * ROWS;
    __shared__ float4 sums[kJoinWarps][D / 4];
    __shared__ float totals[kJoinWarps];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
    const int chunks = (p.max_nodes * p.group + per - 1) / per, kvh = blockIdx.x / chunks;
    const int at = (blockIdx.x - kvh * chunks) * per + warp / WARPS * ROWS;
    uint32_t ent[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        ent[i] = p.ent[lane * N + i];
    pdl_wait();
    Seq s;
    const long long U = ws.first[p.B], first = ws.first[b];
    const Units un = units_of<Form>(p, b, &s, false);
    const int rows = un.segments > 0 ? min(ROWS, s.nodes * p.group - at) : 0;
    if (WARPS == 1 && rows <= 0)
        return;
    float o[ROWS][N], sum[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        sum[j] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            o[j][i] = 0.f;
    }
    if (rows > 0) {
        const int seg = kvh * (un.segments / p.c.kv_heads) + at / Form::rows, r = at % Form::rows;
        const long long W = workers_for(U, ws.most, ws.least);
        const long long start = first + (long long)seg * (un.tiles + Form::extra) + Form::extra;
        // the workers that have its first and its last tile
        const int w0 = (int)(((start + 1) * W - 1) / U);
        const int w1 = (int)(((start + un.tiles) * W - 1) / U);
        const long long slot0 = (long long)b * ws.segments + seg;
        float mx[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
            mx[j] = kNone;
        if constexpr (WARPS > 1) {
            for (int w = w0 + lane; w <= w1; w += 32)
                mx[0] = fmaxf(mx[0], ws.stat[(slot0 + w) * 2 * ws.rows + r]);
#pragma unroll
            for (int k = 16; k; k >>= 1)
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], k));
        } else {
            for (int w = w0; w <= w1; ++w)
#pragma unroll
                for (int j = 0; j < ROWS; ++j)
                    if (j < rows)
                        mx[j] = fmaxf(mx[j], ws.stat[(slot0 + w) * 2 * ws.rows + r + j]);
        }
#pragma unroll(WARPS > 1 ? 4 : 1)
        for (int w = w0 + warp % WARPS; w <= w1; w += WARPS) {
            const float *st = ws.stat + (slot0 + w) * 2 * ws.rows + r;
            const float4 *src = reinterpret_cast<const float4 *>(
                ws.part + ((slot0 + w) * ws.rows + r) * D + lane * N);
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                if (j >= rows)
                    continue;
                const float f = ex2(st[j] - mx[j]);
                sum[j] += f * st[ws.rows + j];
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    const float4 v = src[j * (D / 4) + i / 4];
                    o[j][i] += f * v.x, o[j][i + 1] += f * v.y;
                    o[j][i + 2] += f * v.z, o[j][i + 3] += f * v.w;
                }
            }
        }
    }
    if constexpr (WARPS > 1) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            sums[warp][lane * (N / 4) + i / 4] =
                make_float4(o[0][i], o[0][i + 1], o[0][i + 2], o[0][i + 3]);
        if (lane == 0)
            totals[warp] = sum[0];
        __syncthreads();
        if (warp % WARPS > 0 || rows <= 0)
            return;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
            sum[0] += totals[warp + w];
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 v = sums[warp + w][lane * (N / 4) + i / 4];
                o[0][i] += v.x, o[0][i + 1] += v.y, o[0][i + 2] += v.z, o[0][i + 3] += v.w;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
        if (j < rows)
            finish_row<E, D>(p, s, kvh, at + j, ent, reinterpret_cast<float *>(sums[warp]), o[j],
                             sum[j]);
}

template <class E, int D, class Form, int WARPS, int ROWS>
cudaError_t join_with(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st) {
    constexpr int per = kJoinWarps / WARPS * ROWS;
    const int chunks = (p.max_nodes * p.group + per - 1) / per;
    return launch_pdl(join_pieces<E, D, Form, WARPS, ROWS>, dim3(p.c.kv_heads * chunks, p.B),
                      dim3(32 * kJoinWarps), 0, st, p, ws);
}
template <class E, int D, class Form>
cudaError_t join_as(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st) {
    if ((long long)p.max_nodes * p.q_heads * p.B >= kManyRows)
        return join_with<E, D, Form, 1, 4>(p, ws, st);
    return join_with<E, D, Form, kJoinWarps, 1>(p, ws, st);
}

template <int D, class Form>
cudaError_t join(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, cudaStream_t st) {
    return dtype == OQ_BF16 ? join_as<__nv_bfloat16, D, Form>(p, ws, st)
                            : join_as<__half, D, Form>(p, ws, st);
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

int narrow_workers(const KvAttendParams &p, int sms) {
#define OQ_CALL(B) kv_attend_workers_b##B(p, sms)
    OQ_BY_BITS(p.c.bits, OQ_CALL)
#undef OQ_CALL
}
cudaError_t launch_narrow(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, int splits,
                          cudaStream_t st) {
#define OQ_CALL(B) launch_kv_attend_b##B(p, ws, dtype, splits, st)
    OQ_BY_BITS(p.c.bits, OQ_CALL)
#undef OQ_CALL
}
cudaError_t launch_wide(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st) {
#define OQ_CALL(B) launch_kv_wide_b##B(p, ws, st)
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
        e = launch_narrow(p, ws, dtype, 0, st);
    return e == cudaSuccess ? join<D, NarrowForm<NT>>(p, ws, dtype, st) : e;
}

cudaError_t run_wide(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st) {
    cudaError_t e = launch_pdl(list_work<WideForm>, dim3(1), dim3(32), 0, st, p, ws);
    if (e == cudaSuccess)
        e = launch_wide(p, ws, st);
    return e == cudaSuccess ? join_as<__nv_bfloat16, 128, WideForm>(p, ws, st) : e;
}

// How a call runs: tiles of 128 rows (kv_wide.cuh) for many rows a key head of 128, else of 8 or, of
// heads of 128, 16 (kv_attend.cuh), the latter by clusters where all tokens that the page tables can
// hold are little work; and where its workspace's arrays lie.  fp16 stays with the small tiles: its
// outputs are eight times as fine as bf16's, and one fp16 number for each element of a query, a key and
// a weight, as the large tiles have them, left an error of 1.2e-3 where the output's rounding is 2.1e-4.
struct Plan {
    bool wide;
    int tile;                     // rows of a tile
    int splits;                   // of a cluster; 0: workers
    size_t stat_at, first_at, queries_at, factors_at, bytes;
    KvAttendSpace ws;
};

Plan plan_for(const KvAttendParams &p, int dtype, int num_sms) {
    Plan a = {};
    const int rows = p.max_nodes * p.group;
    a.wide = p.c.d == 128 && dtype == OQ_BF16 && rows >= kWideRows;
    a.tile = a.wide ? 128 : rows <= 8 || p.c.d == 256 ? 8 : 16;
    a.ws.rows = rows < a.tile ? rows : a.tile;
    a.ws.segments = p.c.kv_heads * ((rows + a.tile - 1) / a.tile);
    const long long all = (long long)p.B * a.ws.segments;
    const long long tokens = (long long)p.table_width << p.c.page_log2;
    const bool two = a.tile == 8 && p.c.d == 128;        // CTAs an SM, of attend_near
    if (!a.wide && all <= num_sms && all * tokens <= 16 * (two ? kNearTiles : kNearOther)) {
        // all CTAs at once, and a tile for every warp (one CTA an SM: clusters do not fill every part
        // of the GPU, and 128 CTAs in clusters of 8 took 21 us, 64 in clusters of 4 12)
        const long long room = two ? 2 * num_sms : num_sms * 3 / 4;
        a.splits = 1;
        while (a.splits < 16 && all * a.splits * 2 <= room && tokens >= 256ll * a.splits)
            a.splits *= 2;
        return a;
    }
    a.ws.most = a.wide ? num_sms : narrow_workers(p, num_sms);
    // a wide worker is an SM, a narrow one a warp, which should not be set up for less than this
    a.ws.least = a.wide ? 1 : 4;
    const size_t slots = (size_t)all + a.ws.most;
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    a.stat_at = up(slots * a.ws.rows * p.c.d * 4);
    a.first_at = a.stat_at + up(slots * a.ws.rows * 8);
    a.queries_at = a.first_at + up((size_t)(p.B + 1) * 8);
    a.factors_at =
        a.queries_at + (a.wide ? 0 : up((size_t)all * a.tile * p.c.d * (dtype == OQ_BF16 ? 2 : 4)));
    a.bytes = a.factors_at + (a.wide ? 0 : up((size_t)all * a.tile * 4));
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
        return attend::run_wide(p, a.ws, st);
    if (a.splits > 0)
        return attend::launch_narrow(p, a.ws, dtype, a.splits, st);
    if (p.c.d == 128)
        return a.tile == 8 ? attend::run_narrow<128, 1>(p, a.ws, dtype, st)
                           : attend::run_narrow<128, 2>(p, a.ws, dtype, st);
    return attend::run_narrow<256, 1>(p, a.ws, dtype, st);
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
