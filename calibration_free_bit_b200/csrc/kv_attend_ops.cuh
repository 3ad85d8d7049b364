// kv_attend_ops.cuh -- what the forms of the cache's attention share (kv_attend.cuh, kv_wide.cuh):
// a sequence's rows and lengths with their checks, fp16 pairs, the softmax's constants, and the
// list of work that a launch's workers share out evenly.
#pragma once

#include <math_constants.h>

#include "kv_internal.h"
#include "kv_ops.cuh"

namespace oq {
namespace attend {

using namespace kvops;

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
    else if (prefix < 0 ||
             (long long)prefix + (r1 - r0) > ((long long)p.table_width << p.c.page_log2))
        err = AT_ERR_LEN;
    if (err) {
        if (tell)
            atomicOr(p.err, err);
        return false;
    }
    s->row0 = r0;
    s->nodes = r1 - r0;
    s->prefix = prefix;
    return true;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// What fp16 leaves of a and b.
__device__ __forceinline__ uint32_t half2_rest(float a, float b, uint32_t hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return half2_bits(a - f.x, b - f.y);
}

// A row's reference m is raised only when a score passes it by kSlack (in powers of two), so most
// steps need no reduction over lanes; weights reach 2^kSlack kWeightScale = 2^14 in fp16.
constexpr float kSlack = 8.0f, kWeightScale = 64.0f;
constexpr float kNone = -3.402823466e38f;             // reference of a row that has seen nothing: no
                                                     // finite score is below it

// The power of two above a norm, with room for a quarter more, in [2^-100, 2^127].
__device__ __forceinline__ float norm_scale(float v) {
    const uint32_t p2 = (__float_as_uint(v * 1.25f) & 0x7f800000u) + 0x00800000u;
    return __uint_as_float(min(max(p2, 27u << 23), 254u << 23));
}

// ---- rows ----
// Row r of a tile of 8 nt: the rotated query of the key head's row `at` (zeros without one), by a
// warp, as fp16 over the power of two below its largest element; with SPLIT also what that leaves.
// It goes to `to` as the lanes of a matrix instruction take it, [part][row / 8][step][lane][4] with
// lane = 4 (row % 8) + quarter of the row.  Returns the factor of its scores.
template <class E, int D, bool SPLIT>
__device__ __forceinline__ float rotate_row(const KvAttendParams &p, const Seq &s, int kvh, int at,
                                            bool real, const uint32_t (&ent)[D / 32], float *xs,
                                            int r, int nt, __half *to) {
    constexpr int N = D / 32, KS = D / 16;
    const int lane = threadIdx.x & 31;
    float z[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        z[i] = 0.f;
    if (real) {
        const int node = at / p.group, e = at - node * p.group;
        const E *q = static_cast<const E *>(p.q) + (long long)(s.row0 + node) * p.q_stride +
                     (kvh * p.group + e) * D;
#pragma unroll
        for (int i = 0; i < N; ++i)
            xs[i * 32 + lane] = to_f32(q[i * 32 + lane]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float v = xs[ent[i] & 0x7fffu];
            z[i] = (ent[i] & 0x8000u) ? -v : v;
        }
        warp_wht<D>(z, p.h, lane);
        __syncwarp();
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
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float v = z[i] * down;
        const __half hi = __float2half_rn(v);
        const int x = lane * N + i, y = x % (D / 4);
        const int o = (((r >> 3) * KS + (y >> 2)) * 32 + (r & 7) * 4 + x / (D / 4)) * 4 + (y & 3);
        to[o] = hi;
        if constexpr (SPLIT)
            to[nt * 8 * D + o] = __float2half_rn(v - __half2float(hi));
    }
    return up * p.qk_scale;
}

// The key head's row `at` from its sums (lane l has elements l D/32 on) and its weights' sum: R^T,
// and out.  A row that saw nothing gives zeros.
template <class E, int D>
__device__ __forceinline__ void finish_row(const KvAttendParams &p, const Seq &s, int kvh, int at,
                                           const uint32_t (&ent)[D / 32], float *xs,
                                           float (&o)[D / 32], float sum) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    warp_wht<D>(o, p.h, lane);
    const float inv = sum == 0.f ? 0.f : p.o_scale / sum;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i)
        xs[ent[i] & 0x7fffu] = inv * ((ent[i] & 0x8000u) ? -o[i] : o[i]);
    __syncwarp();
    const int node = at / p.group, e = at - node * p.group;
    E *y = static_cast<E *>(p.out) + (long long)(s.row0 + node) * p.out_stride +
           (kvh * p.group + e) * D;
#pragma unroll
    for (int i = 0; i < N; ++i)
        y[i * 32 + lane] = from_f32<E>(xs[i * 32 + lane]);
}

// ---- work lists ----
// A segment is one sequence's tile of rows of one key head; its units are the sequence's tiles of
// tokens, and before them `Extra` that stand for the time that a segment's setting up takes.  The
// units of all segments in a row (sequence, key head, row tile) are shared out evenly to W workers,
// a contiguous range each, whatever the lengths: worker w has units w U / W to (w + 1) U / W.  What
// a worker has of a segment's tiles is a piece; piece (segment s, worker w) has slot s + w of the
// workspace (one of the two grows from a piece to the next, so slots are distinct), where segments
// count as if every sequence had the most rows.
struct Units {
    int tiles, segments;          // of one sequence; 0 segments: nothing to do
};
template <class Form>             // Form::tokens, rows, extra
__device__ __forceinline__ Units units_of(const KvAttendParams &p, int b, Seq *s, bool tell) {
    Units u = {0, 0};
    if (load_seq(p, b, s, tell) && s->nodes > 0) {
        u.tiles = (s->prefix + s->nodes + Form::tokens - 1) / Form::tokens;
        u.segments = p.c.kv_heads * ((s->nodes * p.group + Form::rows - 1) / Form::rows);
    }
    return u;
}
template <class Form> __device__ __forceinline__ long long all_units(const Units &u) {
    return (long long)(u.tiles + Form::extra) * u.segments;
}

// Workers that share U units: `most`, fewer while one has less than `least` units.
__device__ __forceinline__ long long workers_for(long long U, int most, int least) {
    const long long w = (U + least - 1) / least;
    return w < 1 ? 1 : (w < most ? w : most);
}

// By one warp of a launch: the units before each sequence to ws.first[0 .. B], and unusable
// sequences are reported.
template <class Form>
__device__ __forceinline__ void list_units(const KvAttendParams &p, const KvAttendSpace &ws) {
    const int lane = threadIdx.x & 31;
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        long long n = 0;
        if (b0 + lane < p.B) {
            Seq s;
            n = all_units<Form>(units_of<Form>(p, b0 + lane, &s, true));
        }
        long long sum = n;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, sum, k);
            sum += lane >= k ? o : 0;
        }
        if (b0 + lane < p.B)
            ws.first[b0 + lane] = base + sum - n;
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0)
        ws.first[p.B] = base;
}

// A worker's range of units, and the sequence that it starts in (with the units before that).
struct Walk {
    long long u, u1, before;
    int b;
};

// Worker `worker`'s range from ws.first, by a whole warp.
__device__ __forceinline__ Walk take_range(const KvAttendParams &p, const KvAttendSpace &ws,
                                           long long worker) {
    const int lane = threadIdx.x & 31;
    const long long U = ws.first[p.B], W = workers_for(U, ws.most, ws.least);
    Walk w = {0, 0, 0, 0};
    if (worker >= W || U == 0)
        return w;
    w.u = worker * U / W;
    w.u1 = (worker + 1) * U / W;
    // the last sequence with first[b] <= u, in [lo, hi): 32 places at a time
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const unsigned in = __ballot_sync(0xffffffffu, at < hi && ws.first[at < hi ? at : lo] <= w.u);
        lo += (31 - __clz(in)) * step;                // lane 0's place always is
        hi = min(hi, lo + step);
    }
    w.b = lo;
    w.before = ws.first[lo];
    return w;
}

// The next piece of a range: a run of tiles of one segment.
struct Piece {
    Seq s;
    int b, seg, tile0, n, kvh, row_base, nrows, total;
};
template <class Form>
__device__ __forceinline__ bool next_piece(const KvAttendParams &p, Walk &w, Piece &q) {
    while (w.u < w.u1) {
        const Units un = units_of<Form>(p, w.b, &q.s, false);
        const long long all = all_units<Form>(un);
        if (w.u >= w.before + all) {
            w.before += all;
            ++w.b;
            continue;
        }
        const int len = un.tiles + Form::extra;
        q.b = w.b;
        q.seg = (int)((w.u - w.before) / len);
        const int from = (int)((w.u - w.before) - (long long)q.seg * len);
        const int n = (int)min((long long)(len - from), w.u1 - w.u);
        w.u += n;
        q.tile0 = max(from - Form::extra, 0);
        q.n = from + n - Form::extra - q.tile0;
        if (q.n <= 0)
            continue;                                 // none of its tiles
        const int row_tiles = un.segments / p.c.kv_heads;
        q.kvh = q.seg / row_tiles;
        q.row_base = (q.seg - q.kvh * row_tiles) * Form::rows;
        q.nrows = min(Form::rows, q.s.nodes * p.group - q.row_base);
        q.total = q.s.prefix + q.s.nodes;
        return true;
    }
    return false;
}

// The forms: tiles of many rows (kv_wide.cuh) and of 8 NT (kv_attend.cuh).  `extra`, us: 16 sequences with
// 61 nodes 165, 160 and 162 with 2, 3 and 4; 64 sequences of single tokens 87.3, 87.0 and 87.0 with 3, 4
// and 6, 8 sequences of 40 key heads 45.8, 47.4 and 47.5.  The small tiles' 4 is not the fastest there: it
// is what a worker has at least (kv_attend.cu, `least`), and in a small call, where each worker has just
// that, a sequence whose units are a multiple of 4 is then cut at the same places, and rounded alike,
// whether or not another beside it is skipped.
struct WideForm {
    static constexpr int tokens = 128, rows = 128, extra = 3;
};
template <int NT> struct NarrowForm {
    static constexpr int tokens = 16, rows = 8 * NT, extra = 4;
};

}  // namespace attend
}  // namespace oq
