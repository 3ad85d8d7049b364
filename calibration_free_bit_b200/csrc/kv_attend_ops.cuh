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
constexpr float kNone = -1e30f;                      // reference of a row that has seen nothing

// ---- work lists ----
// A segment is one sequence's tile of rows of one key head; its units are the sequence's tiles of
// tokens.  The units of all segments in a row (sequence, key head, row tile) are shared out evenly
// to W workers, a contiguous range each, whatever the lengths: worker w has units w U / W to
// (w + 1) U / W.  A worker's part of a segment is a piece; piece (segment s, worker w) has slot
// s + w of the workspace (one of the two grows from a piece to the next, so slots are distinct),
// where segments count as if every sequence had the most rows.
struct Units {
    int tiles, segments;          // of one sequence; 0 segments: nothing to do
};
template <int TOKENS, int ROWS>
__device__ __forceinline__ Units units_of(const KvAttendParams &p, int b, Seq *s, bool tell) {
    Units u = {0, 0};
    if (load_seq(p, b, s, tell) && s->nodes > 0) {
        u.tiles = (s->prefix + s->nodes + TOKENS - 1) / TOKENS;
        u.segments = p.c.kv_heads * ((s->nodes * p.group + ROWS - 1) / ROWS);
    }
    return u;
}

// Workers that share U units: `most`, fewer while one has less than `least` units.
__device__ __forceinline__ long long workers_for(long long U, int most, int least) {
    const long long w = (U + least - 1) / least;
    return w < 1 ? 1 : (w < most ? w : most);
}

// A worker's range of units, and the sequence that it starts in (with the units before that).
struct Walk {
    long long u, u1, before;
    int b;
};

// Worker `worker`'s range, by a whole warp.  With `tell`, the units before each sequence go to
// ws.first[0 .. B] and unusable sequences are reported: one warp of the launch does that.
template <int TOKENS, int ROWS>
__device__ __forceinline__ Walk take_range(const KvAttendParams &p, const KvAttendSpace &ws,
                                           long long worker, bool tell) {
    const int lane = threadIdx.x & 31, each = (p.B + 31) / 32;
    auto count = [&](int b, bool t) -> long long {
        if (b >= p.B)
            return 0;
        Seq s;
        const Units u = units_of<TOKENS, ROWS>(p, b, &s, t);
        return (long long)u.tiles * u.segments;
    };
    // a lane has `each` sequences in a row
    long long mine = 0;
    for (int k = 0; k < each; ++k)
        mine += count(lane * each + k, tell);
    long long upto = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, upto, k);
        upto += lane >= k ? o : 0;
    }
    const long long U = __shfl_sync(0xffffffffu, upto, 31);
    if (tell) {
        long long at = upto - mine;
        for (int k = 0; k < each && lane * each + k < p.B; ++k) {
            ws.first[lane * each + k] = at;
            at += count(lane * each + k, false);
        }
        if (lane == 0)
            ws.first[p.B] = U;
    }
    const long long W = workers_for(U, ws.most, ws.least);
    Walk w = {0, 0, 0, 0};
    if (worker >= W || U == 0)
        return w;
    w.u = worker * U / W;
    w.u1 = (worker + 1) * U / W;
    const int owner = __ffs(__ballot_sync(0xffffffffu, upto > w.u)) - 1;
    w.before = __shfl_sync(0xffffffffu, upto - mine, owner);
    // within the owner's sequences, 32 at a time
    for (int b0 = owner * each;; b0 += 32) {
        const bool in = b0 + lane < (owner + 1) * each;
        const long long n = in ? count(b0 + lane, false) : 0;
        long long sum = n;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, sum, k);
            sum += lane >= k ? o : 0;
        }
        const unsigned past = __ballot_sync(0xffffffffu, w.before + sum > w.u);
        if (past) {
            const int at = __ffs(past) - 1;
            w.before += __shfl_sync(0xffffffffu, sum - n, at);
            w.b = b0 + at;
            return w;
        }
        w.before += __shfl_sync(0xffffffffu, sum, 31);
    }
}

// The next piece of a range: a run of tiles of one segment.
struct Piece {
    Seq s;
    int b, seg, tile0, n, kvh, row_base, nrows, total;
};
template <int TOKENS, int ROWS>
__device__ __forceinline__ bool next_piece(const KvAttendParams &p, Walk &w, Piece &q) {
    while (w.u < w.u1) {
        const Units un = units_of<TOKENS, ROWS>(p, w.b, &q.s, false);
        const long long all = (long long)un.tiles * un.segments;
        if (w.u >= w.before + all) {
            w.before += all;
            ++w.b;
            continue;
        }
        q.b = w.b;
        q.seg = (int)((w.u - w.before) / un.tiles);
        q.tile0 = (int)((w.u - w.before) - (long long)q.seg * un.tiles);
        q.n = (int)min((long long)(un.tiles - q.tile0), w.u1 - w.u);
        const int row_tiles = un.segments / p.c.kv_heads;
        q.kvh = q.seg / row_tiles;
        q.row_base = (q.seg - q.kvh * row_tiles) * ROWS;
        q.nrows = min(ROWS, q.s.nodes * p.group - q.row_base);
        q.total = q.s.prefix + q.s.nodes;
        w.u += q.n;
        return true;
    }
    return false;
}

}  // namespace attend
}  // namespace oq
