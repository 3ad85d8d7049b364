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

// Total units, by a whole warp; with `first`, the units before each sequence to first[0 .. B].
template <int TOKENS, int ROWS>
__device__ __forceinline__ long long count_units(const KvAttendParams &p, long long *first) {
    const int lane = threadIdx.x & 31;
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        long long n = 0;
        if (b0 + lane < p.B) {
            Seq s;
            const Units u = units_of<TOKENS, ROWS>(p, b0 + lane, &s, first != nullptr);
            n = (long long)u.tiles * u.segments;
        }
        long long sum = n;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, sum, k);
            sum += lane >= k ? o : 0;
        }
        if (first != nullptr && b0 + lane < p.B)
            first[b0 + lane] = base + sum - n;
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (first != nullptr && lane == 0)
        first[p.B] = base;
    return base;
}

// The sequence that unit u is in, by a whole warp, and the units before it.
template <int TOKENS, int ROWS>
__device__ __forceinline__ int find_sequence(const KvAttendParams &p, long long u,
                                             long long *before) {
    const int lane = threadIdx.x & 31;
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        long long n = 0;
        if (b0 + lane < p.B) {
            Seq s;
            const Units w = units_of<TOKENS, ROWS>(p, b0 + lane, &s, false);
            n = (long long)w.tiles * w.segments;
        }
        long long sum = n;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, sum, k);
            sum += lane >= k ? o : 0;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + sum > u);
        if (past) {
            const int at = __ffs(past) - 1;
            *before = base + __shfl_sync(0xffffffffu, sum - n, at);
            return b0 + at;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    *before = base;
    return p.B;
}

// Workers that share U units: `most`, fewer while one has less than `least` units.
__device__ __forceinline__ long long workers_for(long long U, int most, int least) {
    const long long w = (U + least - 1) / least;
    return w < 1 ? 1 : (w < most ? w : most);
}

}  // namespace attend
}  // namespace oq
