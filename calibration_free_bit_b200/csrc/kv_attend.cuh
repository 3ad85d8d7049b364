// kv_attend.cuh -- attention of drafted tokens over the quantised cache, one instance a bit width
// (kv_attend_b*.cu); launch_kv_attend (kv_attend.cu) picks it.  Work list: kv_attend_ops.cuh.
//
// o = sum_t p_t v_hat_t, p = softmax_t(scale * q . k_hat_t), over the visible cached tokens t of
// the row's sequence: its prefix, and those of its drafted tokens that the row's mask names (bit
// j: node j; without a mask, nodes up to its own).  R is orthogonal, so q . k_hat = (R q) .
// centroid[code] s / sqrt(d): a row's query is rotated once, before the loop, and R^T is applied
// once, to the finished row.
//
// What bounds it is the cache's bytes (a token of one head: two rows of codes and two norms), and
// right behind them shared memory: two codes a lookup.  So:
//   - the rows of one key head (its query heads times the nodes) share a pass over its tokens, in
//     tiles of 8 NT rows; a unit of work is 16 tokens of a tile, taken by one warp.  Much work
//     (attend_tiles): all warps of all SMs have the same number of units, none waits for another,
//     what a warp has of a segment goes to the workspace, and a second kernel joins the pieces in a
//     fixed order.  Little work (attend_near): a cluster of CTAs takes a segment, and its warps meet
//     in shared memory, in one launch without a workspace;
//   - a warp's tiles come into its own ring in shared memory by asynchronous copies (a tile's rows
//     of a head lie together), several tiles ahead of their use, without a register; a lane's codes
//     go through a table in shared memory with a column a lane (no bank conflicts) into the operand
//     of a matrix instruction;
//   - products are transposed, S^T = K Q^T and O^T = V^T P^T (mma.sync m16n8k16): the 16-wide side
//     is the cache, so 8 rows fill an instruction and an accumulator takes 32 registers.  The
//     instruction's order of a row's elements is free as long as both operands agree, which is how
//     a lane can own consecutive bytes of a row.  tcgen05 would need the decoded tile in shared or
//     tensor memory and has nothing to gain at these row counts.
// B200, 4 bits, 8 key heads of 128: 64 sequences of 37 to 8191 tokens 87 us (codes and norms at 3.3 TB/s;
// the data pipe of shared memory busy 72 % of attend_tiles, its issue slots 63 %), one of 4096 tokens
// 11.0 us by a cluster a head.
// Scores, softmax statistics and sums are fp32.  fp16 enters in three places: the rotated query
// (over a power of two of its own), the centroids (times alpha, see build_kv_lut) and the weights
// p s_v, which are taken relative to a power of two above the row's largest s_v and times 2^6 to
// 2^14: what a token adds is resolved down to 2^-31 of the largest.  With SPLIT (fp16 outputs) a
// query and a weight enter as sums of two fp16 numbers, and so do the centroids of 6 and 8 bits, which
// are too many for alpha to help: errors of 2.1e-4 to 2.5e-4 of an output's length, of which its own
// rounding is 2.1e-4 (queries alone: 2.6e-4 at 2 bits, 3.1e-4 at 4, 5.9e-4 at 8).
#pragma once

#include <cooperative_groups.h>

#include "k1_ops.cuh"
#include "kv_attend_ops.cuh"
#include "kv_internal.h"
#include "kv_lut.cuh"
#include "kv_ops.cuh"
#include "sm100_common.cuh"

namespace oq {
namespace attend {

using namespace kvops;

// c += a b: a 16 x 16 (row), b 16 x 8 (column), fp16 in, fp32 out.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <int D, int BITS> struct Shape {
    static constexpr int row_bytes = D * BITS / 8;
    static constexpr int k_bytes = row_bytes / 4;     // a lane's share of a key row
    static constexpr int kw = k_bytes / 4;
    // a lane's share of a value row is an eighth; 6 bytes (3 bits, D = 128) are taken out of the
    // 12 that two lanes share
    static constexpr bool v_shared = row_bytes % 32 != 0;
    static constexpr int v_bytes = v_shared ? row_bytes / 4 : row_bytes / 8;
    static constexpr int vw = v_bytes / 4;            // words loaded
    static constexpr int vu = v_shared ? 2 : vw;      // words used
};

// A warp's ring of tiles in shared memory: 16 key rows, 16 value rows and their norms each, brought in
// by asynchronous copies of 16 bytes a lane as many tiles ahead as there are slots.  (A tile's rows lie
// together, so a lane's addresses cost little; bulk copies by one lane took 120 instructions a tile,
// with nothing to do for the other lanes, and 102 us instead of 87 for
// 64 sequences of 37 to 8191 tokens, 8 heads of 128, 4 bits, pages of 16.)
// Row j of a tile's matrices is token order(j) of its 16: the four value rows that a warp reads in one
// go then lie together.
__device__ __forceinline__ int order(int j) { return (j & 8) + ((j & 7) >> 1) + ((j & 1) << 2); }

template <int D, int BITS, int SLOTS> struct Ring {
    using S = Shape<D, BITS>;
    static constexpr int rows = 16 * S::row_bytes;
    static constexpr int kn_at = 2 * rows, vn_at = kn_at + 64;
    static constexpr int slot = vn_at + 64;           // keys, values, their norms
    static constexpr int bytes = SLOTS * slot;
    uint32_t at, put, got;                            // address; offsets of the next to fill and read
    uint32_t known;                                   // bit i: the page of the i-th last tile is one

    __device__ __forceinline__ void init(uint32_t own) {
        at = own;
        put = got = known = 0;
    }
    __device__ __forceinline__ static void copy16(uint32_t to, const void *from) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    }
    // The next slot (its last readers are done) takes 16 tokens of a page from `in` on.  A missing
    // page leaves it as it was.
    __device__ __forceinline__ void fetch(const KvAttendParams &p, int page, int in, int kvh,
                                          int lane) {
        const bool ok = page >= 0 && page < p.c.pages;
        known = (known << 1) | (ok ? 1u : 0u);
        if (ok) {
            const uint32_t to = at + put + lane * 16;
            const long long row =
                (((long long)page * p.c.kv_heads + kvh) << p.c.page_log2) + in;
            const uint8_t *k = p.c.codes[0] + row * S::row_bytes + lane * 16;
            const uint8_t *v = p.c.codes[1] + row * S::row_bytes + lane * 16;
#pragma unroll
            for (int i = 0; i < rows; i += 512)
                if (i + 512 <= rows || i + lane * 16 < rows) {
                    copy16(to + i, k + i);
                    copy16(to + rows + i, v + i);
                }
            if (lane < 8)
                copy16(to + kn_at, pick(p.c.norms, lane >> 2) + row + (lane & 3) * 4);
        }
        put = put + slot == bytes ? 0 : put + slot;
    }
    __device__ __forceinline__ static void commit() {
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // The oldest slot of SLOTS: its address, and whether its page is one.
    __device__ __forceinline__ uint32_t take(bool &ok) {
        asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
        __syncwarp();
        const uint32_t from = at + got;
        ok = (known >> (SLOTS - 1)) & 1u;
        got = got + slot == bytes ? 0 : got + slot;
        return from;
    }
};

// Words of shared memory, in the widest loads that ALIGN bytes allow.
template <int W, int ALIGN>
__device__ __forceinline__ void take_words(uint32_t (&w)[W], uint32_t at) {
    if constexpr (ALIGN % 16 == 0 && W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < W; i += 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(at + 4 * i));
    } else if constexpr (ALIGN % 8 == 0 && W % 2 == 0) {
#pragma unroll
        for (int i = 0; i < W; i += 2)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[i]), "=r"(w[i + 1]) : "r"(at + 4 * i));
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[i]) : "r"(at + 4 * i));
    }
}

// This lane's elements (g D/8 on) of a value row.
template <int D, int BITS>
__device__ __forceinline__ void take_share(uint32_t (&w)[Shape<D, BITS>::vu], uint32_t row, int g) {
    using S = Shape<D, BITS>;
    if constexpr (S::v_shared) {                     // 48 of the 96 bits of two lanes
        uint32_t v[3];
        take_words<3, 4>(v, row + (g >> 1) * S::v_bytes);
        w[0] = (g & 1) ? (v[1] >> 16) | (v[2] << 16) : v[0];
        w[1] = (g & 1) ? v[2] >> 16 : v[1];
    } else {
        take_words<S::vu, S::v_bytes>(w, row + g * S::v_bytes);
    }
}

// A warp's queries: the B operands of S^T = K Q^T (row n = g, elements c D/4 + 4 ks + {0, 1}, {2, 3}).
template <int D, int NT, bool SPLIT> struct Queries {
    static constexpr int KS = D / 16;
    static constexpr int words = NT * KS * 32 * (SPLIT ? 2 : 1);     // uint2 of a tile
    uint2 f[NT * KS * (SPLIT ? 2 : 1)];
    __device__ __forceinline__ void take(const uint2 *from) {       // at this lane
#pragma unroll
        for (int i = 0; i < NT * KS * (SPLIT ? 2 : 1); ++i)
            f[i] = from[i * 32];
    }
    __device__ __forceinline__ uint2 operator()(int part, int n, int ks) const {
        return f[(part * NT + n) * KS + ks];
    }
};

// What a warp has summed up of a segment, for rows 2c, 2c + 1 (and 8 n on).
template <int D, int NT> struct Sums {
    static constexpr int KS = D / 16;
    float acc[NT][KS][4];
    float m[NT][2], l[NT][2];                     // reference and sum
    float vs[NT][2], vinv[NT][2];                 // power of two over s_v, kWeightScale over it
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[n][j][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                m[n][i] = kNone, l[n][i] = 0.f, vs[n][i] = 0.f, vinv[n][i] = 0.f;
        }
    }
    // l over all lanes, acc in units of one.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int k = 4; k < 32; k <<= 1)
                    l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], k);
                const float f = vs[n][i] * (1.0f / kWeightScale);
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    acc[n][j][i] *= f;
                    acc[n][j][2 + i] *= f;
                }
            }
    }
};

// Tiles t, t + stride, ... below `last` of one segment, by a warp.  `start` is called once the first
// tiles are on their way, and fills `q`, `qs` (score factors of rows 2c, 2c + 1) and `masks`.
// `col`: lut_column's.
template <LutForm FORM, int D, int BITS, int NT, bool SPLIT, int SLOTS, class Start>
__device__ __forceinline__ void walk_tiles(const KvAttendParams &p, uint32_t col,
                                           Ring<D, BITS, SLOTS> &ring, const Seq &s, int b, int kvh,
                                           int t, int stride, int last, Queries<D, NT, SPLIT> &q,
                                           float (&qs)[NT][2], const unsigned long long *masks,
                                           Sums<D, NT> &o, Start start) {
    using S = Shape<D, BITS>;
    using R = Ring<D, BITS, SLOTS>;
    constexpr int KS = D / 16;
    constexpr bool RESTS = SPLIT && BITS >= 6;        // of the centroids
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int *table = p.table + (long long)b * p.table_width;
    const int in_page = (1 << p.c.page_log2) - 1;
    bool bad_page = false;
    // where this lane's parts of a slot lie
    const uint32_t k_off = order(g) * S::row_bytes + c * S::k_bytes, n_off = R::kn_at + 4 * order(g);
    const uint32_t v_off = R::rows + c * S::row_bytes;
    auto place = [&](int t) -> int {              // a tile's page
        return t < last ? table[(t << 4) >> p.c.page_log2] : -1;
    };
    __syncwarp();
    for (int k = 0; k < SLOTS; ++k) {
        ring.fetch(p, place(t + k * stride), ((t + k * stride) << 4) & in_page, kvh, lane);
        ring.commit();
    }
    int page = place(t + SLOTS * stride);
    start();

    for (; t < last; t += stride) {
        const int ahead = t + SLOTS * stride, page1 = place(ahead + stride);
        const int tok = t << 4;
        bool ok;
        const uint32_t tile = ring.take(ok);
        uint32_t kr[2][S::kw];
        float kn[2], vn[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            take_words<S::kw, S::k_bytes>(kr[i], tile + k_off + 8 * i * S::row_bytes);
            uint32_t u[1];
            take_words<1, 4>(u, tile + n_off + 32 * i);
            kn[i] = __uint_as_float(u[0]);
            take_words<1, 4>(u, tile + n_off + 32 * i + (R::vn_at - R::kn_at));
            vn[i] = __uint_as_float(u[0]);
        }
        // S^T = K Q^T, in two sums
        float st[NT][4], s2[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                st[n][i] = s2[n][i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t a[4], rest[4];
            quad<BITS, FORM>(kr[0], ks, col, a[0], a[2], rest[0], rest[2]);
            quad<BITS, FORM>(kr[1], ks, col, a[1], a[3], rest[1], rest[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint2 w = q(0, n, ks);
                mma16816((ks & 1) ? s2[n] : st[n], a, w.x, w.y);
                if constexpr (SPLIT) {
                    if constexpr (RESTS)
                        mma16816((ks & 1) ? s2[n] : st[n], rest, w.x, w.y);
                    w = q(1, n, ks);
                    mma16816((ks & 1) ? s2[n] : st[n], a, w.x, w.y);
                }
            }
        }
        // scores of tokens order(g), + 8 and rows 2c, 2c + 1, in powers of two
        bool grow = false;
        const bool edge = !ok || tok + 16 > s.prefix;     // the page is missing, or it has nodes
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                st[n][i] = (st[n][i] + s2[n][i]) * (kn[i >> 1] * qs[n][i & 1]);
        if (edge) {
            // (a missing page's slot has what was there before: finite codes, any norms)
            bad_page |= !ok;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int node = tok + order(g) + 8 * (i >> 1) - s.prefix;
                    const bool see = ok && (node < 0 || (node < s.nodes &&
                                     ((masks[8 * n + 2 * c + (i & 1)] >> node) & 1ull)));
                    if (!see)
                        st[n][i] = -CUDART_INF_F;
                    else
                        grow |= vn[i >> 1] > o.vs[n][i & 1];
                }
        } else {
            const float v = fmaxf(vn[0], vn[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                grow |= v > o.vs[n][0] || v > o.vs[n][1];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                grow |= fmaxf(st[n][i], st[n][2 + i]) > o.m[n][i] + kSlack;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float up = fmaxf(st[n][i], st[n][2 + i]);
                    float v = fmaxf(st[n][i] > -CUDART_INF_F ? vn[0] : 0.f,
                                    st[n][2 + i] > -CUDART_INF_F ? vn[1] : 0.f);
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) {
                        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, k));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
                    }
                    up = fmaxf(up, o.m[n][i]);
                    f[i] = ex2(o.m[n][i] - up);
                    o.m[n][i] = up;
                    o.l[n][i] *= f[i];
                    if (v > o.vs[n][i]) {
                        const float nv = norm_scale(v);
                        f[i] *= o.vs[n][i] / nv;
                        o.vs[n][i] = nv;
                        o.vinv[n][i] = kWeightScale / nv;
                    }
                }
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o.acc[n][j][i] *= f[i & 1];
            }
        }
        // weights
        uint32_t pb[NT][2], pr[NT][2];                // and what fp16 leaves of them
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = ex2(st[n][i] - o.m[n][i & 1]);
                o.l[n][i & 1] += e;
                w[i] = e * (vn[i >> 1] * o.vinv[n][i & 1]);
            }
            if (edge) {                               // what is not seen may have any norm
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (st[n][i] == -CUDART_INF_F)
                        w[i] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t hi = half2_bits(w[2 * k], w[2 * k + 1]);
                pb[n][k] = transpose8x8(hi);
                if constexpr (SPLIT)
                    pr[n][k] = transpose8x8(half2_rest(w[2 * k], w[2 * k + 1], hi));
            }
        }
        // O^T += V^T P^T: rows of tile j are elements g D/8 + 2j and 2j + 1
        uint32_t vw[4][S::vu];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            take_share<D, BITS>(vw[i], tile + v_off + (4 * (i & 1) + 8 * (i >> 1)) * S::row_bytes, g);
        __syncwarp();                                 // all have read the slot
        ring.fetch(p, page, (ahead << 4) & in_page, kvh, lane);
        ring.commit();
        page = page1;
        mixed<BITS>(vw[0], vw[1]);
        mixed<BITS>(vw[2], vw[3]);
#pragma unroll
        for (int j = 0; j < KS; j += 2) {
            uint32_t x[4], y[4], rx[4], ry[4];
            quad_of_two<BITS, FORM>(vw[0], vw[1], j / 2, col, x, rx);
            quad_of_two<BITS, FORM>(vw[2], vw[3], j / 2, col, y, ry);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t a[4] = {x[2 * h], x[2 * h + 1], y[2 * h], y[2 * h + 1]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma16816(o.acc[n][j + h], a, pb[n][0], pb[n][1]);
                    if constexpr (SPLIT)
                        mma16816(o.acc[n][j + h], a, pr[n][0], pr[n][1]);
                }
                if constexpr (RESTS) {
                    const uint32_t ra[4] = {rx[2 * h], rx[2 * h + 1], ry[2 * h], ry[2 * h + 1]};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816(o.acc[n][j + h], ra, pb[n][0], pb[n][1]);
                }
            }
        }
    }
    if (bad_page && lane == 0)
        atomicOr(p.err, AT_ERR_PAGE);
}

__device__ __forceinline__ unsigned long long mask_of(const KvAttendParams &p, const Seq &s,
                                                      int row, int nrows, int row_base) {
    if (row >= nrows)
        return 0ull;
    const int node = (row_base + row) / p.group;
    return p.mask ? (unsigned long long)p.mask[s.row0 + node] : (2ull << node) - 1ull;
}

// ---- much work: a worker a warp ----
// Shared memory by address (a CTA's own starts at 1024): a table of 64 KB, or of 8, at the first
// multiple of its size, the warps' own parts (masks, ring) before and behind it.
template <int D, int BITS, int NT, bool SPLIT> struct Stream {
    // of the one CTA on an SM: as many as registers allow (12 took 106 us, 16 took 101)
    static constexpr int warps = D == 128 && NT == 1 ? 16 : 8;
    static constexpr int rows = 8 * NT;
    static constexpr int lut = Lut<BITS, WIDE>::bytes, lut_at = lut;
    static constexpr int most = 227 * 1024 + kSharedStart;
    template <int SLOTS> static constexpr int own_of() {
        return (rows * 8 + Ring<D, BITS, SLOTS>::bytes + 127) / 128 * 128;
    }
    template <int SLOTS> static constexpr bool fits() {
        return (lut_at - kSharedStart) / own_of<SLOTS>() + (most - lut_at - lut) / own_of<SLOTS>() >= warps;
    }
    static constexpr int slots = fits<4>() ? 4 : fits<3>() ? 3 : 2;
    static constexpr int own = own_of<slots>(), before = (lut_at - kSharedStart) / own;
    static constexpr int behind = warps > before ? warps - before : 0;
    static constexpr int bytes = lut_at + lut + behind * own - kSharedStart;
    static_assert(fits<slots>() && bytes <= 227 * 1024, "shared memory");
    __device__ static int own_at(int warp) {
        return warp < before ? kSharedStart + warp * own : lut_at + lut + (warp - before) * own;
    }
};

template <int D, int BITS, int NT, bool SPLIT>
__global__ void __launch_bounds__(32 * Stream<D, BITS, NT, SPLIT>::warps, 1)
attend_tiles(const KvAttendParams p, const KvAttendSpace ws) {
    using M = Stream<D, BITS, NT, SPLIT>;
    using Q = Queries<D, NT, SPLIT>;
    constexpr int KS = D / 16;
    extern __shared__ __align__(1024) unsigned char raw[];
    if (!starts_there(raw)) {                             // not where the layout expects it
        if (threadIdx.x == 0)
            atomicOr(p.err, AT_ERR_WAIT);
        return;
    }
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int own = M::own_at(warp);
    unsigned long long *masks = reinterpret_cast<unsigned long long *>(at_address(raw, own));
    fill_lut<BITS, WIDE>(at_address(raw, M::lut_at), p.lut);
    const uint32_t col = lut_column<BITS, WIDE>(M::lut_at, lane);
    Ring<D, BITS, M::slots> ring;
    ring.init(own + M::rows * 8);
    __syncthreads();
    pdl_wait();
    // neighbouring workers on different SMs: few units reach all of them
    const long long worker = (long long)warp * gridDim.x + blockIdx.x;
    Walk walk = take_range(p, ws, worker);
    Piece piece;
    while (next_piece<NarrowForm<NT>>(p, walk, piece)) {
        Q q;
        float qs[NT][2];
        Sums<D, NT> o;
        o.clear();
        walk_tiles<WIDE, D, BITS, NT, SPLIT>(
            p, col, ring, piece.s, piece.b, piece.kvh, piece.tile0, 1, piece.tile0 + piece.n, q, qs, masks,
            o, [&] {
                const long long seg = (long long)piece.b * ws.segments + piece.seg;
                const uint2 *from = ws.queries + seg * Q::words + lane;
                __syncwarp();
                if (lane < M::rows)
                    masks[lane] = mask_of(p, piece.s, lane, piece.nrows, piece.row_base);
                __syncwarp();
                q.take(from);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qs[n][i] = ws.factors[seg * M::rows + 8 * n + 2 * c + i];
            });
        // ---- the piece goes to its slot ----
        o.finish();
        const long long slot = (long long)piece.b * ws.segments + piece.seg + worker;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * n + 2 * c + i;
                if (r >= piece.nrows)
                    continue;
                if (g == 0) {
                    ws.stat[slot * 2 * ws.rows + r] = o.m[n][i];
                    ws.stat[(slot * 2 + 1) * ws.rows + r] = o.l[n][i];
                }
                float4 *dst =
                    reinterpret_cast<float4 *>(ws.part + (slot * ws.rows + r) * D + g * (D / 8));
#pragma unroll
                for (int j = 0; j < KS; j += 2)
                    dst[j / 2] = make_float4(o.acc[n][j][i], o.acc[n][j][2 + i],
                                             o.acc[n][j + 1][i], o.acc[n][j + 1][2 + i]);
            }
    }
}

// ---- little work: a cluster a segment ----
// Shared memory by address, as above, with the smaller table: two CTAs fit on an SM.
template <int D, int BITS, int NT, bool SPLIT> struct Near {
    static constexpr int warps = 8, rows = 8 * NT;
    using Q = Queries<D, NT, SPLIT>;
    using R = Ring<D, BITS, 2>;
    static constexpr int stride = D + 4;                                     // floats
    static constexpr int q_at = kSharedStart;
    static constexpr int x_at = q_at + Q::words * 8;                         // [warps][D] floats
    static constexpr int mask_at = x_at + warps * D * 4;
    static constexpr int stat_at = mask_at + rows * 8;                       // factor, m, l: [rows]
    static constexpr int warp_at = stat_at + rows * 12;                      // m, l: [warps][rows]
    static constexpr int fin_at = warp_at + warps * rows * 8;                // [rows][stride] floats
    static constexpr int lut_at = 32768;
    static constexpr int ring_at = lut_at + Lut<BITS, PLACED>::bytes;
    // and over both, once the tokens are done with, the warps' sums: [warps][rows][stride] floats
    static constexpr int most(int a, int b) { return a > b ? a : b; }
    static constexpr int bytes =
        lut_at + most(ring_at - lut_at + warps * R::bytes, warps * rows * stride * 4) - kSharedStart;
    static_assert(fin_at + rows * stride * 4 <= lut_at && fin_at % 16 == 0 && bytes <= 227 * 1024,
                  "shared memory");
};

template <class E, int D, int BITS, int NT, bool SPLIT>
__global__ void __launch_bounds__(32 * Near<D, BITS, NT, SPLIT>::warps)
attend_near(const KvAttendParams p, const int row_tiles) {
    using M = Near<D, BITS, NT, SPLIT>;
    using Q = Queries<D, NT, SPLIT>;
    constexpr int N = D / 32, KS = D / 16;
    extern __shared__ __align__(1024) unsigned char raw[];
    namespace cg = cooperative_groups;
    if (!starts_there(raw)) {                             // not where the layout expects it
        if (threadIdx.x == 0)
            atomicOr(p.err, AT_ERR_WAIT);
        cg::this_cluster().sync();                         // the others read this block's memory
        cg::this_cluster().sync();
        return;
    }
    uint2 *qm = reinterpret_cast<uint2 *>(at_address(raw, M::q_at));
    float *xs = reinterpret_cast<float *>(at_address(raw, M::x_at));
    unsigned long long *masks = reinterpret_cast<unsigned long long *>(at_address(raw, M::mask_at));
    float *factor = reinterpret_cast<float *>(at_address(raw, M::stat_at));
    float *row_m = factor + M::rows, *row_l = row_m + M::rows;

    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int rank = blockIdx.x, splits = gridDim.x;       // the cluster is the whole x dimension
    const int kvh = blockIdx.y / row_tiles, row_base = (blockIdx.y - kvh * row_tiles) * M::rows;
    const int b = blockIdx.z;
    fill_lut<BITS, PLACED>(at_address(raw, M::lut_at), p.lut);
    const uint32_t col = lut_column<BITS, PLACED>(rank_bits(raw) | M::lut_at, lane);
    typename M::R ring;
    ring.init(rank_bits(raw) | (M::ring_at + warp * M::R::bytes));
    uint32_t ent[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        ent[i] = p.ent[lane * N + i];
    pdl_wait();
    Seq s;
    if (!load_seq(p, b, &s, blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0))
        return;                                            // the whole cluster returns
    const int nrows = min(M::rows, s.nodes * p.group - row_base);
    if (nrows <= 0)
        return;
    const int tiles = (s.prefix + s.nodes + 15) >> 4, share = (tiles + splits - 1) / splits;
    Q q;
    float qs[NT][2];
    Sums<D, NT> o;
    o.clear();
    walk_tiles<PLACED, D, BITS, NT, SPLIT>(
        p, col, ring, s, b, kvh, rank * share + warp, M::warps, min(tiles, (rank + 1) * share), q, qs,
        masks, o, [&] {
            for (int r = warp; r < M::rows; r += M::warps) {
                const float f = rotate_row<E, D, SPLIT>(p, s, kvh, row_base + r, r < nrows, ent,
                                                        xs + warp * D, r, NT,
                                                        reinterpret_cast<__half *>(qm));
                if (lane == 0) {
                    factor[r] = f;
                    masks[r] = mask_of(p, s, r, nrows, row_base);
                }
            }
            __syncthreads();                               // and the table is complete
            q.take(qm + lane);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    qs[n][i] = factor[8 * n + 2 * c + i];
        });
    o.finish();
    // ---- the block's warps meet ----
    float *parts = reinterpret_cast<float *>(at_address(raw, M::lut_at));
    float *warp_m = reinterpret_cast<float *>(at_address(raw, M::warp_at));
    float *warp_l = warp_m + M::warps * M::rows;
    float *fin = reinterpret_cast<float *>(at_address(raw, M::fin_at));
    __syncthreads();                                      // the table and the rings are done with
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = warp * M::rows + 8 * n + 2 * c + i;
            float4 *to = reinterpret_cast<float4 *>(parts + r * M::stride + g * (D / 8));
#pragma unroll
            for (int j = 0; j < KS; j += 2)
                to[j / 2] = make_float4(o.acc[n][j][i], o.acc[n][j][2 + i], o.acc[n][j + 1][i],
                                        o.acc[n][j + 1][2 + i]);
            if (g == 0) {
                warp_m[r] = o.m[n][i];
                warp_l[r] = o.l[n][i];
            }
        }
    __syncthreads();
#pragma unroll
    for (int r = warp; r < M::rows; r += M::warps) {
        float mx = kNone, sum = 0.f, x[N];
#pragma unroll
        for (int w = 0; w < M::warps; ++w)
            mx = fmaxf(mx, warp_m[w * M::rows + r]);
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = 0.f;
#pragma unroll
        for (int w = 0; w < M::warps; ++w) {
            const float f = ex2(warp_m[w * M::rows + r] - mx);
            sum += f * warp_l[w * M::rows + r];
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(parts + (w * M::rows + r) * M::stride +
                                                                   lane * N + i);
                x[i] += f * v.x, x[i + 1] += f * v.y, x[i + 2] += f * v.z, x[i + 3] += f * v.w;
            }
        }
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4 *>(fin + r * M::stride + lane * N + i) =
                make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        if (lane == 0) {
            row_m[r] = mx;
            row_l[r] = sum;
        }
    }
    // ---- the cluster's blocks meet: rank k finishes rows k, k + splits, ... ----
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int r = rank + splits * warp; r < nrows; r += splits * M::warps) {
        // a lane each of the ranks' references and sums, then their rows in turn
        const float mk = lane < splits ? *cl.map_shared_rank(row_m + r, lane) : kNone;
        const float lk = lane < splits ? *cl.map_shared_rank(row_l + r, lane) : 0.f;
        float mx = mk;
#pragma unroll
        for (int k = 16; k; k >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        const float f = ex2(mk - mx);
        float sum = f * lk;
#pragma unroll
        for (int k = 16; k; k >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, k);
        float x[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = 0.f;
#pragma unroll 8
        for (int k = 0; k < splits; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, k);
            const float4 *src = reinterpret_cast<const float4 *>(
                cl.map_shared_rank(fin + r * M::stride + lane * N, k));
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 v = src[i / 4];
                x[i] += fk * v.x, x[i + 1] += fk * v.y, x[i + 2] += fk * v.z, x[i + 3] += fk * v.w;
            }
        }
        finish_row<E, D>(p, s, kvh, row_base + r, ent, xs + warp * D, x, sum);
    }
    cl.sync();                                            // shared memory stays until all have read
}

template <int D, int BITS, int NT, bool SPLIT>
cudaError_t launch_stream(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st) {
    using M = Stream<D, BITS, NT, SPLIT>;
    auto *kern = attend_tiles<D, BITS, NT, SPLIT>;
    static PerDevice ready;
    const cudaError_t e = ready.once([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, M::bytes);
    });
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kern, dim3(ws.most / M::warps), dim3(32 * M::warps), (size_t)M::bytes, st, p,
                      ws);
}

template <class E, int D, int BITS, int NT, bool SPLIT>
cudaError_t launch_near(const KvAttendParams &p, int splits, cudaStream_t st) {
    using M = Near<D, BITS, NT, SPLIT>;
    auto *kern = attend_near<E, D, BITS, NT, SPLIT>;
    static PerDevice ready;
    const cudaError_t e = ready.once([&] {
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               M::bytes);
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return err;
    });
    if (e != cudaSuccess)
        return e;
    const int row_tiles = (p.max_nodes * p.group + M::rows - 1) / M::rows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, p.c.kv_heads * row_tiles, p.B);
    cfg.blockDim = dim3(32 * M::warps);
    cfg.dynamicSmemBytes = M::bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p, row_tiles);
}

template <int BITS, int D, int NT>
cudaError_t launch_tile(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, int splits,
                        cudaStream_t st) {
    if (splits > 0)
        return dtype == OQ_BF16 ? launch_near<__nv_bfloat16, D, BITS, NT, false>(p, splits, st)
                                : launch_near<__half, D, BITS, NT, true>(p, splits, st);
    return dtype == OQ_BF16 ? launch_stream<D, BITS, NT, false>(p, ws, st)
                            : launch_stream<D, BITS, NT, true>(p, ws, st);
}

// Heads of 256 have no registers for two tiles of 8 rows.
template <int BITS>
cudaError_t launch_bits(const KvAttendParams &p, const KvAttendSpace &ws, int dtype, int splits,
                        cudaStream_t st) {
    if (p.c.d == 256)
        return launch_tile<BITS, 256, 1>(p, ws, dtype, splits, st);
    return p.max_nodes * p.group <= 8 ? launch_tile<BITS, 128, 1>(p, ws, dtype, splits, st)
                                      : launch_tile<BITS, 128, 2>(p, ws, dtype, splits, st);
}

// Workers of attend_tiles on `sms` SMs.
template <int BITS> int workers_bits(const KvAttendParams &p, int sms) {
    if (p.c.d == 256)
        return sms * Stream<256, BITS, 1, false>::warps;
    return sms * (p.max_nodes * p.group <= 8 ? Stream<128, BITS, 1, false>::warps
                                             : Stream<128, BITS, 2, false>::warps);
}

}  // namespace attend
}  // namespace oq
