// kv_attend.cuh -- attention of drafted tokens over the quantised cache, one instance a bit width
// (kv_attend_b*.cu); launch_kv_attend (kv_attend.cu) picks it.
//
// o = sum_t p_t v_hat_t, p = softmax_t(scale * q . k_hat_t), over the visible cached tokens t of
// the row's sequence: its prefix, and those of its drafted tokens that the row's mask names (bit
// j: node j; without a mask, nodes up to its own).  R is orthogonal, so q . k_hat = (R q) .
// centroid[code] s / sqrt(d): a row's query is rotated once, before the loop, and R^T is applied
// once, to the finished row.
//
// What bounds it is the cache's bytes (a token of one head: two rows of codes and two norms), and
// behind them the decode of two codes to a pair of fp16 centroids.  So:
//   - the rows of one key head (its query heads times the nodes) share a pass over its tokens, in
//     tiles of 8 NT rows, and a tile's tokens are split over a cluster of CTAs (flash decoding),
//     whose partial results meet in shared memory: one launch, no workspace, a fixed order;
//   - codes go from global memory straight to the registers of the lane that decodes them, 16 bytes
//     and less at a time, a step ahead of their use, and through a table in shared memory with a
//     column a lane (no bank conflicts) into the operand of a matrix instruction;
//   - products are transposed, S^T = K Q^T and O^T = V^T P^T (mma.sync m16n8k16): the 16-wide side
//     is the cache, so 8 rows fill an instruction and an accumulator takes 32 registers.  The
//     instruction's order of a row's elements is free as long as both operands agree, which is how
//     a lane can own consecutive bytes of a row.  tcgen05 would need the decoded tile in shared or
//     tensor memory and has nothing to gain at these row counts.
// Scores, softmax statistics and sums are fp32.  fp16 enters in three places: the rotated query
// (over a power of two of its own), the centroids (times alpha, see build_kv_lut) and the weights
// p s_v, which are taken relative to a power of two above the row's largest s_v and times 2^6 to
// 2^14: what a token adds is resolved down to 2^-31 of the largest.  With SPLIT (fp16 outputs) query and
// weights enter as a sum of two fp16 numbers, so that only the centroids' rounding is left.
#pragma once

#include <cooperative_groups.h>

#include "kv_attend_ops.cuh"
#include "kv_internal.h"
#include "kv_lut.cuh"
#include "kv_ops.cuh"

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

constexpr int kWarps = 4;
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

// One step's 16 tokens: codes and norms as this lane needs them.
template <int D, int BITS> struct Tile {
    using S = Shape<D, BITS>;
    uint32_t k[2][S::kw];        // key rows of tokens g, g + 8: elements c D/4 ..
    uint32_t v[4][S::vw];        // value rows of tokens 2c, 2c+1, 2c+8, 2c+9: elements g D/8 ..
    float kn[2], vn[2];          // norms of tokens g, g + 8
    bool ok;                     // the page exists

    __device__ __forceinline__ void load(const KvAttendParams &p, int page, int at, int kvh, int g,
                                         int c) {
        ok = page >= 0 && page < p.c.pages;
        if (!ok) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                kn[i] = vn[i] = 0.f;
#pragma unroll
                for (int j = 0; j < S::kw; ++j)
                    k[i][j] = 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < S::vw; ++j)
                    v[i][j] = 0;
            return;
        }
        const long long row = (((long long)page * p.c.kv_heads + kvh) << p.c.page_log2) + at;
        const uint8_t *kr = p.c.codes[0] + row * S::row_bytes;
        const uint8_t *vr = p.c.codes[1] + row * S::row_bytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            load_words<S::kw, S::k_bytes>(k[i], kr + (g + 8 * i) * S::row_bytes + c * S::k_bytes);
            kn[i] = __ldg(p.c.norms[0] + row + g + 8 * i);
            vn[i] = __ldg(p.c.norms[1] + row + g + 8 * i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            load_words<S::vw, S::v_bytes>(
                v[i], vr + (2 * c + (i & 1) + 8 * (i >> 1)) * S::row_bytes +
                          (S::v_shared ? g >> 1 : g) * S::v_bytes);
    }

    // The words of value row i that hold this lane's elements.
    __device__ __forceinline__ void values(int i, int g, uint32_t (&w)[S::vu]) const {
        if constexpr (S::v_shared) {                 // 48 of 96 bits
            w[0] = (g & 1) ? (v[i][1] >> 16) | (v[i][2] << 16) : v[i][0];
            w[1] = (g & 1) ? v[i][2] >> 16 : v[i][1];
        } else {
#pragma unroll
            for (int j = 0; j < S::vw; ++j)
                w[j] = v[i][j];
        }
    }
};

template <int D, int BITS, int NT, bool SPLIT> struct Smem {
    static constexpr int rows = 8 * NT;
    // queries stay in shared memory where registers do not hold them beside the accumulators
    static constexpr bool q_shared = D == 256 && NT == 2;
    static constexpr int part = (D / 16) * NT * 4 * 32 * 4 + NT * 8 * 32 * 4;  // a warp's state
    static constexpr int fin_stride = D + 4;                                 // floats
    static constexpr int big_a = Lut<BITS, true>::bytes > (kWarps / 2) * part
                                     ? Lut<BITS, true>::bytes : (kWarps / 2) * part;
    static constexpr int fin = rows * fin_stride * 4;
    static constexpr int big = (big_a > fin ? big_a : fin);                  // table, then partials
    static constexpr int q_at = big;
    static constexpr int q_half = rows * D;                                  // halves
    static constexpr int q_bytes = q_half * 2 * (SPLIT ? 2 : 1);
    static constexpr int x_at = q_at + q_bytes;                              // [kWarps][D] floats
    static constexpr int mask_at = x_at + kWarps * D * 4;
    static constexpr int stat_at = mask_at + rows * 8;                       // qs, m, l: [rows]
    static constexpr int bytes = stat_at + rows * 12;
};

template <class E, int D, int BITS, int NT, bool SPLIT>
__global__ void __launch_bounds__(32 * kWarps)
attend_tiles(const KvAttendParams p, const int row_tiles) {
    using S = Shape<D, BITS>;
    using M = Smem<D, BITS, NT, SPLIT>;
    constexpr int N = D / 32, KS = D / 16;
    extern __shared__ __align__(128) unsigned char sm[];
    namespace cg = cooperative_groups;
    unsigned char *lut = sm;
    __half *qh = reinterpret_cast<__half *>(sm + M::q_at);
    float *xs = reinterpret_cast<float *>(sm + M::x_at);
    unsigned long long *masks = reinterpret_cast<unsigned long long *>(sm + M::mask_at);
    float *qscale = reinterpret_cast<float *>(sm + M::stat_at);
    float *row_m = qscale + M::rows, *row_l = row_m + M::rows;

    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int rank = blockIdx.x, splits = gridDim.x;       // the cluster is the whole x dimension
    const int kvh = blockIdx.y / row_tiles, tile = blockIdx.y - kvh * row_tiles;
    const int b = blockIdx.z;
    fill_lut<BITS, true>(lut, p.lut);
    uint32_t ent[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        ent[i] = p.ent[lane * N + i];
    pdl_wait();
    Seq s;
    if (!load_seq(p, b, &s, blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0))
        return;                                            // the whole cluster returns
    const int rows_all = s.nodes * p.group, row_base = tile * M::rows;
    if (row_base >= rows_all)
        return;
    const int nrows = min(M::rows, rows_all - row_base);

    // ---- this warp's tokens: tiles of 16, every kWarps-th of the rank's share; the first are on
    // their way while the queries are rotated ----
    const int total = s.prefix + s.nodes;
    const int tiles = (total + 15) >> 4, share = (tiles + splits - 1) / splits;
    const int last = min(tiles, (rank + 1) * share);
    const int *table = p.table + (long long)b * p.table_width;
    const int in_page = (1 << p.c.page_log2) - 1;
    const uint32_t col = lut_column<BITS>(lane);
    int t = rank * share + warp;
    Tile<D, BITS> ping, pong;
    int page = 0;
    bool bad_page = false;
    if (t < last) {
        ping.load(p, table[(t << 4) >> p.c.page_log2], (t << 4) & in_page, kvh, g, c);
        if (t + kWarps < last)
            page = table[((t + kWarps) << 4) >> p.c.page_log2];
    }

    // ---- rotated queries, fp16 over a power of two a row ----
    for (int r = warp; r < M::rows; r += kWarps) {
        float z[N];
        if (r < nrows) {
            const int node = (row_base + r) / p.group, e = (row_base + r) - node * p.group;
            const long long row = s.row0 + node;
            const E *q = static_cast<const E *>(p.q) + row * p.q_stride + (kvh * p.group + e) * D;
#pragma unroll
            for (int i = 0; i < N; ++i)
                xs[warp * D + i * 32 + lane] = to_f32(q[i * 32 + lane]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float v = xs[warp * D + (ent[i] & 0x7fffu)];
                z[i] = (ent[i] & 0x8000u) ? -v : v;
            }
            warp_wht<D>(z, p.h, lane);
            if (lane == 0)
                masks[r] = p.mask ? (unsigned long long)p.mask[row] : (2ull << node) - 1ull;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                z[i] = 0.f;
            if (lane == 0)
                masks[r] = 0;
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
            // as the lanes take it: [row / 8][step][lane][4], lane = 4 (row % 8) + quarter
            const int x = lane * N + i, y = x % (D / 4);
            const int to = (((r >> 3) * KS + (y >> 2)) * 32 + (r & 7) * 4 + x / (D / 4)) * 4 + (y & 3);
            qh[to] = hi;
            if constexpr (SPLIT)
                qh[M::q_half + to] = __float2half_rn(v - __half2float(hi));
        }
        if (lane == 0)
            qscale[r] = up * p.qk_scale;
        __syncwarp();
    }
    __syncthreads();
    // B operands of S^T = K Q^T: row n = g, elements c D/4 + 4 ks + {0, 1}, {2, 3}
    const uint2 *qsm = reinterpret_cast<const uint2 *>(qh) + lane;
    uint2 qf[M::q_shared ? 1 : NT][M::q_shared ? 1 : KS];
    uint2 ql[SPLIT && !M::q_shared ? NT : 1][SPLIT && !M::q_shared ? KS : 1];
    if constexpr (!M::q_shared) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                qf[n][ks] = qsm[(n * KS + ks) * 32];
                if constexpr (SPLIT)
                    ql[n][ks] = qsm[M::q_half / 4 + (n * KS + ks) * 32];
            }
    }
    float qs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        qs[n][0] = qscale[8 * n + 2 * c];
        qs[n][1] = qscale[8 * n + 2 * c + 1];
    }

    float acc[NT][KS][4];
    float m[NT][2], l[NT][2];                     // reference and sum
    float vs[NT][2], vinv[NT][2];                 // power of two over s_v, kWeightScale over it
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

    // One step: 16 tokens from token 16 t on.
    auto step = [&](const Tile<D, BITS> &cur, int t) {
        // S^T = K Q^T
        float st[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                st[n][i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t a[4];
            quad<BITS, true>(lut, cur.k[0], ks, col, a[0], a[2]);
            quad<BITS, true>(lut, cur.k[1], ks, col, a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint2 q = M::q_shared ? qsm[(n * KS + ks) * 32]
                                      : qf[M::q_shared ? 0 : n][M::q_shared ? 0 : ks];
                mma16816(st[n], a, q.x, q.y);
                if constexpr (SPLIT) {
                    q = M::q_shared ? qsm[M::q_half / 4 + (n * KS + ks) * 32]
                                    : ql[M::q_shared ? 0 : n][M::q_shared ? 0 : ks];
                    mma16816(st[n], a, q.x, q.y);
                }
            }
        }
        // scores of tokens g, g + 8 and rows 2c, 2c + 1, in powers of two
        bool grow = false;
        const int tok = t << 4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                st[n][i] *= cur.kn[i >> 1] * qs[n][i & 1];
        if (!cur.ok || tok + 16 > s.prefix) {             // the page is missing, or the tile has nodes
            bad_page |= !cur.ok;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int node = tok + g + 8 * (i >> 1) - s.prefix;
                    const bool see = cur.ok && (node < 0 || (node < s.nodes &&
                                     ((masks[8 * n + 2 * c + (i & 1)] >> node) & 1ull)));
                    if (!see)
                        st[n][i] = -CUDART_INF_F;
                    else
                        grow |= cur.vn[i >> 1] > vs[n][i & 1];
                }
        } else {
            const float v = fmaxf(cur.vn[0], cur.vn[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                grow |= v > vs[n][0] || v > vs[n][1];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                grow |= fmaxf(st[n][i], st[n][2 + i]) > m[n][i] + kSlack;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float up = fmaxf(st[n][i], st[n][2 + i]);
                    float v = fmaxf(st[n][i] > -CUDART_INF_F ? cur.vn[0] : 0.f,
                                    st[n][2 + i] > -CUDART_INF_F ? cur.vn[1] : 0.f);
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) {
                        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, k));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
                    }
                    up = fmaxf(up, m[n][i]);
                    f[i] = ex2(m[n][i] - up);
                    m[n][i] = up;
                    l[n][i] *= f[i];
                    if (v > vs[n][i]) {
                        // the power of two above, with room for a quarter more, in [2^-100, 2^127]
                        const uint32_t p2 =
                            (__float_as_uint(v * 1.25f) & 0x7f800000u) + 0x00800000u;
                        const float nv = __uint_as_float(min(max(p2, 27u << 23), 254u << 23));
                        f[i] *= vs[n][i] / nv;
                        vs[n][i] = nv;
                        vinv[n][i] = kWeightScale / nv;
                    }
                }
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[n][j][i] *= f[i & 1];
            }
        }
        // weights
        uint32_t pb[NT][2], pl[SPLIT ? NT : 1][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = ex2(st[n][i] - m[n][i & 1]);
                l[n][i & 1] += e;
                w[i] = e * (cur.vn[i >> 1] * vinv[n][i & 1]);
            }
            if (!cur.ok || tok + 16 > s.prefix) {         // what is not seen may have any norm
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
                    pl[n][k] = transpose8x8(half2_rest(w[2 * k], w[2 * k + 1], hi));
            }
        }
        // O^T += V^T P^T: rows of tile j are elements g D/8 + 2j and 2j + 1
        uint32_t vw[4][S::vu];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            cur.values(i, g, vw[i]);
        mixed<BITS>(vw[0], vw[1]);
        mixed<BITS>(vw[2], vw[3]);
#pragma unroll
        for (int j = 0; j < KS; j += 2) {
            uint32_t x[4], y[4];
            quad_of_two<BITS, true>(lut, vw[0], vw[1], j / 2, col, x);
            quad_of_two<BITS, true>(lut, vw[2], vw[3], j / 2, col, y);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t a[4] = {x[2 * h], x[2 * h + 1], y[2 * h], y[2 * h + 1]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma16816(acc[n][j + h], a, pb[n][0], pb[n][1]);
                    if constexpr (SPLIT)
                        mma16816(acc[n][j + h], a, pl[n][0], pl[n][1]);
                }
            }
        }
    };
    // the tile after t, and the page of the one after that
    auto fetch = [&](Tile<D, BITS> &to, int t) {
        const int tn = t + kWarps;
        if (tn < last) {
            to.load(p, page, (tn << 4) & in_page, kvh, g, c);
            if (tn + kWarps < last)
                page = table[((tn + kWarps) << 4) >> p.c.page_log2];
        }
    };
    for (; t < last; t += 2 * kWarps) {
        fetch(pong, t);
        step(ping, t);
        if (t + kWarps >= last)
            break;
        fetch(ping, t + kWarps);
        step(pong, t + kWarps);
    }
    if (bad_page && lane == 0)
        atomicOr(p.err, AT_ERR_PAGE);

    // ---- the block's warps meet ----
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
#pragma unroll
    for (int half = kWarps / 2; half >= 1; half >>= 1) {
        __syncthreads();                                  // the table / the last round is done with
        float *mine = reinterpret_cast<float *>(sm + (warp & (half - 1)) * M::part) + lane;
        if (warp >= half && warp < 2 * half) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mine[((n * KS + j) * 4 + i) * 32] = acc[n][j][i];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mine[(NT * KS * 4 + n * 4 + i) * 32] = m[n][i];
                    mine[(NT * KS * 4 + n * 4 + 2 + i) * 32] = l[n][i];
                }
            }
        }
        __syncthreads();
        if (warp < half) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[2], h[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float om = mine[(NT * KS * 4 + n * 4 + i) * 32];
                    const float ol = mine[(NT * KS * 4 + n * 4 + 2 + i) * 32];
                    const float mn = fmaxf(m[n][i], om);
                    f[i] = ex2(m[n][i] - mn);
                    h[i] = ex2(om - mn);
                    m[n][i] = mn;
                    l[n][i] = l[n][i] * f[i] + ol * h[i];
                }
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[n][j][i] = acc[n][j][i] * f[i & 1] +
                                       mine[((n * KS + j) * 4 + i) * 32] * h[i & 1];
            }
        }
    }
    __syncthreads();
    float *fin = reinterpret_cast<float *>(sm);           // [rows][fin_stride]
    if (warp == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * n + 2 * c + i;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    fin[r * M::fin_stride + g * (D / 8) + 2 * j] = acc[n][j][i];
                    fin[r * M::fin_stride + g * (D / 8) + 2 * j + 1] = acc[n][j][2 + i];
                }
                if (g == 0) {
                    row_m[r] = m[n][i];
                    row_l[r] = l[n][i];
                }
            }
    }
    // ---- the cluster's blocks meet: rank k finishes rows k, k + splits, ... ----
    cg::cluster_group cl = cg::this_cluster();
    if (splits > 1)
        cl.sync();
    else
        __syncthreads();
    for (int r = rank + splits * warp; r < nrows; r += splits * kWarps) {
        float mx = kNone;
        for (int k = 0; k < splits; ++k)
            mx = fmaxf(mx, *cl.map_shared_rank(row_m + r, k));
        float o[N], sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            o[i] = 0.f;
        for (int k = 0; k < splits; ++k) {
            const float f = ex2(*cl.map_shared_rank(row_m + r, k) - mx);
            sum += f * *cl.map_shared_rank(row_l + r, k);
            const float4 *src = reinterpret_cast<const float4 *>(
                cl.map_shared_rank(fin + r * M::fin_stride + lane * N, k));
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 v = src[i / 4];
                o[i] += f * v.x, o[i + 1] += f * v.y, o[i + 2] += f * v.z, o[i + 3] += f * v.w;
            }
        }
        warp_wht<D>(o, p.h, lane);
        const float inv = sum == 0.f ? 0.f : p.o_scale / sum;      // nothing seen: zeros
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i)
            xs[warp * D + (ent[i] & 0x7fffu)] = inv * ((ent[i] & 0x8000u) ? -o[i] : o[i]);
        __syncwarp();
        const int node = (row_base + r) / p.group, e = (row_base + r) - node * p.group;
        E *y = static_cast<E *>(p.out) + (s.row0 + node) * p.out_stride + (kvh * p.group + e) * D;
#pragma unroll
        for (int i = 0; i < N; ++i)
            y[i * 32 + lane] = from_f32<E>(xs[warp * D + i * 32 + lane]);
    }
    if (splits > 1)
        cl.sync();                                        // shared memory stays until all have read
}

template <class E, int D, int BITS, int NT, bool SPLIT>
cudaError_t launch_tiles(const KvAttendParams &p, int splits, cudaStream_t st) {
    using M = Smem<D, BITS, NT, SPLIT>;
    auto *kern = attend_tiles<E, D, BITS, NT, SPLIT>;
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
    const int rows = p.max_nodes * p.group, row_tiles = (rows + M::rows - 1) / M::rows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, p.c.kv_heads * row_tiles, p.B);
    cfg.blockDim = dim3(32 * kWarps);
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

template <class E, int D, int BITS, bool SPLIT>
cudaError_t launch_rows(const KvAttendParams &p, int splits, cudaStream_t st) {
    const int rows = p.max_nodes * p.group;
    if (rows <= 8)
        return launch_tiles<E, D, BITS, 1, SPLIT>(p, splits, st);
    return launch_tiles<E, D, BITS, 2, SPLIT>(p, splits, st);
}

template <int BITS>
cudaError_t launch_bits(const KvAttendParams &p, int dtype, int splits, cudaStream_t st) {
    if (dtype == OQ_BF16)
        return p.c.d == 128 ? launch_rows<__nv_bfloat16, 128, BITS, false>(p, splits, st)
                            : launch_rows<__nv_bfloat16, 256, BITS, false>(p, splits, st);
    return p.c.d == 128 ? launch_rows<__half, 128, BITS, true>(p, splits, st)
                        : launch_rows<__half, 256, BITS, true>(p, splits, st);
}

}  // namespace attend
}  // namespace oq
