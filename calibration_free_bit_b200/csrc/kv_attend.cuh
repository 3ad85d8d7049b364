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
//     tiles of 8 NT rows; a unit of work is 16 tokens of a tile, a worker is one warp, all warps of
//     all SMs have the same number of units, and no warp waits for another.  What a warp has of a
//     segment goes to the workspace; a second kernel joins the pieces in a fixed order;
//   - codes go from global memory straight to the registers of the lane that decodes them, 16 bytes
//     and less at a time, a unit ahead of their use, and through a table in shared memory with a
//     column a lane (no bank conflicts) into the operand of a matrix instruction;
//   - products are transposed, S^T = K Q^T and O^T = V^T P^T (mma.sync m16n8k16): the 16-wide side
//     is the cache, so 8 rows fill an instruction and an accumulator takes 32 registers.  The
//     instruction's order of a row's elements is free as long as both operands agree, which is how
//     a lane can own consecutive bytes of a row.  tcgen05 would need the decoded tile in shared or
//     tensor memory and has nothing to gain at these row counts.
// Scores, softmax statistics and sums are fp32.  fp16 enters in three places: the rotated query
// (over a power of two of its own), the centroids (times alpha, see build_kv_lut) and the weights
// p s_v, which are taken relative to a power of two above the row's largest s_v and times 2^6 to
// 2^14: what a token adds is resolved down to 2^-31 of the largest.  With SPLIT (fp16 outputs) query
// and weights enter as a sum of two fp16 numbers, so that only the centroids' rounding is left.
#pragma once
#ifndef KW
#define KW 16
#endif

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

// One unit's 16 tokens: codes and norms as this lane needs them.
template <int D, int BITS> struct Tile {
    using S = Shape<D, BITS>;
    uint32_t k[2][S::kw];        // key rows of tokens g, g + 8: elements c D/4 ..
    uint32_t v[4][S::vw];        // value rows of tokens 2c, 2c+1, 2c+8, 2c+9: elements g D/8 ..
    float kn[2], vn[2];          // norms of tokens g, g + 8
    bool ok;                     // the page exists

    // (codes of a missing page stay as they are: they are not seen, and the norms are 0)
    __device__ __forceinline__ void keys(const KvAttendParams &p, int page, int at, int kvh, int g,
                                         int c) {
        ok = page >= 0 && page < p.c.pages;
        kn[0] = kn[1] = vn[0] = vn[1] = 0.f;
        if (ok) {
            const long long row = (((long long)page * p.c.kv_heads + kvh) << p.c.page_log2) + at;
            const uint8_t *kr = p.c.codes[0] + row * S::row_bytes + g * S::row_bytes + c * S::k_bytes;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                load_words<S::kw, S::k_bytes>(k[i], kr + 8 * i * S::row_bytes);
                kn[i] = __ldg(p.c.norms[0] + row + g + 8 * i);
                vn[i] = __ldg(p.c.norms[1] + row + g + 8 * i);
            }
        }
    }
    __device__ __forceinline__ void values(const KvAttendParams &p, int page, int at, int kvh,
                                           int g, int c) {
        if (page >= 0 && page < p.c.pages) {
            const long long row = (((long long)page * p.c.kv_heads + kvh) << p.c.page_log2) + at;
            const uint8_t *vr = p.c.codes[1] + row * S::row_bytes + 2 * c * S::row_bytes +
                                (S::v_shared ? g >> 1 : g) * S::v_bytes;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_words<S::vw, S::v_bytes>(v[i],
                                              vr + ((i & 1) + 8 * (i >> 1)) * S::row_bytes);
        }
    }

    // The words of value row i that hold this lane's elements.
    __device__ __forceinline__ void share(int i, int g, uint32_t (&w)[S::vu]) const {
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
    // Warps of the one CTA on an SM: as many as its registers hold.
    static constexpr int warps = D == 128 && NT == 1 ? (SPLIT || BITS == 8 ? 12 : KW) : 8;   // KW
    static constexpr int rows = 8 * NT;
    // queries stay in shared memory where registers do not hold them beside the accumulators
    static constexpr bool q_shared = D == 256 && NT == 2;
    static constexpr int q_words = rows * D / 4 * (SPLIT ? 2 : 1);           // uint2
    // a warp's own: queries (q_shared) and masks
    static constexpr int mask_at = q_shared ? q_words * 8 : 0;
    static constexpr int own = mask_at + rows * 8;
    static constexpr int bytes = Lut<BITS, true>::bytes + warps * own;
};

template <class E, int D, int BITS, int NT, bool SPLIT>
__global__ void __launch_bounds__(32 * Smem<D, BITS, NT, SPLIT>::warps, 1)
attend_tiles(const KvAttendParams p, const KvAttendSpace ws) {
    using S = Shape<D, BITS>;
    using M = Smem<D, BITS, NT, SPLIT>;
    constexpr int KS = D / 16;
    extern __shared__ __align__(128) unsigned char sm[];
    unsigned char *lut = sm;

    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    unsigned char *own = sm + Lut<BITS, true>::bytes + warp * M::own;
    unsigned long long *masks = reinterpret_cast<unsigned long long *>(own + M::mask_at);
    fill_lut<BITS, true>(lut, p.lut);
    __syncthreads();
    pdl_wait();
    const uint32_t col = lut_column<BITS>(lane);
    // neighbouring workers on different SMs: few units reach all of them
    const long long worker = (long long)warp * gridDim.x + blockIdx.x;
    Walk walk = take_range(p, ws, worker);
    Piece piece;
    while (next_piece<NarrowForm<NT>>(p, walk, piece)) {
    const Seq &s = piece.s;
    const int kvh = piece.kvh, nrows = piece.nrows;
    const int last = piece.tile0 + piece.n;
    const int *table = p.table + (long long)piece.b * p.table_width;
    const int in_page = (1 << p.c.page_log2) - 1;
    int t = piece.tile0;
    Tile<D, BITS> cur;
    bool bad_page = false;
    // a tile's place: its page now, where its rows are when they are loaded
    auto place = [&](int t) -> int { return t < last ? __ldg(table + ((t << 4) >> p.c.page_log2)) : -1; };
    int page = place(t), page1 = place(t + 1);
    cur.keys(p, page, (t << 4) & in_page, kvh, g, c);
    cur.values(p, page, (t << 4) & in_page, kvh, g, c);

    // B operands of S^T = K Q^T: row n = g, elements c D/4 + 4 ks + {0, 1}, {2, 3} (rotate_queries)
    const long long sigma = (long long)piece.b * ws.segments + piece.seg;
    const uint2 *qg = ws.queries + sigma * M::q_words + lane;
    const uint2 *qsm = reinterpret_cast<const uint2 *>(own) + lane;
    uint2 qf[M::q_shared ? 1 : NT][M::q_shared ? 1 : KS];
    uint2 ql[SPLIT && !M::q_shared ? NT : 1][SPLIT && !M::q_shared ? KS : 1];
    if constexpr (!M::q_shared) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                qf[n][ks] = __ldcg(qg + (n * KS + ks) * 32);
                if constexpr (SPLIT)
                    ql[n][ks] = __ldcg(qg + ((NT + n) * KS + ks) * 32);
            }
    } else {
        __syncwarp();
        for (int i = 0; i < M::q_words / 32; ++i)
            reinterpret_cast<uint2 *>(own)[i * 32 + lane] = __ldcg(qg + i * 32);
    }
    float qs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        qs[n][0] = __ldcg(ws.factors + sigma * M::rows + 8 * n + 2 * c);
        qs[n][1] = __ldcg(ws.factors + sigma * M::rows + 8 * n + 2 * c + 1);
    }
    __syncwarp();
    if (lane < M::rows) {
        const int node = (piece.row_base + lane) / p.group;
        masks[lane] = lane >= nrows ? 0ull
                      : p.mask      ? (unsigned long long)p.mask[s.row0 + node]
                                    : (2ull << node) - 1ull;
    }
    __syncwarp();

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

    for (; t < last; ++t) {
        const int page2 = place(t + 2);
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
                    q = M::q_shared ? qsm[((NT + n) * KS + ks) * 32]
                                    : ql[M::q_shared ? 0 : n][M::q_shared ? 0 : ks];
                    mma16816(st[n], a, q.x, q.y);
                }
            }
        }
        // the next unit's keys are under way from here, its values from the end of this one: each a
        // part of a unit ahead of its use, in the registers that this unit has done with
        const float kn[2] = {cur.kn[0], cur.kn[1]}, vn[2] = {cur.vn[0], cur.vn[1]};
        const bool ok = cur.ok;
        cur.keys(p, page1, ((t + 1) << 4) & in_page, kvh, g, c);
        // scores of tokens g, g + 8 and rows 2c, 2c + 1, in powers of two
        bool grow = false;
        const int tok = t << 4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                st[n][i] *= kn[i >> 1] * qs[n][i & 1];
        if (!ok || tok + 16 > s.prefix) {             // the page is missing, or the tile has nodes
            bad_page |= !ok;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int node = tok + g + 8 * (i >> 1) - s.prefix;
                    const bool see = ok && (node < 0 || (node < s.nodes &&
                                     ((masks[8 * n + 2 * c + (i & 1)] >> node) & 1ull)));
                    if (!see)
                        st[n][i] = -CUDART_INF_F;
                    else
                        grow |= vn[i >> 1] > vs[n][i & 1];
                }
        } else {
            const float v = fmaxf(vn[0], vn[1]);
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
                    float v = fmaxf(st[n][i] > -CUDART_INF_F ? vn[0] : 0.f,
                                    st[n][2 + i] > -CUDART_INF_F ? vn[1] : 0.f);
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
                w[i] = e * (vn[i >> 1] * vinv[n][i & 1]);
            }
            if (!ok || tok + 16 > s.prefix) {         // what is not seen may have any norm
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
            cur.share(i, g, vw[i]);
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
        cur.values(p, page1, ((t + 1) << 4) & in_page, kvh, g, c);
        page1 = page2;
    }
    if (bad_page && lane == 0)
        atomicOr(p.err, AT_ERR_PAGE);

    // ---- the piece goes to its slot ----
    const long long slot = (long long)piece.b * ws.segments + piece.seg + worker;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int k = 4; k < 32; k <<= 1)
                l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], k);
            const int r = 8 * n + 2 * c + i;
            if (r >= nrows)
                continue;
            if (g == 0) {
                ws.stat[slot * 2 * ws.rows + r] = m[n][i];
                ws.stat[(slot * 2 + 1) * ws.rows + r] = l[n][i];
            }
            const float f = vs[n][i] * (1.0f / kWeightScale);
            float4 *dst = reinterpret_cast<float4 *>(ws.part + (slot * ws.rows + r) * D + g * (D / 8));
#pragma unroll
            for (int j = 0; j < KS; j += 2)
                dst[j / 2] = make_float4(acc[n][j][i] * f, acc[n][j][2 + i] * f,
                                         acc[n][j + 1][i] * f, acc[n][j + 1][2 + i] * f);
        }
    }
}

template <class E, int D, int BITS, int NT, bool SPLIT>
cudaError_t launch_tiles(const KvAttendParams &p, KvAttendSpace ws, cudaStream_t st) {
    using M = Smem<D, BITS, NT, SPLIT>;
    auto *kern = attend_tiles<E, D, BITS, NT, SPLIT>;
    static PerDevice ready;
    const cudaError_t e = ready.once([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, M::bytes);
    });
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kern, dim3(ws.most / M::warps), dim3(32 * M::warps), (size_t)M::bytes, st, p,
                      ws);
}

// Workers of a launch on `sms` SMs.
template <int D, int BITS> int workers_on(int sms, bool split, int rows) {
    if (rows <= 8)
        return sms * (split ? Smem<D, BITS, 1, true>::warps : Smem<D, BITS, 1, false>::warps);
    return sms * (split ? Smem<D, BITS, 2, true>::warps : Smem<D, BITS, 2, false>::warps);
}

template <class E, int D, int BITS, bool SPLIT>
cudaError_t launch_rows(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st) {
    if (p.max_nodes * p.group <= 8)
        return launch_tiles<E, D, BITS, 1, SPLIT>(p, ws, st);
    return launch_tiles<E, D, BITS, 2, SPLIT>(p, ws, st);
}

template <int BITS>
cudaError_t launch_bits(const KvAttendParams &p, const KvAttendSpace &ws, int dtype,
                        cudaStream_t st) {
    if (dtype == OQ_BF16)
        return p.c.d == 128 ? launch_rows<__nv_bfloat16, 128, BITS, false>(p, ws, st)
                            : launch_rows<__nv_bfloat16, 256, BITS, false>(p, ws, st);
    return p.c.d == 128 ? launch_rows<__half, 128, BITS, true>(p, ws, st)
                        : launch_rows<__half, 256, BITS, true>(p, ws, st);
}

template <int BITS> int workers_bits(const KvAttendParams &p, int dtype, int sms) {
    const int rows = p.max_nodes * p.group;
    return p.c.d == 128 ? workers_on<128, BITS>(sms, dtype != OQ_BF16, rows)
                        : workers_on<256, BITS>(sms, dtype != OQ_BF16, rows);
}

}  // namespace attend
}  // namespace oq
