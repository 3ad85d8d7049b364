// kv_wide.cuh -- the cache's attention for many rows a key head (trees of drafted tokens), heads of
// 128: tcgen05 with tiles of 128 rows by 128 tokens.  Method and checks: kv_attend.cuh; work list:
// kv_attend_ops.cuh; the pieces of a segment are joined by a second kernel (kv_attend.cu).
//
// One CTA per SM walks a contiguous range of units.  For a piece it rotates the 128 queries (one
// tcgen05.mma with the rotation's dense operand) and keeps them as the A operand in shared memory;
// then, per unit, decoder warps turn the codes of 128 tokens into the fp16 operands K (elements
// contiguous, K-major) and V (the same layout, read as N-major), a row a thread (of 6 and 8 bits half
// a row); S = Q K^T goes to tensor memory, two units' in turn; two softmax threads own a row, one for
// either half of the tokens, and put the weights, the A operand of O += P V, beside S, so that the next
// products do not wait for the last.  They take the weights with the row's reference as it is and look
// for a larger score on the way; only if a row of the two warps has passed it (kSlack) is a unit done
// again.
// A unit needs about a thousand cycles each of shared memory (at 4 bits 16384 lookups of two codes, 64
// KB of operands stored), of exponentials (16384) and of issue slots, and half of that of the tensor
// cores; it takes 4300, since none of its steps (decode, S, softmax, P V) has warps enough to hide its
// latencies, and more warps have too few registers.  B200, 4 bits: 2 sequences of 131 000 tokens with 31
// nodes, 8 key heads: 281 us in all (codes and norms at 1.02 TB/s); 8 bits: 16 sequences of 129 to 4095
// tokens with 61 nodes 160 us, 43 of them set-up and joining of their 256 segments.
//   - A group of 32 tokens that all rows see, with key norms of one order (nearly all of a prefix), has
//     them in the operand, times 2^-e: its scores share one factor, and the search for a new maximum is
//     a maximum over raw products.  Of any other group (with nodes, a loud key, a NaN) the operand is
//     bare centroids, and the norms multiply the products in fp32, token by token (a product is below
//     2^12, and the cache's write stores no norm above 2^64).  Value norms enter with the weights, a row
//     at a time.  So what a row does not see never reaches it, nor what stands beside it.  (Trees of 31
//     nodes as above take 416 us when all groups are bare, their norms spread over e^+-2 rms.)
//   - Queries, products of centroid and norm, and weights are one fp16 number each: errors of 1.8e-3 to
//     1.9e-3 of an output's length, of which its own rounding to bf16 is 1.65e-3.  A weight is resolved
//     down to 2^-31 of the longest value that its row sees.
#pragma once

#include "kv_attend_ops.cuh"
#include "kv_internal.h"
#include "kv_lut.cuh"
#include "kv_ops.cuh"
#include "sm100_common.cuh"

namespace oq {
namespace attend {

using namespace sm100;
using kvops::prmt;

namespace wide {

constexpr int kRows = 128, kTokens = 128, D = 128;
// Warps: softmax, four or eight decoders each for keys and values, and one that issues the products.
// (17 in all leave 96 registers a thread and 25 leave 72, since one scheduler has the odd warp: at 72,
// with 6 and 8 bits, 76 bytes a thread are spilled.)
constexpr int kSoftWarps = 8;
template <int BITS> struct Shape {
    static constexpr int parts = BITS > 4 ? 2 : 1;    // decoder threads a row
    static constexpr int dec_warps = 8 * parts;
    static constexpr int threads = 32 * (kSoftWarps + dec_warps + 1);
};
constexpr int kTile = 128 * D * 2;                    // an operand: 32 KB

// Shared memory by address (a CTA's own starts at 1024): the table at a multiple of its size, the
// operands behind it at multiples of 1024.
struct Smem {
    static constexpr int vn_at = kSharedStart;        // [2][128] value norms
    static constexpr int vm_at = vn_at + 1024;        // [2][128] the same over their power of two
    static constexpr int kn_at = vm_at + 1024;        // [2][128] factors of the tokens' products
    static constexpr int vlog_at = kn_at + 1024;      // [2][4] the powers' logarithms
    static constexpr int vmax_at = vlog_at + 32;      // [2][4] largest value norms
    static constexpr int bad_at = vmax_at + 32;       // [2][4] tokens of missing pages
    static constexpr int bare_at = bad_at + 32;       // [2][4] whether a group's factors differ
    static constexpr int pair_at = bare_at + 32;      // [2][2][128]: what a row's two threads tell
    static constexpr int work_at = pair_at + 2048;
    static constexpr int bars_at = work_at + 64;
    static constexpr int lut_at = 32768;
    static constexpr int q_at = 65536;
    static constexpr int k_at = q_at + kTile;         // two stages
    static constexpr int v_at = q_at + 3 * kTile;     // two stages
    static constexpr int bytes = q_at + 5 * kTile - kSharedStart;
    static_assert(bars_at + 128 <= lut_at && bytes <= 227 * 1024, "shared memory");
};
enum { B_K = 0, B_V = 2, B_S = 4, B_P = 6, B_PV = 8, B_Q = 10 };   // two each to B_Q

__device__ __forceinline__ uint32_t operand_at(int r, int ch) {
    return (uint32_t)(ch >> 3) * 16384u + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

// V as the B operand of P V: N (elements) contiguous.  Atoms of 64 elements by 8 tokens; the next
// 8 tokens lie 1024 bytes on, the next 64 elements 16 KB.
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(16384 >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ uint32_t idesc_q() {      // both operands bf16
    return idesc_f16(128, 128) | (1u << 7) | (1u << 10);
}

// 16 columns of tensor memory (the wait is in the same statement: nothing may touch the registers, not
// even a copy or a spill, while the load is on its way).
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
                 "%11, %12, %13, %14, %15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                   "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                   "r"(r[6]), "r"(r[7]) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

}  // namespace wide

template <int BITS>
__global__ void __launch_bounds__(wide::Shape<BITS>::threads, 1)
attend_wide(const KvAttendParams p, const uint4 *r_img, const KvAttendSpace ws) {
    using namespace wide;
    using S = wide::Smem;
    constexpr int kParts = Shape<BITS>::parts, kDecWarps = Shape<BITS>::dec_warps;
    constexpr int kThreads = Shape<BITS>::threads;
    extern __shared__ __align__(1024) unsigned char raw[];
    constexpr uint32_t base = 0;                      // offsets are addresses
    if (!starts_there(raw)) {                         // not where the layout expects it
        if (threadIdx.x == 0)
            atomicOr(p.err, AT_ERR_WAIT);
        return;
    }
    const uint32_t bars = base + S::bars_at;
    auto bar = [&](int i) { return bars + 8u * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(at_address(raw, S::bars_at + 112));
    volatile int *gone = reinterpret_cast<volatile int *>(at_address(raw, S::bars_at + 116));
    Walk *work = reinterpret_cast<Walk *>(at_address(raw, S::work_at));
    float *vn_s = reinterpret_cast<float *>(at_address(raw, S::vn_at));
    float *vm_s = reinterpret_cast<float *>(at_address(raw, S::vm_at));
    float *vlog_s = reinterpret_cast<float *>(at_address(raw, S::vlog_at));
    float *kn_s = reinterpret_cast<float *>(at_address(raw, S::kn_at));
    float *vmax_s = reinterpret_cast<float *>(at_address(raw, S::vmax_at));
    uint32_t *bad_s = reinterpret_cast<uint32_t *>(at_address(raw, S::bad_at));
    uint32_t *bare_s = reinterpret_cast<uint32_t *>(at_address(raw, S::bare_at));
    float *pair_s = reinterpret_cast<float *>(at_address(raw, S::pair_at));

    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    fill_lut<BITS, PLACED>(at_address(raw, S::lut_at), p.lut);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_K + i), kDecWarps / 2);
            mbar_init(bar(B_V + i), kDecWarps / 2);
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_P + i), kSoftWarps);
            mbar_init(bar(B_PV + i), 1);
        }
        mbar_init(bar(B_Q), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *gone = 0;
    }
    pdl_wait();
    if (warp == kSoftWarps + kDecWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        const Walk w = take_range(p, ws, blockIdx.x);
        if (lane == 0)
            *work = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    auto wait = [&](int i, uint32_t parity) {
        if (*gone)
            return;
        if (!mbar_wait(bar(i), parity & 1u)) {
            *gone = 1;
            atomicOr(p.err, AT_ERR_WAIT);
        }
    };

    auto meet = [&] {
        __syncwarp();
        tc_fence_before();
        asm volatile("bar.sync 0, %0;" ::"n"(kThreads) : "memory");
        tc_fence_after();
    };
    Walk walk = *work;
    Piece q;
    uint32_t done = 0;                               // units of the pieces so far: u counts them all,
                                                     // its stage is u & 1, its phase there u >> 1
    if (warp < kSoftWarps) {
        // ---------------- softmax: row r's tokens 64 half .. 64 half + 63 of a unit ----------------
        const int half = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t tO = lanes + 256 + 64 * half;
        float *mine_s = pair_s + 256 * half + r;
        const float *other_s = pair_s + 256 * (half ^ 1) + r;
        const int pair = 1 + (warp & 3);             // the barrier of a row's two warps
        auto both = [&] { asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory"); };
        auto any = [&](bool x) -> bool {             // of 64 threads
            uint32_t y;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                         "bar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(y) : "r"((uint32_t)x), "r"(pair) : "memory");
            return y != 0;
        };
        for (uint32_t pieces = 0; next_piece<WideForm>(p, walk, q); ++pieces) {
            const Seq &s = q.s;
            const int n = q.n, tile0 = q.tile0, nrows = q.nrows;
            // the rotation to K's first stage, the raw queries to V's (these warps have seen the end of
            // the last piece's products)
            {
                constexpr int per = kTile / 16 / (32 * kSoftWarps);
                uint4 v[per];
#pragma unroll
                for (int i = 0; i < per; ++i)
                    v[i] = __ldg(r_img + i * 32 * kSoftWarps + threadIdx.x);
#pragma unroll
                for (int i = 0; i < per; ++i)
                    reinterpret_cast<uint4 *>(at_address(raw, S::k_at))[i * 32 * kSoftWarps +
                                                                        threadIdx.x] = v[i];
                const int ch = threadIdx.x & 15;
#pragma unroll
                for (int i = 0; i < per; ++i) {
                    const int row = i * 16 + (threadIdx.x >> 4);
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (row < nrows) {
                        const int node = (q.row_base + row) / p.group;
                        const int e = q.row_base + row - node * p.group;
                        v[i] = *reinterpret_cast<const uint4 *>(
                            static_cast<const __nv_bfloat16 *>(p.q) + (s.row0 + node) * p.q_stride +
                            (q.kvh * p.group + e) * D + ch * 8);
                    }
                }
#pragma unroll
                for (int i = 0; i < per; ++i)
                    *reinterpret_cast<uint4 *>(at_address(raw, S::v_at) +
                                               operand_at(i * 16 + (threadIdx.x >> 4), ch)) = v[i];
            }
            fence_async_smem();
            meet();
            // rotated queries, fp16 over a power of two a row
            wait(B_Q, pieces);
            tc_fence_after();
            float big = 0.f;
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                uint32_t z[32];
                tmem_ld32(lanes + 64 * half + 32 * k, z);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    big = fmaxf(big, fabsf(__uint_as_float(z[i])));
            }
            *mine_s = big;
            both();
            big = fmaxf(big, *other_s);
            // 2^e <= big < 2^(e+1); values over 2^e stay below 2 (2^e and its inverse are normal)
            uint32_t ex = (__float_as_uint(big) >> 23) & 255u;
            ex = ex < 1u ? 1u : (ex > 253u ? 253u : ex);
            const float down = __uint_as_float((254u - ex) << 23);
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                uint32_t z[32];
                tmem_ld32(lanes + 64 * half + 32 * k, z);
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    auto f = [&](int j) { return __uint_as_float(z[i + j]) * down; };
                    *reinterpret_cast<uint4 *>(at_address(raw, S::q_at) +
                                               operand_at(r, 8 * half + 4 * k + i / 8)) =
                        make_uint4(half2_bits(f(0), f(1)), half2_bits(f(2), f(3)),
                                   half2_bits(f(4), f(5)), half2_bits(f(6), f(7)));
                }
            }
            fence_async_smem();
            const float qs = __uint_as_float(ex << 23) * p.qk_scale;   // factor of the row's scores
            unsigned long long mask = 0ull;
            if (r < nrows) {
                const int node = (q.row_base + r) / p.group;
                mask = p.mask ? (unsigned long long)p.mask[s.row0 + node] &
                                    (s.nodes >= 64 ? ~0ull : (1ull << s.nodes) - 1ull)
                              : (2ull << node) - 1ull;
            }
            meet();
            float m = kNone, l = 0.f, vs = 0.f, vinv = 0.f, vlog = 0.f;   // vlog: of vinv
            for (int i = 0; i < n; ++i) {
                const uint32_t u = done + i, st = u & 1u, phase = u >> 1;
                const uint32_t tS = lanes + 128 * st + 64 * half, tP = lanes + 384 + 64 * st + 32 * half;
                const int tok = (tile0 + i) * kTokens;
                wait(B_K + st, phase);                // factors and lost tokens
                wait(B_V + st, phase);                // value norms
                if (u >= 2)
                    wait(B_PV + st, phase - 1);       // the weights' place is free
                wait(B_S + st, phase);
                tc_fence_after();
                const float *kn = kn_s + 128 * st + 64 * half, *vn = vn_s + 128 * st + 64 * half;
                const float4 vm = *reinterpret_cast<const float4 *>(vmax_s + 4 * st);
                const uint4 bad = *reinterpret_cast<const uint4 *>(bad_s + 4 * st);
                const uint4 bare = *reinterpret_cast<const uint4 *>(bare_s + 4 * st);
                const bool edge = tok + kTokens > s.prefix || (bad.x | bad.y | bad.z | bad.w) ||
                                  (bare.x | bare.y | bare.z | bare.w);
                // tokens of this half's group k that this row sees
                auto seen = [&](int k) -> uint32_t {
                    const int first = tok + 64 * half + 32 * k - s.prefix;   // node of its first token
                    uint32_t v;
                    if (first <= -32)
                        v = ~0u;
                    else if (first < 0)
                        v = (uint32_t)(mask << -first) | ((1u << -first) - 1u);
                    else
                        v = first < 64 ? (uint32_t)(mask >> first) : 0u;
                    return v & ~bad_s[4 * st + 2 * half + k];
                };
#pragma unroll 1
                for (int again = 0;; ++again) {
                    // weights with the reference as it is; the row's largest score, and the largest
                    // value norm that it sees
                    float top = -CUDART_INF_F, vtop, sum;
                    if (!edge) {
                        // A group of 32 tokens has its norms over one power of two; that power, over
                        // the row's, enters with the exponent (below 2^-60 fp16 has nothing of it).
                        sum = 0.f;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t y[16];
                            tmem_ld16(tS + 16 * k, y);
                            const float f = qs * kn[16 * k];
                            const float lf = fmaxf(vlog_s[4 * st + 2 * half + (k >> 1)] + vlog, -60.f);
                            const float2 ff = make_float2(f, f), mm = make_float2(lf - m, lf - m);
                            float4 nv[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                nv[j] = *reinterpret_cast<const float4 *>(vm_s + 128 * st + 64 * half +
                                                                          16 * k + 4 * j);
                            float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                            float a[2];
                            uint32_t w[8];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                a[h] = fmaxf(__uint_as_float(y[h]), __uint_as_float(y[2 + h]));
#pragma unroll
                                for (int j = 4 + h; j < 16; j += 4)
                                    a[h] = max3(a[h], __uint_as_float(y[j]),
                                                __uint_as_float(y[j + 2]));
                            }
                            top = fmaxf(top, fmaxf(a[0], a[1]) * f);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float2 x = __ffma2_rn(make_float2(__uint_as_float(y[2 * j]),
                                                                        __uint_as_float(y[2 * j + 1])),
                                                            ff, mm);
                                const float2 e = make_float2(ex2(x.x), ex2(x.y));
                                ls[j & 1] = __fadd2_rn(ls[j & 1], e);
                                const float4 n4 = nv[j >> 1];
                                const float2 pw = __fmul2_rn(e, (j & 1) ? make_float2(n4.z, n4.w)
                                                                        : make_float2(n4.x, n4.y));
                                w[j] = half2_bits(pw.x, pw.y);
                            }
                            sum = fmaf((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y), ex2(-lf), sum);
                            tmem_st8(tP + 8 * k, w);
                        }
                        vtop = fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w));
                    } else {
                        // (selections, no branches: every lane sees other tokens)
                        sum = vtop = 0.f;
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t v = seen(k >> 1) >> (16 * (k & 1));
                            uint32_t y[16], w[8];
                            tmem_ld16(tS + 16 * k, y);
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 n4 = *reinterpret_cast<const float4 *>(vn + 16 * k + j);
                                const float4 k4 = *reinterpret_cast<const float4 *>(kn + 16 * k + j);
                                const float nv[4] = {n4.x, n4.y, n4.z, n4.w};
                                const float nk[4] = {k4.x, k4.y, k4.z, k4.w};
                                float pw[4];
#pragma unroll
                                for (int h = 0; h < 4; ++h) {
                                    const bool see = (v >> (j + h)) & 1u;
                                    const float x =
                                        see ? __uint_as_float(y[j + h]) * nk[h] * qs : -CUDART_INF_F;
                                    const float n1 = see ? nv[h] : 0.f, e = ex2(x - m);
                                    top = fmaxf(top, x);
                                    vtop = fmaxf(vtop, n1);
                                    sum += e;
                                    pw[h] = e * (n1 * vinv);
                                }
                                w[j / 2] = half2_bits(pw[0], pw[1]);
                                w[j / 2 + 1] = half2_bits(pw[2], pw[3]);
                            }
                            tmem_st8(tP + 8 * k, w);
                        }
                    }
                    if (again || !any(top > m + kSlack || vtop > vs)) {
                        l += sum;
                        break;
                    }
                    // a row of the two warps needs another reference: all 32 rows take theirs
                    mine_s[0] = top;
                    mine_s[128] = vtop;
                    both();
                    top = fmaxf(top, other_s[0]);
                    vtop = fmaxf(vtop, other_s[128]);
                    const float up = fmaxf(m, top);
                    float fac = ex2(m - up);
                    m = up;
                    l *= fac;
                    if (vtop > vs) {
                        const float nv = norm_scale(vtop);
                        fac *= vs / nv;
                        vs = nv;
                        vinv = kWeightScale / nv;
                        vlog = 133.f - (float)(__float_as_uint(nv) >> 23);
                    }
                    if (i > 0) {                      // the sums so far, once they are complete
                        wait(B_PV + (st ^ 1u), (u - 1) >> 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < 2; ++k) {
                            uint32_t z[32];
                            tmem_ld32(tO + 32 * k, z);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                z[j] = __float_as_uint(__uint_as_float(z[j]) * fac);
                            tmem_st32(tO + 32 * k, z);
                        }
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(B_P + st));
            }
            // ---- the piece goes to its slot ----
            done += n;
            wait(B_PV + ((done - 1) & 1u), (done - 1) >> 1);
            tc_fence_after();
            const long long slot = (long long)q.b * ws.segments + q.seg + blockIdx.x;
            both();                                   // what the other has written has been read
            *mine_s = l;
            both();
            if (half == 0 && r < nrows) {
                ws.stat[(slot * 2) * ws.rows + r] = m;
                ws.stat[(slot * 2 + 1) * ws.rows + r] = l + *other_s;
            }
            const float fac = vs * (1.0f / kWeightScale);
            float *dst = ws.part + (slot * ws.rows + r) * D + 64 * half;
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                uint32_t z[32];
                tmem_ld32(tO + 32 * k, z);
                if (r < nrows)
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        float o[8];
#pragma unroll
                        for (int h = 0; h < 8; ++h)
                            o[h] = __uint_as_float(z[j + h]) * fac;
                        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                     ::"l"(dst + 32 * k + j), "f"(o[0]), "f"(o[1]), "f"(o[2]),
                                     "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]), "f"(o[7])
                                     : "memory");
                    }
            }
            both();                                   // (before the next piece's first exchange)
        }
    } else if (warp < kSoftWarps + kDecWarps) {
        // ---------------- decoders: half a token's key row or value row a thread ----------------
        const int dt = threadIdx.x - 32 * kSoftWarps;
        while (next_piece<WideForm>(p, walk, q)) {
            const int n = q.n, tile0 = q.tile0, total = q.total, kvh = q.kvh, b = q.b;
            const int w = dt / (128 * kParts), part = (dt >> 7) & (kParts - 1), row = dt & 127;
            const int *table = p.table + (long long)b * p.table_width;
            const uint32_t col = lut_column<BITS, PLACED>(S::lut_at, lane);
            constexpr int words = 4 * BITS / kParts, own = 4 * words;     // a thread's codes, bytes
            // One unit ahead in registers and two ahead on the way to the L2; a page's index is
            // known three ahead, so that no load waits for another.
            struct Row {
                uint32_t codes[words];
                float norm;
                bool missing, valid;
            };
            auto page_of = [&](int i) -> int {
                const int tok = (tile0 + i) * kTokens + row;
                return i < n && tok < total ? table[tok >> p.c.page_log2] : -1;
            };
            auto row_of = [&](int i, int page) -> long long {
                return (((long long)page * p.c.kv_heads + kvh) << p.c.page_log2) +
                       (((tile0 + i) * kTokens + row) & ((1 << p.c.page_log2) - 1));
            };
            auto fetch = [&](int i, int page) {
                if (page >= 0 && page < p.c.pages) {
                    const uint8_t *at = pick(p.c.codes, w) + row_of(i, page) * (D * BITS / 8) + part * own;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
                }
            };
            auto load = [&](Row &to, int i, int page) {
                const bool real = i < n && (tile0 + i) * kTokens + row < total;
                to.valid = page >= 0 && page < p.c.pages;
                to.missing = real && !to.valid;
                to.norm = 0.f;
                if (to.valid) {
                    const long long at = row_of(i, page);
                    load_words<words, own>(
                        to.codes, pick(p.c.codes, w) + at * (D * BITS / 8) + part * own);
                    to.norm = pick(p.c.norms, w)[at];
                } else {
#pragma unroll
                    for (int k = 0; k < words; ++k)
                        to.codes[k] = 0;
                }
            };
            Row cur, nxt;
            int page1 = page_of(1), page2 = page_of(2);
            load(cur, 0, page_of(0));
            fetch(1, page1);
            meet();
            meet();
            for (int i = 0; i < n; ++i) {
                const uint32_t u = done + i, st = u & 1u, phase = u >> 1;
                load(nxt, i + 1, page1);
                fetch(i + 2, page2);
                const int page3 = page_of(i + 3);
                const float norm = cur.norm;
                const bool valid = cur.valid, missing = cur.missing;
                // the largest norm of the warp's 32 tokens (one group)
                float top = valid && norm > 0.f && norm < CUDART_INF_F ? norm : 0.f;
                top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
                const uint32_t lost = __ballot_sync(0xffffffffu, missing);
                uint32_t ex = (__float_as_uint(top) >> 23) & 255u;
                ex = ex < 28u ? 28u : (ex > 253u ? 253u : ex);
                // keys of a group of the prefix whose norms (0 apart) are within 2^6 of one another take
                // them along, as sums of two fp16 numbers (one alone moved a row's scores by up to 2^-12)
                const bool bare =
                    w > 0 || (tile0 + i) * kTokens + (row | 31) >= q.s.prefix ||
                    !__all_sync(0xffffffffu, norm == 0.f || (norm <= top && norm * 64.f >= top &&
                                                             norm >= 0x1p-99f));
                const float by = norm * __uint_as_float((254u - ex) << 23);
                const __half2 by_hi = __float2half2_rn(by);
                const __half2 by_lo = __float2half2_rn(by - __low2float(by_hi));
                // K's stage is free after S, its factors after the softmax, V's and its norms after P V
                if (u >= 2)
                    wait((w == 0 ? B_S : B_PV) + st, phase - 1);
                unsigned char *to = at_address(raw, (w == 0 ? S::k_at : S::v_at) + st * kTile);
                // four chunks of 8 elements at a time, so that their lookups are under way together
                // (the compiler does not move a load over a store to the operand)
#pragma unroll
                for (int k = 0; k < 16 / kParts; k += 4) {
                    uint4 v[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        quad<BITS, PLACED>(cur.codes, 2 * (k + h), col, v[h].x, v[h].y);
                        quad<BITS, PLACED>(cur.codes, 2 * (k + h) + 1, col, v[h].z, v[h].w);
                    }
                    if (!bare) {
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            __half2 *x = reinterpret_cast<__half2 *>(&v[h]);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                x[j] = __hfma2(x[j], by_hi, __hmul2(x[j], by_lo));
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        *reinterpret_cast<uint4 *>(to + operand_at(row, 16 / kParts * part + k + h)) = v[h];
                }
                cur = nxt;
                page1 = page2;
                page2 = page3;
                if (w == 0) {
                    if (part == 0) {
                        if (u >= 2)
                            wait(B_P + st, phase - 1);
                        kn_s[128 * st + row] = bare ? norm : __uint_as_float(ex << 23);
                        if (lane == 0) {
                            bad_s[4 * st + (warp & 3)] = lost;
                            bare_s[4 * st + (warp & 3)] = bare;
                            if (lost)
                                atomicOr(p.err, AT_ERR_PAGE);
                        }
                    }
                } else if (part == 0) {
                    vn_s[128 * st + row] = norm;
                    vm_s[128 * st + row] = norm * __uint_as_float((254u - ex) << 23);
                    if (lane == 0) {
                        vmax_s[4 * st + (warp & 3)] = top;
                        vlog_s[4 * st + (warp & 3)] = (float)(int)(ex - 127u);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar((w == 0 ? B_K : B_V) + st));
            }
            done += n;
        }
    } else {
        // ---------------- products: S two units ahead of P V ----------------
        while (next_piece<WideForm>(p, walk, q)) {
            const int n = q.n;
            meet();
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_ss(tmem, sw128_desc(base + S::v_at + (k >> 2) * 16384) + 2 * (k & 3),
                           sw128_desc(base + S::k_at + (k >> 2) * 16384) + 2 * (k & 3),
                           idesc_q(), k != 0);
                mma_commit(bar(B_Q));
            }
            meet();
            if (lane == 0) {
#pragma unroll 1
                for (int i = -2; i < n; ++i) {
                    if (i >= 0) {                     // O += P V of unit i
                        const uint32_t u = done + i, st = u & 1u;
                        wait(B_V + st, u >> 1);
                        wait(B_P + st, u >> 1);
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_ts(tmem + 256, tmem + 384 + 64 * st + 8 * k,
                                   v_desc(base + S::v_at + st * kTile + k * 2048),
                                   idesc_f16(128, 128) | (1u << 16), i > 0 || k != 0);
                        mma_commit(bar(B_PV + st));
                    }
                    if (i + 2 < n) {                  // S = Q K^T of unit i + 2 (S of unit i is read)
                        const uint32_t u = done + i + 2, st = u & 1u;
                        wait(B_K + st, u >> 1);
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_ss(tmem + 128 * st,
                                   sw128_desc(base + S::q_at + (k >> 2) * 16384) + 2 * (k & 3),
                                   sw128_desc(base + S::k_at + st * kTile + (k >> 2) * 16384) +
                                       2 * (k & 3),
                                   idesc_f16(128, 128), k != 0);
                        mma_commit(bar(B_S + st));
                    }
                }
            }
            __syncwarp();
            done += n;
        }
    }
    // Every product has been waited for by the softmax warps, so the tensor memory is free.
    meet();
    if (warp == kSoftWarps + kDecWarps)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

template <int BITS>
cudaError_t launch_wide(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st) {
    auto *kern = attend_wide<BITS>;
    static PerDevice ready;
    const cudaError_t e = ready.once([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    wide::Smem::bytes);
    });
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kern, dim3(ws.most), dim3(wide::Shape<BITS>::threads), (size_t)wide::Smem::bytes, st, p,
                      static_cast<const uint4 *>(p.r_img), ws);
}

}  // namespace attend
}  // namespace oq
