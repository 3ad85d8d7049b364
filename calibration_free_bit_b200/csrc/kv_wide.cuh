// kv_wide.cuh -- the cache's attention for many rows a key head (trees of drafted tokens), heads of
// 128: tcgen05 with tiles of 128 rows by 128 tokens.  Method and checks: kv_attend.cuh; work list:
// kv_attend_ops.cuh; the pieces of a segment are joined by a second kernel (kv_attend.cu).
//
// One CTA per SM walks a contiguous range of units.  For a piece it rotates the 128 queries (one
// tcgen05.mma with the rotation's dense operand) and keeps them as the A operand in shared memory;
// then, per unit, decoder warps turn the codes of 128 tokens into the fp16 operands K (elements
// contiguous, K-major) and V (the same layout, read as N-major), one row a thread; S = Q K^T goes to
// tensor memory; a softmax thread owns a row, takes S from there and puts the weights back as the A
// operand of O += P V.  Two softmax groups take the units in turn, each with its own S, O and row
// statistics, so that one's exponentials run beside the other's products; they meet at the end.
// What bounds a unit: shared memory (16384 table lookups and 64 KB of operands stored), the
// exponentials (16384), and the issue slots of both, about a thousand cycles each.
//   - Key norms enter the operand (times 2^-e, e by 32 tokens, so that fp16 holds any norm): scores
//     of a group of 32 tokens then share one factor, and the search for a new maximum is a maximum
//     over raw products.  Value norms enter with the weights, a row at a time, so that what a row
//     does not see (a NaN, an infinity) never reaches it.
#pragma once

#include <type_traits>

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
// Warps: two softmax groups, eight decoders each for keys and values, and a group of four of which
// two issue products (the others leave).
constexpr int kSoftWarps = 8, kDecWarps = 16;
constexpr int kThreads = 32 * (kSoftWarps + kDecWarps + 4);
constexpr int kWorking = 32 * (kSoftWarps + kDecWarps + 2);       // that meet at barrier 0
constexpr int kTile = 128 * D * 2;                    // an operand: 32 KB

// Shared memory by address (a CTA's own starts at 1024): the table at a multiple of its size, the
// operands behind it at multiples of 1024.
struct Smem {
    static constexpr int vn_at = kSharedStart;        // [2][128] value norms
    static constexpr int kexp_at = vn_at + 1024;      // [2][4] powers of two of the key norms
    static constexpr int vmax_at = kexp_at + 32;      // [2][4] largest value norms
    static constexpr int bad_at = vmax_at + 32;       // [2][4] tokens of missing pages
    static constexpr int qs_at = bad_at + 32;         // [128] score factor of a row
    static constexpr int mask_at = qs_at + 512;       // [128]
    static constexpr int stat_at = mask_at + 1024;    // [2][3][128]: m, l, s_v scale
    static constexpr int work_at = stat_at + 3072;
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

template <bool BF16> __device__ __forceinline__ uint32_t idesc_q() {
    return idesc_f16(128, 128) | (BF16 ? (1u << 7) | (1u << 10) : 0u);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

}  // namespace wide

template <class E, int BITS>
__global__ void __launch_bounds__(wide::kThreads, 1)
attend_wide(const KvAttendParams p, const uint4 *r_img, const KvAttendSpace ws) {
    using namespace wide;
    using S = wide::Smem;
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
    float *kexp_s = reinterpret_cast<float *>(at_address(raw, S::kexp_at));
    float *vmax_s = reinterpret_cast<float *>(at_address(raw, S::vmax_at));
    uint32_t *bad_s = reinterpret_cast<uint32_t *>(at_address(raw, S::bad_at));
    float *qs_s = reinterpret_cast<float *>(at_address(raw, S::qs_at));
    unsigned long long *mask_s = reinterpret_cast<unsigned long long *>(at_address(raw, S::mask_at));
    float *stat_s = reinterpret_cast<float *>(at_address(raw, S::stat_at));

    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    fill_lut<BITS, PLACED>(at_address(raw, S::lut_at), p.lut);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_K + i), kDecWarps / 2);
            mbar_init(bar(B_V + i), kDecWarps / 2);
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_P + i), 4);
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
        asm volatile("bar.sync 0, %0;" ::"n"(kWorking) : "memory");
        tc_fence_after();
    };
    Walk walk = *work;
    Piece q;
    uint32_t used[2] = {0, 0};                       // units so far of either group

    if (warp < kSoftWarps) {
        // ---------------- softmax: group `me` has units me, me + 2, ... ----------------
        uint32_t pieces = 0;
        while (next_piece<WideForm>(p, walk, q)) {
            const Seq &s = q.s;
            const int n = q.n, tile0 = q.tile0, nrows = q.nrows;
            // the rotation to K's first stage (the raw queries go to V's)
            for (int i = threadIdx.x; i < kTile / 16; i += 32 * kSoftWarps)
                reinterpret_cast<uint4 *>(at_address(raw, S::k_at))[i] = __ldg(r_img + i);
            if (threadIdx.x < kRows) {
                const int node = (q.row_base + threadIdx.x) / p.group;
                mask_s[threadIdx.x] =
                    threadIdx.x >= nrows ? 0ull
                    : p.mask ? (unsigned long long)p.mask[s.row0 + node] &
                                   (s.nodes >= 64 ? ~0ull : (1ull << s.nodes) - 1ull)
                             : (2ull << node) - 1ull;
            }
            fence_async_smem();
            meet();
            if (warp < 4) {
                // rotated queries, fp16 over a power of two a row
                wait(B_Q, pieces);
                tc_fence_after();
                const uint32_t mine = tmem + ((uint32_t)(32 * warp) << 16);
                float big = 0.f;
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    uint32_t z[32];
                    tmem_ld32(mine + 32 * k, z);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        big = fmaxf(big, fabsf(__uint_as_float(z[i])));
                }
                // 2^e <= big < 2^(e+1); values over 2^e stay below 2 (2^e and its inverse are normal)
                uint32_t ex = (__float_as_uint(big) >> 23) & 255u;
                ex = ex < 1u ? 1u : (ex > 253u ? 253u : ex);
                const float up = __uint_as_float(ex << 23), down = __uint_as_float((254u - ex) << 23);
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    uint32_t z[32];
                    tmem_ld32(mine + 32 * k, z);
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        auto f = [&](int j) { return __uint_as_float(z[i + j]) * down; };
                        *reinterpret_cast<uint4 *>(at_address(raw, S::q_at) +
                                                   operand_at(threadIdx.x, 4 * k + i / 8)) =
                            make_uint4(half2_bits(f(0), f(1)), half2_bits(f(2), f(3)),
                                       half2_bits(f(4), f(5)), half2_bits(f(6), f(7)));
                    }
                }
                qs_s[threadIdx.x] = up * p.qk_scale;
                fence_async_smem();
            }
            meet();
            const int me = warp >> 2, r = threadIdx.x & 127;
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t tS = tmem + lanes + 128 * me, tO = tmem + lanes + 256 + 128 * me;
            const float qs = qs_s[r];
            const unsigned long long mask = mask_s[r];
            float m = kNone, l = 0.f, vs = 0.f, vinv = 0.f;
            for (int i = me; i < n; i += 2) {
                const uint32_t c = used[me] + (i >> 1);
                const int tok = (tile0 + i) * kTokens;
                wait(B_K + me, c);                    // exponents and lost tokens
                wait(B_S + me, c);
                tc_fence_after();
                const float *ke = kexp_s + 4 * me, *vn = vn_s + 128 * me;
                wait(B_V + me, c);                    // value norms
                const float4 vm = *reinterpret_cast<const float4 *>(vmax_s + 4 * me);
                const uint4 bad = *reinterpret_cast<const uint4 *>(bad_s + 4 * me);
                const bool edge = tok + kTokens > s.prefix || (bad.x | bad.y | bad.z | bad.w);
                // tokens of group k that this row sees
                auto seen = [&](int k) -> uint32_t {
                    const int first = tok + 32 * k - s.prefix;        // node of its first token
                    uint32_t v;
                    if (first <= -32)
                        v = ~0u;
                    else if (first < 0)
                        v = (uint32_t)(mask << -first) | ((1u << -first) - 1u);
                    else
                        v = first < 64 ? (uint32_t)(mask >> first) : 0u;
                    return v & ~bad_s[4 * me + k];
                };
                // the row's largest score and the largest value norm that it sees
                float top = -CUDART_INF_F, vtop;
                if (!edge) {
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        uint32_t z[32];
                        tmem_ld32(tS + 32 * k, z);
                        float a[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            a[h] = fmaxf(__uint_as_float(z[h]), __uint_as_float(z[2 + h]));
#pragma unroll
                            for (int j = 4 + h; j < 32; j += 4)
                                a[h] = max3(a[h], __uint_as_float(z[j]), __uint_as_float(z[j + 2]));
                        }
                        top = fmaxf(top, fmaxf(a[0], a[1]) * (qs * ke[k]));
                    }
                    vtop = fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w));
                } else {
                    vtop = 0.f;
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t v = seen(k);
                        const float f = qs * ke[k];
                        uint32_t z[32];
                        tmem_ld32(tS + 32 * k, z);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if ((v >> j) & 1u) {
                                top = fmaxf(top, __uint_as_float(z[j]) * f);
                                vtop = fmaxf(vtop, vn[32 * k + j]);
                            }
                    }
                }
                if (__any_sync(0xffffffffu, top > m + kSlack || vtop > vs)) {
                    const float up = fmaxf(m, top);
                    float fac = ex2(m - up);
                    m = up;
                    l *= fac;
                    if (vtop > vs) {
                        const float nv = norm_scale(vtop);
                        fac *= vs / nv;
                        vs = nv;
                        vinv = kWeightScale / nv;
                    }
                    if (i >= 2) {                     // the sums so far, once they are complete
                        wait(B_PV + me, c - 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            uint32_t z[32];
                            tmem_ld32(tO + 32 * k, z);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                z[j] = __float_as_uint(__uint_as_float(z[j]) * fac);
                            tmem_st32(tO + 32 * k, z);
                        }
                    }
                }
                if (!edge) {
                    float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    const float2 mm = make_float2(-m, -m), vi = make_float2(vinv, vinv);
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        uint32_t z[32], w[16];
                        tmem_ld32(tS + 32 * k, z);
                        const float f = qs * ke[k];
                        const float2 ff = make_float2(f, f);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 nv = *reinterpret_cast<const float4 *>(vn + 32 * k + j);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float2 x = __ffma2_rn(
                                    make_float2(__uint_as_float(z[j + 2 * h]),
                                                __uint_as_float(z[j + 2 * h + 1])), ff, mm);
                                const float2 e = make_float2(ex2(x.x), ex2(x.y));
                                ls[h] = __fadd2_rn(ls[h], e);
                                const float2 n2 = h ? make_float2(nv.z, nv.w)
                                                    : make_float2(nv.x, nv.y);
                                const float2 pw = __fmul2_rn(e, __fmul2_rn(n2, vi));
                                w[j / 2 + h] = half2_bits(pw.x, pw.y);
                            }
                        }
                        tmem_st16(tS + 16 * k, w);
                    }
                    l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                } else {
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        uint32_t z[32], w[16];
                        tmem_ld32(tS + 32 * k, z);
                        const uint32_t v = seen(k);
                        const float f = qs * ke[k];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float pw[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                pw[h] = 0.f;
                                if ((v >> (j + h)) & 1u) {
                                    const float e = ex2(fmaf(__uint_as_float(z[j + h]), f, -m));
                                    l += e;
                                    pw[h] = e * (vn[32 * k + j + h] * vinv);
                                }
                            }
                            w[j / 2] = half2_bits(pw[0], pw[1]);
                        }
                        tmem_st16(tS + 16 * k, w);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(B_P + me));
            }
            // ---- the groups meet, and the piece goes to its slot ----
            const int mine = (n + 1 - me) / 2;       // units of this group
            if (mine > 0) {
                wait(B_PV + me, used[me] + mine - 1);
                tc_fence_after();
            }
            stat_s[me * 384 + r] = m;
            stat_s[me * 384 + 128 + r] = l;
            stat_s[me * 384 + 256 + r] = vs * (1.0f / kWeightScale);
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const float om = stat_s[(me ^ 1) * 384 + r], ol = stat_s[(me ^ 1) * 384 + 128 + r];
            const float mx = fmaxf(m, om);
            const float fac = ex2(m - mx) * vs * (1.0f / kWeightScale);
            float *buf = reinterpret_cast<float *>(at_address(raw, S::k_at));        // [element][row]
            if (me == 1 && mine > 0) {
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    uint32_t z[32];
                    tmem_ld32(tO + 32 * k, z);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        buf[(32 * k + j) * 128 + r] = __uint_as_float(z[j]) * fac;
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (me == 0) {
                const long long slot = (long long)q.b * ws.segments + q.seg + blockIdx.x;
                if (r < nrows) {
                    ws.stat[(slot * 2) * ws.rows + r] = mx;
                    ws.stat[(slot * 2 + 1) * ws.rows + r] = l * ex2(m - mx) + ol * ex2(om - mx);
                }
                float *dst = ws.part + (slot * ws.rows + r) * D;
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    uint32_t z[32];
                    tmem_ld32(tO + 32 * k, z);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float o = __uint_as_float(z[j]) * fac;
                        if (n > 1)
                            o += buf[(32 * k + j) * 128 + r];
                        z[j] = __float_as_uint(o);
                    }
                    if (r < nrows)
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                         ::"l"(dst + 32 * k + j), "r"(z[j]), "r"(z[j + 1]),
                                         "r"(z[j + 2]), "r"(z[j + 3]), "r"(z[j + 4]),
                                         "r"(z[j + 5]), "r"(z[j + 6]), "r"(z[j + 7]) : "memory");
                }
            }
            meet();
            used[0] += (n + 1) / 2;
            used[1] += n / 2;
            ++pieces;
        }
    } else if (warp < kSoftWarps + kDecWarps) {
        // ---------------- decoders: half a token's key row or value row a thread ----------------
        const int dt = threadIdx.x - 32 * kSoftWarps;
        while (next_piece<WideForm>(p, walk, q)) {
            const int n = q.n, tile0 = q.tile0, total = q.total, kvh = q.kvh, b = q.b;
            const int ch = dt & 15;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = i * 32 + (dt >> 4);
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < q.nrows) {
                    const int node = (q.row_base + r) / p.group, e = q.row_base + r - node * p.group;
                    v = *reinterpret_cast<const uint4 *>(
                        static_cast<const E *>(p.q) + (q.s.row0 + node) * p.q_stride +
                        (kvh * p.group + e) * D + ch * 8);
                }
                *reinterpret_cast<uint4 *>(at_address(raw, S::v_at) + operand_at(r, ch)) = v;
            }
            fence_async_smem();
            meet();
            meet();
            const int w = dt >> 8, part = (dt >> 7) & 1, row = dt & 127;
            const int *table = p.table + (long long)b * p.table_width;
            const uint32_t col = lut_column<BITS, PLACED>(S::lut_at, lane);
            constexpr int words = 2 * BITS;               // 64 codes
            // One unit ahead in registers and two ahead on the way to the L2; a page's index is
            // known three ahead, so that no load waits for another.
            struct Row {
                uint32_t codes[words];
                float norm;
                bool missing, valid;
            };
            auto page_of = [&](int i) -> int {
                const int tok = (tile0 + i) * kTokens + row;
                return i < n && tok < total ? __ldg(table + (tok >> p.c.page_log2)) : -1;
            };
            auto row_of = [&](int i, int page) -> long long {
                return (((long long)page * p.c.kv_heads + kvh) << p.c.page_log2) +
                       (((tile0 + i) * kTokens + row) & ((1 << p.c.page_log2) - 1));
            };
            auto fetch = [&](int i, int page) {
                if (page >= 0 && page < p.c.pages) {
                    const uint8_t *at = pick(p.c.codes, w) + row_of(i, page) * (D * BITS / 8) + part * (8 * BITS);
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
                    load_words<words, 8 * BITS>(
                        to.codes, pick(p.c.codes, w) + at * (D * BITS / 8) + part * (8 * BITS));
                    to.norm = __ldg(pick(p.c.norms, w) + at);
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
            for (int i = 0; i < n; ++i) {
                const int st = i & 1;
                const uint32_t c = used[st] + (i >> 1);
                load(nxt, i + 1, page1);
                fetch(i + 2, page2);
                const int page3 = page_of(i + 3);
                const float norm = cur.norm;
                const bool valid = cur.valid, missing = cur.missing;
                // the largest norm of the warp's 32 tokens (they are one group of scores)
                float top = valid && norm < CUDART_INF_F ? norm : 0.f;
#pragma unroll
                for (int k = 16; k; k >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
                const uint32_t lost = __ballot_sync(0xffffffffu, missing);
                uint32_t ex = (__float_as_uint(top) >> 23) & 255u;
                ex = ex < 28u ? 28u : (ex > 253u ? 253u : ex);
                const __half2 by = __float2half2_rn(norm * __uint_as_float((254u - ex) << 23));
                // K's stage is free after S, V's and the norms' after P V
                if (c > 0)
                    wait((w == 0 ? B_S : B_PV) + st, c - 1);
                unsigned char *to = at_address(raw, (w == 0 ? S::k_at : S::v_at) + st * kTile);
                // four chunks of 8 elements at a time, so that their lookups are under way together
                // (the compiler does not move a load over a store to the operand)
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    uint4 v[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        quad<BITS, PLACED>(cur.codes, 2 * (k + h), col, v[h].x, v[h].y);
                        quad<BITS, PLACED>(cur.codes, 2 * (k + h) + 1, col, v[h].z, v[h].w);
                    }
                    if (w == 0) {
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            __half2 *x = reinterpret_cast<__half2 *>(&v[h]);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                x[j] = __hmul2(x[j], by);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        *reinterpret_cast<uint4 *>(to + operand_at(row, 8 * part + k + h)) = v[h];
                }
                cur = nxt;
                page1 = page2;
                page2 = page3;
                if (w == 0) {
                    if (c > 0)
                        wait(B_PV + st, c - 1);
                    if (part == 0 && lane == 0) {
                        kexp_s[4 * st + (warp & 3)] = __uint_as_float(ex << 23);
                        bad_s[4 * st + (warp & 3)] = lost;
                        if (lost)
                            atomicOr(p.err, AT_ERR_PAGE);
                    }
                } else if (part == 0) {
                    vn_s[128 * st + row] = norm;
                    if (lane == 0)
                        vmax_s[4 * st + (warp & 3)] = top;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar((w == 0 ? B_K : B_V) + st));
            }
            meet();
            used[0] += (n + 1) / 2;
            used[1] += n / 2;
        }
    } else {
        const int which = warp - kSoftWarps - kDecWarps;
        if (which >= 2)
            return;
        while (next_piece<WideForm>(p, walk, q)) {
            const int n = q.n;
            meet();
            if (which == 0 && lane == 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_ss(tmem, sw128_desc(base + S::v_at + (k >> 2) * 16384) + 2 * (k & 3),
                           sw128_desc(base + S::k_at + (k >> 2) * 16384) + 2 * (k & 3),
                           idesc_q<std::is_same<E, __nv_bfloat16>::value>(), k != 0);
                mma_commit(bar(B_Q));
            }
            meet();
            if (which == 0 && lane == 0) {
                // ---------------- S = Q K^T ----------------
                for (int i = 0; i < n; ++i) {
                    const int st = i & 1;
                    const uint32_t c = used[st] + (i >> 1);
                    wait(B_K + st, c);
                    if (c > 0)
                        wait(B_PV + st, c - 1);           // the weights lie where S goes
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ss(tmem + 128 * st,
                               sw128_desc(base + S::q_at + (k >> 2) * 16384) + 2 * (k & 3),
                               sw128_desc(base + S::k_at + st * kTile + (k >> 2) * 16384) + 2 * (k & 3),
                               idesc_f16(128, 128), k != 0);
                    mma_commit(bar(B_S + st));
                }
            } else if (lane == 0) {
                // ---------------- O += P V ----------------
                for (int i = 0; i < n; ++i) {
                    const int st = i & 1;
                    const uint32_t c = used[st] + (i >> 1);
                    wait(B_V + st, c);
                    wait(B_P + st, c);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(tmem + 256 + 128 * st, tmem + 128 * st + 8 * k,
                               v_desc(base + S::v_at + st * kTile + k * 2048),
                               idesc_f16(128, 128) | (1u << 16), i >= 2 || k != 0);
                    mma_commit(bar(B_PV + st));
                }
            }
            meet();
            used[0] += (n + 1) / 2;
            used[1] += n / 2;
        }
    }
    // Every product has been waited for by the group that uses it, so the tensor memory is free.
    meet();
    if (warp == kSoftWarps + kDecWarps)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

template <class E, int BITS>
cudaError_t launch_wide(const KvAttendParams &p, const KvAttendSpace &ws, cudaStream_t st) {
    auto *kern = attend_wide<E, BITS>;
    static PerDevice ready;
    const cudaError_t e = ready.once([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    wide::Smem::bytes);
    });
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kern, dim3(ws.most), dim3(wide::kThreads), (size_t)wide::Smem::bytes, st, p,
                      static_cast<const uint4 *>(p.r_img), ws);
}

}  // namespace attend
}  // namespace oq
