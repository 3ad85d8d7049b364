// kv_tc.cu -- the cache's write and read with the rotation on the tensor cores (16-bit rows).
//
// A head's row has 128 or 256 elements, so the whole rotation R (permutation, signs, Hadamard
// blocks) is a small dense matrix of +-1 and 0 over sqrt(h): exact in fp16 and bf16, and 2 d FLOP
// an element that the tensor cores have to spare.  What is left is a pass over memory.
//   write  D[row, i] = sum_j x[row, j] R'[i, j]: tcgen05.mma of a tile of 128 rows (M) with R' as
//          the B operand, exact products, fp32 sums in tensor memory.  A thread then owns a row (at
//          d = 256 half of one): norm, codes and packing need no exchange between lanes.
//   read   D[row, j] = sum_i c[code[row, i]] R'[i, j]: a thread decodes its row through the
//          conflict-free table into the A operand, takes the finished row back, scales it and
//          sends it off with one bulk copy.
// One CTA per SM keeps R' (32 KB at d = 128) in shared memory for four groups of 128 threads that
// work on tiles of their own; at d = 256 R' takes 128 KB and leaves room for one group of 256.
// B200, bf16: 32760 tokens of 40 heads of 128 at 8 bits, write 317 us (3.2 TB/s), read 291 us (3.5 TB/s),
// both bound by shared memory (the quantizer's table has one copy at 8 bits, so its lookups conflict;
// lookups, operand and finished rows of a read); 2011 tokens of 8 heads at 4 bits, 9.3 and 7.0 us, of
// which 5 are the set-up; fp16, 5003 tokens of 4 heads of 256 at 2 bits, 20.3 and 14.0 us (values beside
// a boundary take 0.6 and 1.3 of the writes).
#include "k1_ops.cuh"
#include "kv_internal.h"
#include "kv_lut.cuh"
#include "kv_ops.cuh"
#include "kv_rows.cuh"
#include "sm100_common.cuh"

namespace oq {
namespace {

using namespace kvops;
using namespace sm100;
using k1ops::fma_sat;

template <int D> struct Geo {
    static constexpr int groups = D == 128 ? 4 : 1;
    static constexpr int group_threads = D;
    static constexpr int threads = groups * group_threads;
    static constexpr int r_bytes = D * D * 2;
    static constexpr int a_bytes = 128 * D * 2;
    static constexpr int stage_stride = 2 * D + 16;           // a finished row, bank spread
    static constexpr int stage_bytes = 128 * stage_stride;
};

// kind::f16, fp32 accumulator, M = 128, N = D; both operands bf16 or both fp16, K-major.
template <int D, bool BF16> __host__ __device__ constexpr uint32_t idesc() {
    return (1u << 4) | (BF16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(D >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void group_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// Byte offset of 16-byte chunk ch (8 elements) of row r in a K-major, 128-byte-swizzled operand
// of `rows` rows.
__device__ __forceinline__ uint32_t operand_at(int r, int ch, int rows) {
    return (uint32_t)(ch >> 3) * (rows * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

template <int D, bool BF16>
__device__ __forceinline__ void issue_mma(uint32_t tmem, uint32_t sA, uint32_t sR, uint32_t bar,
                                          bool add = false) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
        mma_ss(tmem, sw128_desc(sA + (k >> 2) * (128 * 128)) + 2 * (k & 3),
               sw128_desc(sR + (k >> 2) * (D * 128)) + 2 * (k & 3), idesc<D, BF16>(), add || k != 0);
    mma_commit(bar);
}

// R' into shared memory, tensor memory and barriers: the part of a kernel before its rows.
template <int D>
__device__ __forceinline__ uint32_t set_up(unsigned char *r_sm, const uint4 *r_img, uint32_t bars,
                                           uint32_t *slot) {
    for (int i = threadIdx.x; i < Geo<D>::r_bytes / 16; i += Geo<D>::threads)
        reinterpret_cast<uint4 *>(r_sm)[i] = __ldg(r_img + i);
    if (threadIdx.x < Geo<D>::groups)
        mbar_init(bars + 8 * threadIdx.x, 1);
    if (threadIdx.x < 32) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(slot)), "r"(Geo<D>::groups * D) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return *slot;
}

template <int D> __device__ __forceinline__ void tear_down(uint32_t tmem) {
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x < 32)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                     ::"r"(tmem), "r"(Geo<D>::groups * D));
}

// ---- write ----
template <int D, int BITS> struct WriteSmem {
    static constexpr int tbl_at = Geo<D>::r_bytes + Geo<D>::groups * Geo<D>::a_bytes;
    static constexpr int bytes(int tbl_words) { return 1024 + tbl_at + tbl_words * 4 + 1024 + 64; }
};

// 32 codes (the top bytes of c) -> BITS words, LSB first.
template <int BITS>
__device__ __forceinline__ void pack32(const uint32_t (&c)[32], uint32_t *w) {
    if constexpr (BITS == 2 || BITS == 4 || BITS == 8) {
        constexpr int per = 32 / BITS;
#pragma unroll
        for (int i = 0; i < BITS; ++i) {
            uint32_t part[per];
#pragma unroll
            for (int k = 0; k < per; ++k)
                part[k] = c[i * per + k];
            w[i] = k1ops::pack_codes<BITS>(part);
        }
    } else {
#pragma unroll
        for (int i = 0; i < BITS; ++i)
            w[i] = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const int bit = k * BITS, i = bit >> 5, s = bit & 31;
            const uint32_t v = c[k] >> 24;
            w[i] |= v << s;
            if (s + BITS > 32)
                w[i + 1] |= v >> (32 - s);
        }
    }
}

// One column of this thread's lane of tensor memory (warp-collective).
__device__ __forceinline__ void tmem_ld1(uint32_t at, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r) : "r"(at) : "memory");
}

// Few codes are far apart, so a wrong one beside a boundary shows in fp16 rows; with 8 bits it is off by
// less than their rounding, and is left (300 of a million are beside one, and a second look at each would
// take a tenth of the time; a few of them fall the other way in a smaller call, kv_cache.cu).
template <int BITS> constexpr bool kLook = BITS <= 6;

template <int D, int BITS, bool BF16>
__global__ void __launch_bounds__(Geo<D>::threads, 1)
kv_write_tc(const KvWriteParams p, const uint4 *r_img, const int tbl_words, const int tiles) {
    using G = Geo<D>;
    using X = std::conditional_t<BF16, __nv_bfloat16, __half>;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    unsigned char *sm = raw + (base - smem_u32(raw));
    using W = WriteSmem<D, BITS>;
    float *half_sum = reinterpret_cast<float *>(sm + W::tbl_at + tbl_words * 4);     // D = 256
    uint32_t *slot_sm = reinterpret_cast<uint32_t *>(half_sum + 256);
    const uint32_t bars = smem_u32(slot_sm) + 16;

    pdl_trigger();
    for (int i = threadIdx.x; i < tbl_words / 4; i += G::threads)
        reinterpret_cast<uint4 *>(sm + W::tbl_at)[i] =
            __ldg(reinterpret_cast<const uint4 *>(p.tbl) + i);
    const uint32_t tmem0 = set_up<D>(sm, r_img, bars, slot_sm);
    pdl_wait();

    const int grp = threadIdx.x / G::group_threads, tid = threadIdx.x % G::group_threads;
    const int lane = threadIdx.x & 31, row = tid & 127, part = tid >> 7;
    const uint32_t sR = base, sA = base + G::r_bytes + grp * G::a_bytes, bar = bars + 8 * grp;
    const unsigned char *a_sm = sm + G::r_bytes + grp * G::a_bytes;
    const uint32_t tmem = tmem0 + grp * D;
    const uint32_t my_tmem = tmem + ((uint32_t)(row & ~31) << 16) + part * 128;
    const int heads = p.c.kv_heads, half_tiles = tiles / 2;
    const long long rows = (long long)p.T * heads;
    // this lane's column of the quantizer table, from q = 0 (q starts at the bits of 1.0)
    constexpr uint32_t pitch = BITS <= 4 ? 128 : 4;
    const uint32_t my_tbl =
        base + W::tbl_at + (BITS <= 4 ? lane * 4 : 0) - (0x3F800000u >> p.F) * pitch;

    auto load = [&](int tile) {
        const int w = tile >= half_tiles;
        const long long r0 = (long long)(tile - w * half_tiles) * 128;
        const char *x = static_cast<const char *>(pick(p.x, w));
        constexpr int chunks = D / 8, step = G::group_threads / chunks;
        const int ch = tid % chunks;
        const bool flat = pick(p.x_stride, w) == (long long)heads * D;
#pragma unroll
        for (int i = 0; i < 128 / step; ++i) {
            const int r = i * step + tid / chunks;
            const long long at = r0 + r;
            const bool real = at < rows;
            long long from = 0;
            if (real) {
                if (flat) {
                    from = at * D;
                } else {
                    const long long tok = at / heads;
                    from = tok * pick(p.x_stride, w) + (at - tok * heads) * D;
                }
            }
            cp16(sA + operand_at(r, ch, 128), x + (from + ch * 8) * 2, real);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    bool dead = false;
    uint32_t phase = 0;
    const int stride = gridDim.x * G::groups;
    int tile = blockIdx.x + grp * gridDim.x;
    if (tile < tiles)
        load(tile);
    for (; tile < tiles; tile += stride) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        fence_async_smem();
        tc_fence_before();
        group_sync(1 + grp, G::group_threads);
        if (tid == 0) {
            tc_fence_after();
            issue_mma<D, BF16>(tmem, sA, sR, bar);
        }
        // this thread's row, while the product runs
        const int w = tile >= half_tiles;
        const long long at = (long long)(tile - w * half_tiles) * 128 + row;
        long long dst = -1;
        if (at < rows) {
            const long long tok = at / heads;
            const long long slot = p.slots[tok];
            if (slot_ok(p.c, slot))
                dst = cache_row(p.c, slot, (int)(at - tok * heads));
            else if (slot != -1)
                atomicOr(p.err, KV_ERR_SLOT);
        }
        if (!dead && !mbar_wait(bar, phase)) {
            dead = true;
            atomicOr(p.err, KV_ERR_WAIT);
        }
        phase ^= 1;
        tc_fence_after();
        if (tile + stride < tiles)
            load(tile + stride);                       // the operand is free again
        float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t z[32];
            tmem_ld32(my_tmem + 32 * k, z);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                sums[i & 3] = fmaf(__uint_as_float(z[i]), __uint_as_float(z[i]), sums[i & 3]);
        }
        float sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
        if constexpr (D == 256) {
            half_sum[tid] = sum;
            group_sync(1 + grp, G::group_threads);
            sum = half_sum[row] + half_sum[row + 128];
        }
        const float norm = sqrtf(sum / (float)p.h);
        const float kk = p.K / (norm + p.eps);
        uint32_t out[4 * BITS], beside[4], any = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t z[32];
            tmem_ld32(my_tmem + 32 * k, z);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const uint2 q = k1ops::f2_add_one_rm_bits(fma_sat(__uint_as_float(z[i]), kk, 0.5f),
                                                          fma_sat(__uint_as_float(z[i + 1]), kk, 0.5f));
                z[i] = k1ops::lds32(my_tbl + (q.x >> p.F) * pitch) + q.x * (uint32_t)p.G;
                z[i + 1] = k1ops::lds32(my_tbl + (q.y >> p.F) * pitch) + q.y * (uint32_t)p.G;
            }
            if constexpr (kLook<BITS>) {
                uint32_t least = ~0u;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    least = min(least, distance_to_bound(z[i], p.G));
                beside[k] = 0;
                const bool look = dst >= 0 && looks(norm) && least < bound_width(p.G);
                if (__any_sync(0xffffffffu, look)) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (look && distance_to_bound(z[i], p.G) < bound_width(p.G))
                            beside[k] |= 1u << i;
                    any |= __reduce_or_sync(0xffffffffu, beside[k]) ? 1u << k : 0u;
                }
            }
            pack32<BITS>(z, out + k * BITS);
        }
        if constexpr (kLook<BITS>) {
            // values beside a boundary, by all lanes one at a time (a tile has few of them, and this code
            // for all columns at once would cost it more than they do)
            int left = kLooks;                         // of this lane's row
#pragma unroll 1
            for (; any; any &= any - 1) {
                const int k = __ffs(any) - 1;
                const uint32_t mine = k < 2 ? (k ? beside[1] : beside[0]) : (k > 2 ? beside[3] : beside[2]);
#pragma unroll 1
                for (uint32_t cols = __reduce_or_sync(0xffffffffu, mine); cols; cols &= cols - 1) {
                    const int b = __ffs(cols) - 1, bit = (32 * k + b) * BITS, s = bit & 31;
                    uint32_t z;
                    tmem_ld1(my_tmem + 32 * k + b, z);
                    const uint32_t q = __float_as_uint(
                        __fadd_rd(fma_sat(__uint_as_float(z), kk, 0.5f), 1.0f));
                    const uint32_t was =
                        (k1ops::lds32(my_tbl + (q >> p.F) * pitch) + q * (uint32_t)p.G) >> 24;
                    const bool zero = __uint_as_float(z) == 0.f;
                    uint32_t x = ((mine >> b) & 1u) && zero ? was ^ code_of_zero(BITS) : 0u;
#pragma unroll 1
                    for (uint32_t lanes = __ballot_sync(0xffffffffu, ((mine >> b) & 1u) && !zero && left > 0);
                         lanes; lanes &= lanes - 1) {
                        // a lane's D / 32 elements of the row (which is still the operand, if this was
                        // the group's last tile) and of the rotation's
                        const int l = __ffs(lanes) - 1, r = (row & ~31) + l;
                        constexpr int N = D / 32;
                        const int ch = lane * N / 8, in = lane * N % 8 * 2;
                        const X *from;
                        if (tile + stride < tiles) {
                            const long long at = (long long)(tile - w * half_tiles) * 128 + r;
                            const long long tok = at / heads;
                            from = static_cast<const X *>(pick(p.x, w)) + tok * pick(p.x_stride, w) +
                                   (at - tok * heads) * D + lane * N;
                        } else {
                            from = reinterpret_cast<const X *>(a_sm + operand_at(r, ch, 128) + in);
                        }
                        const X *turn = reinterpret_cast<const X *>(
                            sm + operand_at(part * 128 + 32 * k + b, ch, D) + in);
                        double sum = 0.0, squares = 0.0;
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const double v = to_f32(from[i]);
                            sum += v * (double)to_f32(turn[i]);
                            squares += v * v;
                        }
                        const uint32_t code =
                            code_beside(__shfl_sync(0xffffffffu, was, l), sum, squares,
                                        __shfl_sync(0xffffffffu, norm, l), p.unit, p.bounds, BITS);
                        if (lane == l) {
                            x = was ^ code;
                            --left;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4 * BITS; ++i) {
                        out[i] ^= i == bit >> 5 ? x << s : 0u;
                        if (32 % BITS)
                            out[i] ^= i == (bit >> 5) + 1 && s + BITS > 32 ? x >> (32 - s) : 0u;
                    }
                }
            }
        }
        if (dst >= 0) {
            uint8_t *to = pick(p.c.codes, w) + dst * (D * BITS / 8) + part * (16 * BITS);
            if (BITS % 2 == 0 && p.wide) {
#pragma unroll
                for (int k = 0; k + 7 < 4 * BITS; k += 8)
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                 ::"l"(to + 4 * k), "r"(out[k]), "r"(out[k + 1]), "r"(out[k + 2]),
                                 "r"(out[k + 3]), "r"(out[k + 4]), "r"(out[k + 5]), "r"(out[k + 6]),
                                 "r"(out[k + 7]) : "memory");
            } else {
#pragma unroll
                for (int k = 0; k < 4 * BITS; k += 4)
                    *reinterpret_cast<uint4 *>(to + 4 * k) =
                        make_uint4(out[k], out[k + 1], out[k + 2], out[k + 3]);
            }
            if (part == 0)
                pick(p.c.norms, w)[dst] = norm;
        }
    }
    tear_down<D>(tmem0);
}

// ---- read ----
template <int D, int BITS> struct ReadSmem {
    static constexpr int lut_at = Geo<D>::r_bytes;
    static constexpr int a_at = lut_at + Lut<BITS, ANYWHERE>::bytes;              // 1024-byte aligned
    static constexpr int a_size = (Geo<D>::stage_bytes + 1023) / 1024 * 1024;
    static constexpr int end = a_at + Geo<D>::groups * a_size;
    // barriers and the tensor memory's address; at d = 256 in the last row's padding
    static constexpr int bars_at = D == 256 ? end - 16 : end;
    static constexpr int bytes = 1024 + (D == 256 ? end : end + 64);
};

template <class E> __device__ __forceinline__ uint32_t pair_of(float a, float b) {
    if constexpr (sizeof(E) == 2) {
        union { E e[2]; uint32_t u; } v;
        v.e[0] = from_f32<E>(a);
        v.e[1] = from_f32<E>(b);
        return v.u;
    }
    return 0;
}

template <class E, int D, int BITS>
__global__ void __launch_bounds__(Geo<D>::threads, 1)
kv_read_tc(const KvReadParams p, const uint4 *r_img, const int tiles) {
    using G = Geo<D>;
    using R = ReadSmem<D, BITS>;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    unsigned char *sm = raw + (base - smem_u32(raw));
    uint32_t *slot_sm = reinterpret_cast<uint32_t *>(sm + R::bars_at + 8 * G::groups);
    const uint32_t bars = base + R::bars_at;

    pdl_trigger();
    unsigned char *lut = sm + R::lut_at;
    fill_lut<BITS, ANYWHERE>(lut, p.lut);
    const uint32_t tmem0 = set_up<D>(sm, r_img, bars, slot_sm);
    pdl_wait();

    const int grp = threadIdx.x / G::group_threads, tid = threadIdx.x % G::group_threads;
    const int lane = threadIdx.x & 31, row = tid & 127, part = tid >> 7;
    const uint32_t sR = base, sA = base + R::a_at + grp * R::a_size, bar = bars + 8 * grp;
    unsigned char *a_sm = sm + R::a_at + grp * R::a_size;
    const uint32_t tmem = tmem0 + grp * D;
    const uint32_t my_tmem = tmem + ((uint32_t)(row & ~31) << 16) + part * 128;
    const uint32_t col = lut_column<BITS, ANYWHERE>(base + R::lut_at, lane);
    const int heads = p.c.kv_heads, half_tiles = tiles / 2;
    const long long rows = (long long)p.T * heads;
    constexpr int words = 4 * BITS;                       // of this thread's 128 elements
    // fp16 rows of 6 and 8 bits: a second product adds what fp16 leaves of the centroids (8000 rows of
    // 256: errors of 2.3e-4 to 2.9e-4 of their length, a few other codes among them, and not of 2.9e-4
    // to 3.1e-4; the output's rounding is 2.1e-4)
    constexpr bool kRests = std::is_same<E, __half>::value && BITS >= 6;

    // the codes and norm of this thread's row (zeros and 0 where the slot names none)
    auto load = [&](int tile, uint32_t (&c)[words], float &norm, E *&to) {
        const int w = tile >= half_tiles;
        const long long at = (long long)(tile - w * half_tiles) * 128 + row;
        norm = 0.f;
        to = nullptr;
        long long src = -1;
        if (at < rows) {
            const long long tok = at / heads;
            const int head = (int)(at - tok * heads);
            to = static_cast<E *>(pick(p.y, w)) + tok * pick(p.y_stride, w) + head * D + part * 128;
            const long long slot = p.slots[tok];
            if (slot_ok(p.c, slot))
                src = cache_row(p.c, slot, head);
            else if (slot != -1)
                atomicOr(p.err, KV_ERR_SLOT);
        }
        if (src >= 0) {
            norm = pick(p.c.norms, w)[src];
            load_words<words, 16>(c, pick(p.c.codes, w) + src * (D * BITS / 8) + part * (16 * BITS));
        } else {
#pragma unroll
            for (int i = 0; i < words; ++i)
                c[i] = 0;
        }
    };

    bool dead = false;
    uint32_t phase = 0;
    const int stride = gridDim.x * G::groups;
    int tile = blockIdx.x + grp * gridDim.x;
    uint32_t codes[words];
    float norm = 0.f;
    E *to = nullptr;
    if (tile < tiles)
        load(tile, codes, norm, to);
    for (; tile < tiles; tile += stride) {
        bulk_wait_read<0>();                              // the last tile's rows have left
        group_sync(1 + grp, G::group_threads);
        auto done = [&] {
            if (!dead && !mbar_wait(bar, phase)) {
                dead = true;
                atomicOr(p.err, KV_ERR_WAIT);
            }
            phase ^= 1;
            tc_fence_after();
        };
#pragma unroll
        for (int pass = 0; pass < (kRests ? 2 : 1); ++pass) {
            if (pass)
                done();
            // four chunks of 8 elements at a time, so that their lookups are under way together (the
            // compiler does not move a load over a store to the operand)
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
                uint4 v[4], rest[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    quad<BITS, ANYWHERE>(codes, 2 * (k + h), col, v[h].x, v[h].y, rest[h].x, rest[h].y);
                    quad<BITS, ANYWHERE>(codes, 2 * (k + h) + 1, col, v[h].z, v[h].w, rest[h].z,
                                         rest[h].w);
                }
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    *reinterpret_cast<uint4 *>(a_sm + operand_at(row, part * 16 + k + h, 128)) =
                        pass ? rest[h] : v[h];
            }
            fence_async_smem();
            tc_fence_before();
            group_sync(1 + grp, G::group_threads);
            if (tid == 0) {
                tc_fence_after();
                issue_mma<D, false>(tmem, sA, sR, bar, pass > 0);
            }
        }
        const float s = norm * p.scale;
        E *mine = to;
        if (tile + stride < tiles)
            load(tile + stride, codes, norm, to);
        done();
        unsigned char *stage = a_sm + row * G::stage_stride + part * 256;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t z[32];
            tmem_ld32(my_tmem + 32 * k, z);
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                auto f = [&](int j) { return __uint_as_float(z[i + j]) * s; };
                const uint4 v = make_uint4(pair_of<E>(f(0), f(1)), pair_of<E>(f(2), f(3)),
                                           pair_of<E>(f(4), f(5)), pair_of<E>(f(6), f(7)));
                *reinterpret_cast<uint4 *>(stage + 64 * k + 2 * i) = v;
            }
        }
        fence_async_smem();
        if (mine != nullptr)
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], 256;"
                         ::"l"(mine), "r"(smem_u32(stage)) : "memory");
        bulk_commit();
    }
    bulk_wait_all();
    tear_down<D>(tmem0);
}

template <int D, int BITS, bool BF16>
cudaError_t write_tc(const KvWriteParams &p, const uint4 *r_img, int tbl_words, cudaStream_t st,
                     int num_sms) {
    auto *kern = kv_write_tc<D, BITS, BF16>;
    const int bytes = WriteSmem<D, BITS>::bytes(tbl_words);
    static PerDevice ready;
    cudaError_t e = ready.once([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    });
    if (e != cudaSuccess)
        return e;
    if (bytes > 227 * 1024)
        return cudaErrorInvalidValue;
    const int tiles = 2 * (int)(((long long)p.T * p.c.kv_heads + 127) / 128);
    return launch_pdl(kern, dim3(tiles < num_sms ? tiles : num_sms), dim3(Geo<D>::threads), (size_t)bytes,
                      st, p, r_img, tbl_words, tiles);
}

template <class E, int D, int BITS>
cudaError_t read_tc(const KvReadParams &p, const uint4 *r_img, cudaStream_t st, int num_sms) {
    auto *kern = kv_read_tc<E, D, BITS>;
    constexpr int bytes = ReadSmem<D, BITS>::bytes;
    static_assert(bytes <= 227 * 1024, "shared memory");
    static PerDevice ready;
    cudaError_t e = ready.once([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    if (e != cudaSuccess)
        return e;
    const int tiles = 2 * (int)(((long long)p.T * p.c.kv_heads + 127) / 128);
    return launch_pdl(kern, dim3(tiles < num_sms ? tiles : num_sms), dim3(Geo<D>::threads),
                      (size_t)bytes, st, p, r_img, tiles);
}

template <int D, int BITS>
cudaError_t write_type(const KvWriteParams &p, const uint4 *img, int tbl_words, bool bf16,
                       cudaStream_t st, int num_sms) {
    return bf16 ? write_tc<D, BITS, true>(p, img, tbl_words, st, num_sms)
                : write_tc<D, BITS, false>(p, img, tbl_words, st, num_sms);
}

template <int D, int BITS>
cudaError_t read_type(const KvReadParams &p, const uint4 *img, bool bf16, cudaStream_t st,
                      int num_sms) {
    return bf16 ? read_tc<__nv_bfloat16, D, BITS>(p, img, st, num_sms)
                : read_tc<__half, D, BITS>(p, img, st, num_sms);
}

}  // namespace

cudaError_t launch_kv_write_tc(const KvWriteParams &p, const void *r_img, int tbl_words, bool bf16,
                               cudaStream_t st, int num_sms) {
    const uint4 *img = static_cast<const uint4 *>(r_img);
#define OQ_CASE(B)                                                                     \
    case B:                                                                            \
        return p.c.d == 128 ? write_type<128, B>(p, img, tbl_words, bf16, st, num_sms) \
                            : write_type<256, B>(p, img, tbl_words, bf16, st, num_sms)
    switch (p.c.bits) {
        OQ_CASE(2);
        OQ_CASE(3);
        OQ_CASE(4);
        OQ_CASE(6);
        OQ_CASE(8);
    }
#undef OQ_CASE
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_read_tc(const KvReadParams &p, const void *r_img, bool bf16, cudaStream_t st,
                              int num_sms) {
    const uint4 *img = static_cast<const uint4 *>(r_img);
#define OQ_CASE(B)                                                        \
    case B:                                                               \
        return p.c.d == 128 ? read_type<128, B>(p, img, bf16, st, num_sms) \
                            : read_type<256, B>(p, img, bf16, st, num_sms)
    switch (p.c.bits) {
        OQ_CASE(2);
        OQ_CASE(3);
        OQ_CASE(4);
        OQ_CASE(6);
        OQ_CASE(8);
    }
#undef OQ_CASE
    return cudaErrorInvalidValue;
}

}  // namespace oq
