// kv_lut.cuh -- packed codes to pairs of fp16 centroids through a table in shared memory (the image
// is build_kv_lut's, oq_cache.cpp), for the kernels that read the quantised cache.
#pragma once

#include <cstdint>

namespace oq {
namespace kvops {

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// ---- codes -> pairs of fp16 centroids ----
// Table in shared memory, one copy a lane, so that any entries at once are free of bank conflicts.
// What a decode costs is the address of each lookup, so a table's form and place make that cheap:
//   WIDE    entries of a whole byte (bits 2, 4, 8) 256 bytes apart (the second half is not used), the
//           table at a multiple of 64 KB: one byte permute of the code word and a constant of the
//           lane is the address.  (bits 3, 6: as PLACED)
//   PLACED  entries 128 bytes apart, the table at a multiple of its size: a shift, and a mask and an
//           or in one
//   ANYWHERE  entries 128 bytes apart: a shift, a mask and a sum.
// A lane's column has 8 bytes at bits 2 (16 columns, two lanes each), else 4.
enum LutForm { WIDE, PLACED, ANYWHERE };

template <int BITS, LutForm FORM> struct Lut {
    static constexpr bool whole = BITS != 3 && BITS != 6;
    static constexpr int entries = whole ? 256 : 64;
    static constexpr int pitch = whole && FORM == WIDE ? 256 : 128;
    static constexpr int bytes = entries * pitch;
};

template <int BITS, LutForm FORM>
__device__ __forceinline__ void fill_lut(unsigned char *lut, const uint32_t *src) {
    using L = Lut<BITS, FORM>;
    for (int i = threadIdx.x; i < L::entries * 8; i += blockDim.x) {
        uint4 v;
        if constexpr (BITS == 2) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(src) + (i >> 3));
            v = make_uint4(u.x, u.y, u.x, u.y);
        } else {
            const uint32_t u = __ldg(src + (i >> 3));
            v = make_uint4(u, u, u, u);
        }
        *reinterpret_cast<uint4 *>(lut + (i >> 3) * L::pitch + (i & 7) * 16) = v;
    }
}

// A lane's constant for a table at shared address `at`.
template <int BITS, LutForm FORM>
__device__ __forceinline__ uint32_t lut_column(uint32_t at, int lane) {
    const uint32_t col = BITS == 2 ? (lane & 15) * 8 : lane * 4;
    return Lut<BITS, FORM>::pitch == 256 ? col | (at >> 8) : at + col;
}

__device__ __forceinline__ void table_load(uint32_t &v, uint32_t at) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
}
__device__ __forceinline__ void table_load(uint2 &v, uint32_t at) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
}

// Entry of byte k of w (k a compile-time constant).
template <class V, LutForm FORM>
__device__ __forceinline__ V look8(uint32_t w, int k, uint32_t col) {
    V v;
    if constexpr (FORM == WIDE) {
        table_load(v, prmt(w, col, 0x6504u | ((uint32_t)k << 4)));
    } else {
        const uint32_t sh = (k ? w >> (8 * k - 7) : w << 7) & 0x7f80u;
        table_load(v, FORM == PLACED ? sh | col : sh + col);
    }
    return v;
}

// Entry of the 6 bits of w from bit `at` on.
template <LutForm FORM>
__device__ __forceinline__ uint32_t look6(uint32_t w, int at, uint32_t col) {
    const uint32_t sh = (at >= 7 ? w >> (at - 7) : w << (7 - at)) & (63u << 7);
    uint32_t v;
    table_load(v, FORM == ANYWHERE ? sh + col : sh | col);
    return v;
}

// Bits [at, at + n) of the words w as the low bits of one word (at, n compile-time).
template <int W>
__device__ __forceinline__ uint32_t word_at(const uint32_t (&w)[W], int at, int n) {
    const int i = at >> 5, s = at & 31;
    if (s + n <= 32)
        return w[i] >> s;
    return __funnelshift_r(w[i], w[i + 1 < W ? i + 1 : i], s);
}

// Codes 4 i .. 4 i + 3 of the packed words w as two fp16 pairs; of 6 and 8 bits, whose entries are one
// centroid and what fp16 leaves of it, also the pairs of the rests.
template <int BITS, LutForm FORM, int W>
__device__ __forceinline__ void quad(const uint32_t (&w)[W], int i, uint32_t col, uint32_t &lo,
                                     uint32_t &hi, uint32_t &lo_rest, uint32_t &hi_rest) {
    if constexpr (BITS == 2) {
        const uint2 e = look8<uint2, FORM>(w[i >> 2], i & 3, col);
        lo = e.x;
        hi = e.y;
    } else if constexpr (BITS == 4) {
        lo = look8<uint32_t, FORM>(w[i >> 1], 2 * (i & 1), col);
        hi = look8<uint32_t, FORM>(w[i >> 1], 2 * (i & 1) + 1, col);
    } else if constexpr (BITS == 3) {
        const uint32_t v = word_at(w, 12 * i, 12);
        lo = look6<FORM>(v, 0, col);
        hi = look6<FORM>(v, 6, col);
    } else if constexpr (BITS == 6) {
        const uint32_t v = word_at(w, 24 * i, 24);
        const uint32_t e[4] = {look6<FORM>(v, 0, col), look6<FORM>(v, 6, col),
                               look6<FORM>(v, 12, col), look6<FORM>(v, 18, col)};
        lo = prmt(e[0], e[1], 0x5410), hi = prmt(e[2], e[3], 0x5410);
        lo_rest = prmt(e[0], e[1], 0x7632), hi_rest = prmt(e[2], e[3], 0x7632);
    } else {
        const uint32_t v = w[i];
        const uint32_t e[4] = {look8<uint32_t, FORM>(v, 0, col), look8<uint32_t, FORM>(v, 1, col),
                               look8<uint32_t, FORM>(v, 2, col), look8<uint32_t, FORM>(v, 3, col)};
        lo = prmt(e[0], e[1], 0x5410), hi = prmt(e[2], e[3], 0x5410);
        lo_rest = prmt(e[0], e[1], 0x7632), hi_rest = prmt(e[2], e[3], 0x7632);
    }
}
template <int BITS, LutForm FORM, int W>
__device__ __forceinline__ void quad(const uint32_t (&w)[W], int i, uint32_t col, uint32_t &lo,
                                     uint32_t &hi) {
    uint32_t a, b;
    quad<BITS, FORM>(w, i, col, lo, hi, a, b);
}

// The same codes of two rows x and y (the packed words of each), transposed: o[k] = (code 4 i + k
// of x, that of y).  4-bit codes are merged to bytes of one code of each row first (`mixed`).
template <int BITS, LutForm FORM, int W>
__device__ __forceinline__ void quad_of_two(const uint32_t (&x)[W], const uint32_t (&y)[W], int i,
                                            uint32_t col, uint32_t (&o)[4], uint32_t (&rest)[4]) {
    if constexpr (BITS == 4) {
        // x = even codes of both rows, y = odd ones
        const int k = 2 * (i & 1);
        o[0] = look8<uint32_t, FORM>(x[i >> 1], k, col);
        o[1] = look8<uint32_t, FORM>(y[i >> 1], k, col);
        o[2] = look8<uint32_t, FORM>(x[i >> 1], k + 1, col);
        o[3] = look8<uint32_t, FORM>(y[i >> 1], k + 1, col);
    } else if constexpr (BITS == 6) {
        const uint32_t u = word_at(x, 24 * i, 24), v = word_at(y, 24 * i, 24);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t a = look6<FORM>(u, 6 * k, col), b = look6<FORM>(v, 6 * k, col);
            o[k] = prmt(a, b, 0x5410);
            rest[k] = prmt(a, b, 0x7632);
        }
    } else if constexpr (BITS == 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t a = look8<uint32_t, FORM>(x[i], k, col);
            const uint32_t b = look8<uint32_t, FORM>(y[i], k, col);
            o[k] = prmt(a, b, 0x5410);
            rest[k] = prmt(a, b, 0x7632);
        }
    } else {
        uint32_t a, b, c, d;
        quad<BITS, FORM>(x, i, col, a, b);
        quad<BITS, FORM>(y, i, col, c, d);
        o[0] = prmt(a, c, 0x5410);
        o[1] = prmt(a, c, 0x7632);
        o[2] = prmt(b, d, 0x5410);
        o[3] = prmt(b, d, 0x7632);
    }
}

// Two rows' words as quad_of_two takes them.
template <int BITS, int W>
__device__ __forceinline__ void mixed(uint32_t (&x)[W], uint32_t (&y)[W]) {
    if constexpr (BITS == 4) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t a = x[i], b = y[i];
            x[i] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
            y[i] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
        }
    }
}

// W words of a cache's codes, in the widest loads that the address allows (ALIGN bytes).  Plain loads:
// the kernel that writes them may still run when the one that reads them starts (it waits, but data
// behind the non-coherent path has to stay the same for a kernel's whole life).
template <int W, int ALIGN>
__device__ __forceinline__ void load_words(uint32_t (&w)[W], const uint8_t *p) {
    if constexpr (ALIGN % 16 == 0 && W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    } else if constexpr (ALIGN % 8 == 0 && W % 2 == 0) {
#pragma unroll
        for (int i = 0; i < W; i += 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p + 4 * i);
            w[i] = v.x, w[i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            w[i] = *reinterpret_cast<const uint32_t *>(p + 4 * i);
    }
}

}  // namespace kvops
}  // namespace oq
