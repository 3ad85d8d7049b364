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
// Table in shared memory, one copy a lane: bits 2: entry e = 16 columns of 8 bytes; else 32
// columns of 4 bytes.
template <int BITS> struct Lut {
    static constexpr int entries = BITS == 3 || BITS == 6 ? 64 : 256;
    static constexpr int bytes = entries * 128;
};

template <int BITS>
__device__ __forceinline__ void fill_lut(unsigned char *lut, const uint32_t *src) {
    if constexpr (BITS == 2) {
        for (int i = threadIdx.x; i < 256 * 16; i += blockDim.x)
            reinterpret_cast<uint2 *>(lut)[i] = reinterpret_cast<const uint2 *>(src)[i >> 4];
    } else {
        for (int i = threadIdx.x; i < Lut<BITS>::entries * 8; i += blockDim.x) {
            const uint32_t v = src[i >> 3];
            reinterpret_cast<uint4 *>(lut)[i] = make_uint4(v, v, v, v);
        }
    }
}

// Entry of the group of bits [at, at + n) of w (n <= 8, at a compile-time constant), `col` this
// lane's column offset in bytes.
__device__ __forceinline__ uint32_t look(const unsigned char *lut, uint32_t w, int at, int n,
                                         uint32_t col) {
    const uint32_t mask = ((1u << n) - 1u) << 7;
    const uint32_t sh = at >= 7 ? w >> (at - 7) : w << (7 - at);
    return *reinterpret_cast<const uint32_t *>(lut + ((sh & mask) | col));
}

// Bits [at, at + n) of the words w as the low bits of one word (at, n compile-time).
template <int W>
__device__ __forceinline__ uint32_t word_at(const uint32_t (&w)[W], int at, int n) {
    const int i = at >> 5, s = at & 31;
    if (s + n <= 32)
        return w[i] >> s;
    return __funnelshift_r(w[i], w[i + 1 < W ? i + 1 : i], s);
}

// Codes 4 i .. 4 i + 3 of the packed words w as two fp16 pairs.
template <int BITS, int W>
__device__ __forceinline__ void quad(const unsigned char *lut, const uint32_t (&w)[W], int i,
                                     uint32_t col, uint32_t &lo, uint32_t &hi) {
    if constexpr (BITS == 2) {
        const uint32_t v = w[i >> 2];
        const int at = 8 * (i & 3);
        const uint32_t sh = at >= 7 ? v >> (at - 7) : v << (7 - at);
        const uint2 e = *reinterpret_cast<const uint2 *>(lut + ((sh & 0x7f80u) | col));
        lo = e.x;
        hi = e.y;
    } else if constexpr (BITS == 4) {
        const uint32_t v = w[i >> 1];
        lo = look(lut, v, 16 * (i & 1), 8, col);
        hi = look(lut, v, 16 * (i & 1) + 8, 8, col);
    } else if constexpr (BITS == 3) {
        const uint32_t v = word_at(w, 12 * i, 12);
        lo = look(lut, v, 0, 6, col);
        hi = look(lut, v, 6, 6, col);
    } else if constexpr (BITS == 6) {
        const uint32_t v = word_at(w, 24 * i, 24);
        lo = prmt(look(lut, v, 0, 6, col), look(lut, v, 6, 6, col), 0x5410);
        hi = prmt(look(lut, v, 12, 6, col), look(lut, v, 18, 6, col), 0x5410);
    } else {
        const uint32_t v = w[i];
        lo = prmt(look(lut, v, 0, 8, col), look(lut, v, 8, 8, col), 0x5410);
        hi = prmt(look(lut, v, 16, 8, col), look(lut, v, 24, 8, col), 0x5410);
    }
}

// W words from p, in the widest loads that the address allows (ALIGN bytes).
template <int W, int ALIGN>
__device__ __forceinline__ void load_words(uint32_t (&w)[W], const uint8_t *p) {
    if constexpr (ALIGN % 16 == 0 && W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p + 4 * i));
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    } else if constexpr (ALIGN % 8 == 0 && W % 2 == 0) {
#pragma unroll
        for (int i = 0; i < W; i += 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p + 4 * i));
            w[i] = v.x, w[i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            w[i] = __ldg(reinterpret_cast<const uint32_t *>(p + 4 * i));
    }
}

}  // namespace kvops
}  // namespace oq
