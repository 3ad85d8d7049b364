// kv_ops.cuh -- helpers shared by the rotary-position and quantised-cache kernels: element
// types, 16-byte vectors of them as fp32, one row's rotation by a warp, code extraction.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

namespace oq {
namespace kvops {

template <class E> __device__ __forceinline__ float to_f32(E v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <class E> __device__ __forceinline__ E from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// One of a pair of kernel parameters (indexed by a variable they would go through local memory).
template <class T> __device__ __forceinline__ T pick(T const (&of)[2], int w) {
    return w ? of[1] : of[0];
}

// Shared memory laid out by address (0 .. 1023 are the system's): the bytes at address `at` of a
// kernel's dynamic array, which starts at kSharedStart; a kernel checks that with starts_there.
// (The address that instructions take has a block's rank in its cluster above those 24 bits.)
constexpr int kSharedStart = 1024;
__device__ __forceinline__ unsigned char *at_address(unsigned char *raw, int at) {
    return raw + (at - kSharedStart);
}
__device__ __forceinline__ uint32_t rank_bits(const unsigned char *raw) {
    return (uint32_t)__cvta_generic_to_shared(raw) & 0xff000000u;
}
__device__ __forceinline__ bool starts_there(const unsigned char *raw) {
    return ((uint32_t)__cvta_generic_to_shared(raw) & 0x00ffffffu) == kSharedStart;
}

// 16 bytes of elements <-> fp32 (n of them).
template <class E> struct Vec {
    static constexpr int n = 16 / sizeof(E);
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[n]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(E) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else if constexpr (std::is_same<E, __nv_bfloat16>::value) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                f[2 * i] = h.x;
                f[2 * i + 1] = h.y;
            }
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[n]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(E) == 4) {
                w[i] = __float_as_uint(f[i]);
            } else if constexpr (std::is_same<E, __nv_bfloat16>::value) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The unnormalised block Walsh-Hadamard transform (blocks of h) of a row of D held by a warp:
// lane l has positions l*(D/32) .. l*(D/32) + D/32 - 1.  It is its own transpose.
template <int D>
__device__ __forceinline__ void warp_wht(float (&z)[D / 32], int h, int lane) {
    constexpr int N = D / 32;
#pragma unroll
    for (int s = 1; s < N; s <<= 1)
        if (s < h) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (!(i & s)) {
                    const float a = z[i], b = z[i | s];
                    z[i] = a + b;
                    z[i | s] = a - b;
                }
        }
#pragma unroll
    for (int s = 1; s < 32; s <<= 1)
        if (s * N < h) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float o = __shfl_xor_sync(0xffffffffu, z[i], s);
                z[i] = (lane & s) ? o - z[i] : z[i] + o;
            }
        }
}

// Code k of an LSB-first stream of `bits`-wide codes (bits <= 8) at `row` (byte loads).
__device__ __forceinline__ uint32_t code_at(const uint8_t *row, int k, int bits) {
    const int bit = k * bits, at = bit >> 3, sh = bit & 7;
    uint32_t w = row[at];
    if (sh + bits > 8)
        w |= (uint32_t)row[at + 1] << 8;
    return (w >> sh) & ((1u << bits) - 1u);
}

}  // namespace kvops
}  // namespace oq
