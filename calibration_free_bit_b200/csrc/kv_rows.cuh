// kv_rows.cuh -- rows of the quantised cache by slot, and the error bits of the kernels that write
// and read them (kv_cache.cu, kv_tc.cu).
#pragma once

#include "kv_internal.h"

namespace oq {

enum : unsigned {
    KV_ERR_SLOT = 1u << 0,      // a slot outside the cache
    KV_ERR_WAIT = 1u << 1,      // a bounded wait gave up
};

// Row `slot` of one head in the cache: its index in norms (times row_bytes: in codes).
__device__ __forceinline__ long long cache_row(const KvView &c, long long slot, int head) {
    const long long page = slot >> c.page_log2;
    return ((page * c.kv_heads + head) << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
}
__device__ __forceinline__ bool slot_ok(const KvView &c, long long slot) {
    return slot >= 0 && slot < (c.pages << c.page_log2);
}

// ---- codes beside a boundary ----
// The quantizer's grid (oq_host.cpp, build_grid) has a value in steps of 2^-23 of its span, rounded
// twice on the way; `at`, whose top byte is the code, passes a boundary in steps of G.  A value within
// four steps of one, or of a cell's end (of normal values 5, 15 and 26 in a million at 2, 3 and 4 bits),
// is looked at again: in fp64 from the row itself, so that neither the order of fp32 sums nor the form
// that a call takes decides its code (one code off at 2 bits is an error of the value's own size).  An
// exact 0, which rows of few distinct values have many of, needs no second look, and a row has four at
// most: normal values need a fifth in fewer than one row of 10 million, but one with an element a million
// times the others would have all of its other blocks beside 0, and a call of such rows take 100 times
// as long.
__device__ __forceinline__ uint32_t distance_to_bound(uint32_t at, int G) {
    return at * 256u + (uint32_t)G * 1024u;
}
__device__ __forceinline__ uint32_t bound_width(int G) { return (uint32_t)G * 2048u; }

constexpr int kLooks = 4;       // second looks of a row

// Whether a row of this norm has second looks (all of an empty row is 0; fp32 has no codes for a norm
// that is not finite, or lost in underflow).
__device__ __forceinline__ bool looks(float norm) { return norm > 1e-18f && norm <= 3.402823466e38f; }

// The code of an exact 0: the upper one of the middle boundary.
__device__ __forceinline__ uint32_t code_of_zero(int bits) { return 1u << (bits - 1); }

// `code` or a neighbour, in fp64, by a warp whose lanes have parts of z (the position's sum, sqrt(h)
// times its value) and n (the row's squares); unit = sqrt(d / h).  bounds: 2^bits - 1 boundaries as
// fp32 and, 2^bits further on, what that leaves of them.
__device__ __forceinline__ uint32_t code_beside(uint32_t code, double z, double n, float norm,
                                                double unit, const float *bounds, int bits) {
    const uint32_t L = 1u << bits;
    auto bound = [&](uint32_t j) { return (double)bounds[j] + (double)bounds[L + j]; };
    const double below = code > 0 ? bound(code - 1) : 0.0, above = code + 1 < L ? bound(code) : 0.0;
#pragma unroll
    for (int k = 16; k; k >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, k);
        n += __shfl_xor_sync(0xffffffffu, n, k);
    }
    // sqrt(n) by two steps of Newton's from its fp32 value
    const double half_inv = 0.5f / norm;
    double s = norm;
    s += (n - s * s) * half_inv;
    s += (n - s * s) * half_inv;
    const double v = z * unit;
    s += 1e-8;
    if (code > 0 && v < below * s)
        return code - 1;
    return code + 1 < L && v >= above * s ? code + 1 : code;
}

}  // namespace oq
