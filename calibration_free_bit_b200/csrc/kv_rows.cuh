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
// is looked at again in fp32.
__device__ __forceinline__ uint32_t distance_to_bound(uint32_t at, int G) {
    return at * 256u + (uint32_t)G * 1024u;
}
__device__ __forceinline__ uint32_t bound_width(int G) { return (uint32_t)G * 2048u; }

// The code of the value v, one of `code` and its neighbours, by the boundaries about it.
__device__ __forceinline__ uint32_t code_beside(uint32_t code, float v, float below, float above,
                                                int bits) {
    if (code > 0 && v < below)
        return code - 1;
    return code + 1 < (1u << bits) && v >= above ? code + 1 : code;
}

}  // namespace oq
