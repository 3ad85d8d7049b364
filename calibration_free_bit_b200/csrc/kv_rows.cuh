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

}  // namespace oq
