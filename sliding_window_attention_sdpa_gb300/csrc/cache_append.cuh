// cache_append.cuh -- what the appending kernels share.
#pragma once

#include "cache.cuh"

namespace swa {

// Rows that sequence bi appends, from which source row, behind how many keys;
// -1 rows (recorded) if they cannot be appended. Every thread of the CTA calls it.
struct AppendPlan {
    int64_t src0;
    int32_t n, len;
};

__device__ __forceinline__ AppendPlan append_plan(const CacheAppendArgs& a, int64_t bi)
{
    AppendPlan p;
    p.len = a.c.lengths[bi];
    p.src0 = 0;
    int64_t most = a.index ? a.n : a.s;
    bool ok = p.len >= 0 && p.len <= a.c.cap;
    if (a.thd) {
        p.src0 = a.offsets[bi];
        const int64_t end = a.offsets[bi + 1];
        most = end - p.src0;
        ok = ok && p.src0 >= 0 && most >= 0 && most <= a.s && end <= a.total;
    }
    int64_t n = a.counts ? a.counts[bi] : most;
    ok = ok && n >= 0 && n <= most && p.len + n <= a.c.cap;
    if (a.c.next_pos) ok = ok && a.c.next_pos[bi] >= 0 && a.c.next_pos[bi] + n <= 0x7fffffff;
    bool fine = true;
    if (ok && a.index)
        for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
            const int32_t x = a.index[bi * a.n + i];
            fine = fine && x >= 0 && x < a.s;
        }
    if (!__syncthreads_and(ok && fine)) {
        if (threadIdx.x == 0) set_status(a.c.status, SDPA_ERR_BAD_LENGTHS);
        p.n = -1;
        return p;
    }
    bool paged = true;
    if (n > 0 && a.c.page_table != nullptr) {
        const uint32_t p0 = static_cast<uint32_t>(p.len) / a.c.page_size;
        const uint32_t p1 = static_cast<uint32_t>(p.len + n - 1) / a.c.page_size;
        for (uint32_t i = p0 + threadIdx.x; i <= p1; i += blockDim.x) {
            const int32_t page = a.c.page_table[bi * a.c.max_pages + i];
            paged = paged && page >= 0 && page < a.c.n_pages;
        }
    }
    if (!__syncthreads_and(paged)) {
        if (threadIdx.x == 0) set_status(a.c.status, SDPA_ERR_BOUNDS);
        p.n = -1;
        return p;
    }
    p.n = static_cast<int32_t>(n);
    return p;
}

}  // namespace swa
