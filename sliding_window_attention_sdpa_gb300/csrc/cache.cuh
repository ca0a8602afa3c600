// cache.cuh -- device helpers on the paged cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/sdpa_bwd.h"
#include "cache_internal.h"
#include "seq.cuh"

namespace swa {

// The page-table entry of a slot of sequence bi, and the slot's row in its page
// (a cache with a page table).
__device__ __forceinline__ int32_t cache_entry(const CacheView& c, int64_t bi, uint32_t slot)
{
    return c.page_table[bi * c.max_pages + (c.page_shift >= 0 ? slot >> c.page_shift : slot / c.page_size)];
}

__device__ __forceinline__ uint32_t cache_row(const CacheView& c, uint32_t slot)
{
    return c.page_shift >= 0 ? slot & ((1u << c.page_shift) - 1) : slot % c.page_size;
}

// The page that holds `slot` of sequence bi, or -1 (recorded) if the table's
// entry is outside [0, n_pages); `row` becomes the slot's row in it.
__device__ __forceinline__ int64_t cache_page(const CacheView& c, int64_t bi, uint32_t slot, uint32_t& row)
{
    if (c.page_table == nullptr) {
        row = slot;
        return bi;
    }
    const uint32_t p = c.page_shift >= 0 ? slot >> c.page_shift : slot / c.page_size;
    row = slot - p * c.page_size;
    const int64_t page = c.page_table[bi * c.max_pages + p];
    if (page < 0 || page >= c.n_pages) {
        set_status(c.status, SDPA_ERR_BOUNDS);
        return -1;
    }
    return page;
}

// lengths[bi] within [0, cap]; one out of it is recorded and taken as the
// nearer end.
__device__ __forceinline__ int32_t cache_length(const CacheView& c, int64_t bi, bool& bad)
{
    const int32_t n = c.lengths[bi];
    bad = n < 0 || n > c.cap;
    if (bad) set_status(c.status, SDPA_ERR_BAD_LENGTHS);
    return n < 0 ? 0 : (n > c.cap ? static_cast<int32_t>(c.cap) : n);
}

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t x)
{
    if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(x) << 16);
    return __half2float(__ushort_as_half(x));
}

template <bool BF16>
__device__ __forceinline__ uint16_t from_float(float x)
{
    if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    return __half_as_ushort(__float2half_rn(x));
}

}  // namespace swa
