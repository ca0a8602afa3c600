// cache_internal.h -- argument blocks shared by the cache's host launcher
// (cache_api.cu) and its kernels. Plain structs passed by value.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace swa {

// The cache as the kernels see it (fields as in sdpa_cache).
struct CacheView {
    int64_t b, h_kv, d;
    int64_t n_pages;
    uint32_t page_size, max_pages;
    int32_t page_shift;             // log2 of page_size if it is a power of two, else -1
    int64_t cap;                    // max_pages * page_size, < 2^31
    int32_t bits;                   // 4: groups as in cache4.cuh, strides in bytes (page, -, head)
    uint16_t *k, *v;
    int64_t k_stride[3], v_stride[3];   // page, row, head
    const int32_t* page_table;
    int32_t *lengths, *next_pos, *positions;
    float* weights;
    int32_t* status;
    int32_t stall;                  // test hook: a copy that a wait is for is left out
};

// A unit of the forward's work that is cut between parts: its sequence (-1:
// none), its number in the sequence, the parts that have some of it, and which
// of the first part's two partials is the unit's. Kept by unit where there are
// no more units than parts (so that the join has a CTA per unit), else by the
// part at whose start the unit's first cut is.
struct CacheFwdCut {
    int64_t bi, un;
    int32_t first, last, slot0;
};

// Kernel for a head dimension and a kv-head's number of rows: rows of a unit,
// keys of a tile, CTAs per SM, a unit's fixed cost in tiles.
enum CacheFwdVariant { kRows128x8, kRows64x8, kRows64x16, kTiles128, kTiles64 };
struct CacheFwdPlan {
    int variant, rows, tile, occ, unit_cost;
};
CacheFwdPlan cache_fwd_plan(int64_t d, int64_t rows);

// The same for a cache in 4 bits.
enum Cache4FwdVariant { kQ4Rows128x8, kQ4Rows128x16, kQ4Rows64x8, kQ4Rows64x16, kQ4Tiles };
CacheFwdPlan cache4_fwd_plan(int64_t d, int64_t rows);

struct CacheFwdArgs {
    CacheView c;
    int32_t s_q, h_q, group;
    int64_t window_left;
    float scale_log2;
    const uint16_t *q, *k, *v;
    int64_t q_stride[3], k_stride[3], v_stride[3], o_stride[3];
    const int64_t* tree;
    const int32_t* seq_q_lens;
    const float* sink;
    uint16_t* o;
    float* lse;
    // workspace: per part two partials [rows][d] with their (reference, sum),
    // and the cut that the part names
    int32_t unit_cost;      // a unit's fixed cost in tiles
    int32_t parts, whole;   // whole: one unit per CTA, no workspace
    int32_t cut_by_unit;
    int64_t timeout_ns;     // limit of a wait inside the tile kernel
    float *part_o, *part_ml;
    CacheFwdCut* cuts;
};

// The tile and the rows kernel's: TMA descriptors of the pools' pages (4-D: d,
// head, row, page) in boxes of 64 features x box_rows rows with the 128-byte
// swizzle; box_rows 0: none, every row is gathered. Of a cache in 4 bits there are
// no descriptors, and box_rows is the keys of a bulk copy: a power of two from 16
// that divides a page, at most a warp's step.
struct CacheTileArgs {
    CUtensorMap tm_k, tm_v;
    CacheFwdArgs f;
    int32_t box_rows;
};

struct CacheAppendArgs {
    CacheView c;
    int32_t thd;
    int64_t s, n, total;
    const uint16_t *k, *v;
    int64_t k_stride[3], v_stride[3];
    const int32_t *index, *counts, *offsets;
    int32_t rows_per_cta;
};

struct CacheReadArgs {
    CacheView c;
    int64_t s, rows;        // rows per sequence (without offsets), all output rows
    const int32_t *start, *counts, *offsets;
    uint16_t *k, *v;
    int64_t k_stride[3], v_stride[3];   // batch, token, head
    int32_t splits, per_split;          // a row's heads are shared between so many warps, so many each (set by the launcher)
    int64_t per_warp;                   // rows' sets and shares of a warp
};

struct CacheWeighArgs {
    CUtensorMap tm_k;      // as in CacheTileArgs, boxes of up to 128 rows
    int32_t box_rows, parts;
    int64_t timeout_ns;
    CacheView c;
    int32_t s_q, h_q, group;
    int64_t window_left;
    float scale_log2;
    const uint16_t* q;
    int64_t q_stride[3];
    const float* lse;
    const int32_t* q_pos;
};

struct CacheEvictArgs {
    CacheView c;
    int64_t keep, first, recent;
    int64_t m;             // most rows that a (sequence, kv-head) moves: min(keep, cap - keep)
    int32_t *holes, *tails;  // [b * h_kv][m] free slots below keep, kept slots from keep on
    int32_t* counts;       // [b * h_kv] rows to move; -1: the sequence is not touched
    int64_t timeout_ns;
    int32_t cluster;       // CTAs per head (set by the launcher)
};

// Lets a kernel have `bytes` of dynamic shared memory: asked of the driver once
// per device (`done`: a bit each).
template <class F>
cudaError_t allow_smem(F* kern, int bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

cudaError_t launch_cache_fwd(const CacheTileArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_cache_fwd_tiles(const CacheTileArgs& a, int dtype, cudaStream_t s);
// The join behind a forward kernel whose units have `rows` rows (8, 16 or 256).
cudaError_t launch_cache_fwd_join(const CacheFwdArgs& a, int dtype, int rows, cudaStream_t s);
cudaError_t launch_cache4_fwd_tiles(const CacheTileArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_cache4_fwd(const CacheTileArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_cache4_append(const CacheAppendArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_cache_advance(const CacheAppendArgs& a, cudaStream_t s);
cudaError_t launch_cache_read(const CacheReadArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_cache_append(const CacheAppendArgs& a, cudaStream_t s);
cudaError_t launch_cache_weigh(const CacheWeighArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_cache_evict(const CacheEvictArgs& a, cudaStream_t s);

}  // namespace swa
