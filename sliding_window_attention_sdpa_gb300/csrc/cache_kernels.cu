// cache_kernels.cu -- append and evict on the paged cache.
#include "cache.cuh"
#include "ptx.cuh"

namespace swa {

// ---------------------------------------------------------------- append

namespace {

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

}  // namespace

template <int HD>
__global__ void __launch_bounds__(256) cache_append_kernel(const CacheAppendArgs a)
{
    constexpr uint32_t C = HD / 8;   // 16-byte chunks of a row
    const int64_t bi = blockIdx.x;
    const AppendPlan p = append_plan(a, bi);
    const int32_t r0 = static_cast<int32_t>(imin64(p.n, static_cast<int64_t>(blockIdx.y) * a.rows_per_cta));
    const int32_t r1 = static_cast<int32_t>(imin64(p.n, r0 + static_cast<int64_t>(a.rows_per_cta)));
    if (p.n >= 0) {
        const uint32_t h_kv = static_cast<uint32_t>(a.c.h_kv);
        const uint32_t units = r1 > r0 ? static_cast<uint32_t>(r1 - r0) * h_kv * C : 0;
        for (uint32_t u = threadIdx.x; u < units; u += blockDim.x) {
            const uint32_t c = u % C, rh = u / C, rr = rh / h_kv, g = rh - rr * h_kv;
            const int32_t i = r0 + static_cast<int32_t>(rr);
            const int64_t src = p.src0 + (a.index ? a.index[bi * a.n + i] : i);
            uint32_t row;
            const int64_t page = cache_page(a.c, bi, static_cast<uint32_t>(p.len + i), row);
            const int64_t b0 = a.thd ? 0 : bi;
            const uint4 kx = ld_nc_v4(a.k + b0 * a.k_stride[0] + src * a.k_stride[1] + g * a.k_stride[2] + c * 8);
            const uint4 vx = ld_nc_v4(a.v + b0 * a.v_stride[0] + src * a.v_stride[1] + g * a.v_stride[2] + c * 8);
            *reinterpret_cast<uint4*>(a.c.k + page * a.c.k_stride[0] + row * a.c.k_stride[1] + g * a.c.k_stride[2] +
                                      c * 8) = kx;
            *reinterpret_cast<uint4*>(a.c.v + page * a.c.v_stride[0] + row * a.c.v_stride[1] + g * a.c.v_stride[2] +
                                      c * 8) = vx;
        }
        const uint32_t nr = r1 > r0 ? static_cast<uint32_t>(r1 - r0) : 0;
        for (uint32_t u = threadIdx.x; u < nr * h_kv; u += blockDim.x) {
            const uint32_t g = u / nr;
            const int32_t i = r0 + static_cast<int32_t>(u - g * nr);
            const int64_t at = (bi * a.c.h_kv + g) * a.c.cap + p.len + i;
            if (a.c.positions) a.c.positions[at] = a.c.next_pos[bi] + i;
            if (a.c.weights) a.c.weights[at] = 0.f;
        }
    }
    // one CTA has the whole sequence: it moves the lengths on itself
    if (gridDim.y == 1) {
        __syncthreads();
        if (threadIdx.x == 0 && p.n > 0) {
            a.c.lengths[bi] = p.len + p.n;
            if (a.c.next_pos) a.c.next_pos[bi] += p.n;
        }
    }
}

// Several CTAs shared a sequence's rows: its length moves on after them all.
__global__ void __launch_bounds__(256) cache_advance_kernel(const CacheAppendArgs a)
{
    const AppendPlan p = append_plan(a, blockIdx.x);
    if (threadIdx.x == 0 && p.n > 0) {
        a.c.lengths[blockIdx.x] = p.len + p.n;
        if (a.c.next_pos) a.c.next_pos[blockIdx.x] += p.n;
    }
}

cudaError_t launch_cache_append(const CacheAppendArgs& a0, cudaStream_t s)
{
    CacheAppendArgs a = a0;
    const int64_t most = a.index ? a.n : a.s;
    if (a.c.b == 0 || most == 0) return cudaSuccess;
    a.rows_per_cta = static_cast<int32_t>(imax64(64, (most + 65534) / 65535));
    const dim3 grid(static_cast<unsigned>(a.c.b), static_cast<unsigned>((most + a.rows_per_cta - 1) / a.rows_per_cta));
    if (a.c.d == 64) cache_append_kernel<64><<<grid, 256, 0, s>>>(a);
    else cache_append_kernel<128><<<grid, 256, 0, s>>>(a);
    if (grid.y > 1) cache_advance_kernel<<<static_cast<unsigned>(a.c.b), 256, 0, s>>>(a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- evict

namespace {

// Order of a key among those of its head: larger stays. Protected keys are
// above every weight, NaN above every number; -0 counts as 0.
__device__ __forceinline__ uint32_t evict_rank(const CacheEvictArgs& a, float w, int64_t pos, int64_t next)
{
    if (pos < a.first || pos >= next - a.recent) return 0xffffffffu;
    if (w != w) return 0xfffffffeu;
    const uint32_t x = __float_as_uint(w + 0.f);
    return x & 0x80000000u ? ~x : x | 0x80000000u;
}

constexpr int kSelThreads = 1024;

}  // namespace

// One CTA per (sequence, kv-head): the keep-th largest rank by four passes of
// 8 bits, then the free slots below keep and the kept ones behind it, in order.
__global__ void __launch_bounds__(kSelThreads) cache_evict_select_kernel(const CacheEvictArgs a)
{
    __shared__ uint32_t hist[256];
    __shared__ uint32_t sh_prefix, sh_need;
    __shared__ uint32_t warp_cnt[3][32];
    __shared__ uint32_t base[3];   // ties, holes, tails so far
    const int64_t u = blockIdx.x, bi = u / a.c.h_kv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool bad;
    const int32_t len = cache_length(a.c, bi, bad);
    if (bad || len <= a.keep) {
        if (tid == 0) a.counts[u] = -1;
        return;
    }
    const float* w = a.c.weights + u * a.c.cap;
    const int32_t* pos = a.c.positions + u * a.c.cap;
    const int64_t next = a.c.next_pos[bi];
    uint32_t prefix = 0, need = static_cast<uint32_t>(a.keep);
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int32_t j = tid; j < len; j += kSelThreads) {
            const uint32_t r = evict_rank(a, w[j], pos[j], next);
            if (shift == 24 || (r >> (shift + 8)) == prefix) atomicAdd(&hist[(r >> shift) & 255], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t left = need;
            int d = 255;
            for (; d > 0 && hist[d] < left; --d) left -= hist[d];
            sh_prefix = (prefix << 8) | static_cast<uint32_t>(d);
            sh_need = left;
        }
        __syncthreads();
        prefix = sh_prefix;
        need = sh_need;
        __syncthreads();
    }
    // ranks above `prefix` stay, and the first `need` that equal it
    if (tid < 3) base[tid] = 0;
    __syncthreads();
    for (int32_t j0 = 0; j0 < len; j0 += kSelThreads) {
        const int32_t j = j0 + tid;
        const uint32_t r = j < len ? evict_rank(a, w[j], pos[j], next) : 0;
        const bool tie = j < len && r == prefix;
        const uint32_t below = (1u << lane) - 1;
        const uint32_t bt = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) warp_cnt[0][warp] = __popc(bt);
        __syncthreads();
        uint32_t before = base[0];
        for (int i = 0; i < warp; ++i) before += warp_cnt[0][i];
        const bool kept = j < len && (r > prefix || (tie && before + __popc(bt & below) < need));
        const bool hole = j < len && !kept && j < a.keep, tail = kept && j >= a.keep;
        const uint32_t bh = __ballot_sync(0xffffffffu, hole), bl = __ballot_sync(0xffffffffu, tail);
        if (lane == 0) {
            warp_cnt[1][warp] = __popc(bh);
            warp_cnt[2][warp] = __popc(bl);
        }
        __syncthreads();
        uint32_t hb = base[1], lb = base[2];
        for (int i = 0; i < warp; ++i) {
            hb += warp_cnt[1][i];
            lb += warp_cnt[2][i];
        }
        if (hole) a.holes[u * a.m + hb + __popc(bh & below)] = j;
        if (tail) a.tails[u * a.m + lb + __popc(bl & below)] = j;
        __syncthreads();
        if (tid < 3)
            for (int i = 0; i < 32; ++i) base[tid] += warp_cnt[tid][i];
        __syncthreads();
    }
    if (tid == 0) a.counts[u] = static_cast<int32_t>(base[1]);
}

template <int HD>
__global__ void __launch_bounds__(256) cache_evict_move_kernel(const CacheEvictArgs a)
{
    constexpr uint32_t C = HD / 8;
    const int64_t u = blockIdx.x, bi = u / a.c.h_kv, g = u - bi * a.c.h_kv;
    const int32_t n = a.counts[u];
    if (n < 0) return;
    if (blockIdx.y == 0 && g == 0 && threadIdx.x == 0) a.c.lengths[bi] = static_cast<int32_t>(a.keep);
    for (int64_t x = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x; x < static_cast<int64_t>(n) * C;
         x += static_cast<int64_t>(gridDim.y) * blockDim.x) {
        const uint32_t c = static_cast<uint32_t>(x % C);
        const int64_t i = x / C;
        const uint32_t dst = a.holes[u * a.m + i], src = a.tails[u * a.m + i];
        if (c == 0) {
            a.c.positions[u * a.c.cap + dst] = a.c.positions[u * a.c.cap + src];
            a.c.weights[u * a.c.cap + dst] = a.c.weights[u * a.c.cap + src];
        }
        uint32_t sr, dr;
        const int64_t sp = cache_page(a.c, bi, src, sr), dp = cache_page(a.c, bi, dst, dr);
        if (sp < 0 || dp < 0) continue;
        *reinterpret_cast<uint4*>(a.c.k + dp * a.c.k_stride[0] + dr * a.c.k_stride[1] + g * a.c.k_stride[2] + c * 8) =
            *reinterpret_cast<const uint4*>(a.c.k + sp * a.c.k_stride[0] + sr * a.c.k_stride[1] +
                                            g * a.c.k_stride[2] + c * 8);
        *reinterpret_cast<uint4*>(a.c.v + dp * a.c.v_stride[0] + dr * a.c.v_stride[1] + g * a.c.v_stride[2] + c * 8) =
            *reinterpret_cast<const uint4*>(a.c.v + sp * a.c.v_stride[0] + sr * a.c.v_stride[1] +
                                            g * a.c.v_stride[2] + c * 8);
    }
}

cudaError_t launch_cache_evict(const CacheEvictArgs& a, cudaStream_t s)
{
    const int64_t units = a.c.b * a.c.h_kv;
    if (units == 0 || a.c.cap <= a.keep) return cudaSuccess;
    cache_evict_select_kernel<<<static_cast<unsigned>(units), kSelThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(units),
                    static_cast<unsigned>(imax64(1, imin64((a.m * (a.c.d / 8) + 255) / 256, 256))));
    if (a.c.d == 64) cache_evict_move_kernel<64><<<grid, 256, 0, s>>>(a);
    else cache_evict_move_kernel<128><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace swa
