// cache_kernels.cu -- append and evict on the paged cache.
#include <cooperative_groups.h>

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

// Bound by reading and writing each row once: prompts of 16 sequences (68,000
// rows of 8 kv-heads, d = 128, in bf16) 89 us, 6.2 TB/s. A thread copies 16
// bytes of K and of V at a time; what hides the latency is the number of CTAs
// on an SM, not copies in flight per thread (2 or 4 of each at once: 91 and 106
// us). Whether the sequence can be appended at all is found by every one of its
// CTAs for itself, so that nothing is written of one that cannot.
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
    if (a.c.b == 0) return cudaSuccess;
    // A CTA takes 2048 16-byte pieces of K (8 a thread), one the whole sequence up to 4096: then the second launch
    // (2.7 us) is spared. Prompts of up to 8192 rows, 8 kv-heads, d = 128, with 16 rows a CTA against 64: 6 us against
    // 14 for one sequence, 29 against 48 for 4, 89 against 90 for 16; 8 rows: 5, 28 and 92. At most 2048 CTAs a
    // sequence: each looks through all of its indexes and pages.
    const int64_t per_row = a.c.h_kv * (a.c.d / 8);
    int64_t rows = most * per_row <= 4096 ? most : 2048 / per_row;
    rows = imin64(imax64(rows, most / 2048), (int64_t(1) << 31) / per_row);
    a.rows_per_cta = static_cast<int32_t>(imax64(imax64(rows, 1), (most + 65534) / 65535));
    const dim3 grid(static_cast<unsigned>(a.c.b),
                    static_cast<unsigned>(imax64(1, (most + a.rows_per_cta - 1) / a.rows_per_cta)));
    if (a.c.d == 64) cache_append_kernel<64><<<grid, 256, 0, s>>>(a);
    else cache_append_kernel<128><<<grid, 256, 0, s>>>(a);
    if (grid.y > 1) cache_advance_kernel<<<static_cast<unsigned>(a.c.b), 256, 0, s>>>(a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- evict
//
// A head's kept keys are the `keep` of the highest rank (protected ones above
// every weight). A cluster of up to 16 CTAs takes a (sequence, kv-head): each
// CTA reads its slice of weights and positions once and keeps the ranks in
// shared memory; four passes of 8 bits find the keep-th largest rank, the CTAs'
// histograms added through distributed shared memory; then each warp, in slot
// order, lists the free slots below `keep` and the kept ones from there on. A
// histogram has a column per lane (256 x 32 counters): lanes never meet on a
// counter or a bank, whatever the weights. It is not bound by its reads: 11 us
// for 16 heads of 1100 keys, a chain of barriers and cluster barriers mostly, and
// what grows with a slice, the ranks that four passes and two walks look at each:
// 21.6 us for 72 heads of 16484 keys, 42 for 8 heads of 262161 (slices of 16385
// keys, 16 CTAs a head). The second
// kernel moves the rows, bound by reading and writing each moved row once.

namespace {

// Order of a key among those of its head: larger stays. Protected keys are
// above every weight, NaN above every number; -0 counts as 0.
__device__ __forceinline__ uint32_t evict_rank(const CacheEvictArgs& a, float w, int64_t pos, int64_t next)
{
    // (no branches: the loads of several keys are on their way at once)
    const uint32_t x = __float_as_uint(w + 0.f), flip = static_cast<uint32_t>(static_cast<int32_t>(x) >> 31) | 0x80000000u;
    const uint32_t r = w != w ? 0xfffffffeu : x ^ flip;
    return (pos < a.first) | (pos >= next - a.recent) ? 0xffffffffu : r;
}

constexpr uint32_t kSelFixed = 256 * 32 * 4;       // the histogram; the ranks follow it

}  // namespace

// CACHED: a slice's ranks fit shared memory; else each pass computes them.
// T: threads.
template <bool CACHED, int T>
__global__ void __launch_bounds__(T, 1024 / T) cache_evict_select_kernel(const __grid_constant__ CacheEvictArgs a)
{
    namespace cg = cooperative_groups;
    constexpr int W = T / 32;
    extern __shared__ __align__(16) uint32_t dyn32[];
    uint32_t* hist = dyn32;
    uint32_t* ranks = dyn32 + kSelFixed / 4;
    __shared__ uint32_t tot[2][256];        // this CTA's histogram of a pass
    __shared__ uint32_t mine[3];            // this CTA's ties, free slots, kept slots behind
    __shared__ uint32_t per_warp[3][W];
    __shared__ uint32_t sums[256];          // all CTAs' histogram of a pass
    __shared__ uint32_t digit, left, equal;
    cg::cluster_group cl = cg::this_cluster();
    const uint32_t cs = static_cast<uint32_t>(a.cluster), c = blockIdx.x % cs;
    const int64_t u = blockIdx.x / cs, bi = u / a.c.h_kv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool bad;
    const int32_t len = cache_length(a.c, bi, bad);
    if (bad || len <= a.keep) {             // (the whole cluster)
        if (c == 0 && tid == 0) a.counts[u] = -1;
        grid_dep_launch();
        return;
    }
    const int32_t keep = static_cast<int32_t>(a.keep);
    const float* w = a.c.weights + u * a.c.cap;
    const int32_t* pos = a.c.positions + u * a.c.cap;
    const int64_t next = a.c.next_pos[bi];
    // this CTA's slots [lo, hi), a multiple of 32 per warp
    const int32_t slice = static_cast<int32_t>((((static_cast<int64_t>(len) + cs - 1) / cs) + T - 1) / T * T);
    const int32_t lo = static_cast<int32_t>(imin64(len, static_cast<int64_t>(c) * slice));
    const int32_t hi = static_cast<int32_t>(imin64(len, static_cast<int64_t>(lo) + slice)), n = hi - lo;
    auto rank_of = [&](int32_t i) -> uint32_t {
        if constexpr (CACHED) return ranks[i];
        return evict_rank(a, w[lo + i], pos[lo + i], next);
    };
    if constexpr (CACHED) {
#pragma unroll 8
        for (int32_t i = tid; i < n; i += T) ranks[i] = evict_rank(a, w[lo + i], pos[lo + i], next);
    }
    uint32_t prefix = 0, need = static_cast<uint32_t>(keep);
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
#pragma unroll
        for (int i = 0; i < 8192 / T; ++i) hist[i * T + tid] = 0;
        __syncthreads();
        auto put = [&](uint32_t r) {
            if (pass == 0 || (r >> (shift + 8)) == prefix) atomicAdd(&hist[((r >> shift) & 255) * 32 + lane], 1u);
        };
        if constexpr (CACHED) {
#pragma unroll 2
            for (int32_t i = tid * 4; i < n; i += T * 4) {
                const uint4 r = *reinterpret_cast<const uint4*>(ranks + i);      // (the room is a multiple of 4)
                put(r.x);
                if (i + 1 < n) put(r.y);
                if (i + 2 < n) put(r.z);
                if (i + 3 < n) put(r.w);
            }
        } else {
#pragma unroll 4
            for (int32_t i = tid; i < n; i += T) put(rank_of(i));
        }
        __syncthreads();
        {
            // two or four threads a bin, 16 or 8 columns each (each bin from another bank on)
            constexpr int Q = T / 256, N = 32 / Q;
            const int bin = tid / Q, q = tid % Q;
            uint32_t s = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) s += hist[bin * 32 + ((q * N + i + bin) & 31)];
#pragma unroll
            for (int o = 1; o < Q; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (q == 0) tot[pass & 1][bin] = s;
        }
        // (a buffer is written again two passes on: every CTA has read it by the barrier between)
        cl.sync();
        if (tid < 256) {
            uint32_t x = 0;
#pragma unroll
            for (uint32_t k = 0; k < 16; ++k)
                if (k < cs) x += *cl.map_shared_rank(&tot[pass & 1][tid], k);
            sums[tid] = x;
        }
        __syncthreads();
        if (warp == 0) {
            // lane l: bins 255 - 8l down to 248 - 8l
            uint32_t b[8], s = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += b[i] = sums[255 - 8 * lane - i];
            uint32_t incl = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            // the first bin, from the top, by which `need` are reached (there are at least `need` in all)
            uint32_t before = incl - s;
            if (before < need ? need <= incl : need == 0 && lane == 0) {
                uint32_t d = 255 - 8 * lane;
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if (before + b[i] < need && d == 255u - 8 * lane - i) {
                        before += b[i];
                        --d;
                    }
                digit = d;
                left = need - before;
                equal = sums[d];
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | digit;
        need = left;
        __syncthreads();
    }
    // Ranks above `prefix` stay, and the first `need` (in slot order) that equal it; where those are all, their
    // order does not matter. Each warp looks after consecutive slots.
    if (need == equal) need = 0xffffffffu;
    const int32_t seg = slice / W, i0 = warp * seg, i1 = min(n, i0 + seg);
    const uint32_t below = (1u << lane) - 1;
    // sum of what comes before this warp: earlier CTAs' counts, earlier warps'
    auto before_me = [&](int what) -> uint32_t {
        uint32_t s = lane < warp ? per_warp[what][lane] : 0;
        if (lane < static_cast<int>(c)) s += *cl.map_shared_rank(&mine[what], lane);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    };
    auto count = [&](int what, uint32_t v) {     // of this warp
        if (lane == 0) per_warp[what][warp] = v;
    };
    auto total = [&](int what) {
        if (warp == what) {
            uint32_t s = lane < W ? per_warp[what][lane] : 0;
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) mine[what] = s;
        }
    };
    uint32_t tie0 = 0;
    if (need != 0xffffffffu) {              // (the same in every CTA of the cluster)
        uint32_t ties = 0;
        for (int32_t i = i0 + lane; i - lane < i1; i += 32)
            ties += __popc(__ballot_sync(0xffffffffu, i < i1 && rank_of(i) == prefix));
        count(0, ties);
        __syncthreads();
        total(0);
        cl.sync();
        tie0 = before_me(0);
    }
    // f(slot, free below keep, kept behind it) in slot order, whole warps; a warp's slots mostly lie on one side of
    // `keep`
    auto walk = [&](auto f) {
        uint32_t t = tie0;
        for (int32_t i = i0 + lane; i - lane < i1; i += 128) {
            uint32_t rs[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) rs[q] = i + 32 * q < i1 ? rank_of(i + 32 * q) : 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool in = i + 32 * q < i1;
                const uint32_t r = rs[q];
                bool kept = in && r >= prefix;
                if (need != 0xffffffffu) {
                    const uint32_t bt = __ballot_sync(0xffffffffu, in && r == prefix);
                    kept = in && (r > prefix || (r == prefix && t + __popc(bt & below) < need));
                    t += __popc(bt);
                }
                const int32_t j = lo + i + 32 * q, j0 = j - lane;
                f(j, j0 < keep ? __ballot_sync(0xffffffffu, in && !kept && j < keep) : 0u,
                  j0 + 31 >= keep ? __ballot_sync(0xffffffffu, kept && j >= keep) : 0u);
            }
        }
    };
    uint32_t holes = 0, tails = 0;
    walk([&](int32_t, uint32_t h, uint32_t t) {
        holes += __popc(h);
        tails += __popc(t);
    });
    count(1, holes);
    count(2, tails);
    __syncthreads();
    total(1);
    total(2);
    cl.sync();
    uint32_t h0 = before_me(1), t0 = before_me(2);
    if (c == cs - 1 && warp == W - 1 && lane == 0) a.counts[u] = static_cast<int32_t>(h0 + holes);
    walk([&](int32_t j, uint32_t h, uint32_t t) {
        if ((h >> lane) & 1) a.holes[u * a.m + h0 + __popc(h & below)] = j;
        if ((t >> lane) & 1) a.tails[u * a.m + t0 + __popc(t & below)] = j;
        h0 += __popc(h);
        t0 += __popc(t);
    });
    grid_dep_launch();
    cl.sync();      // no CTA ends while another reads its counts
}

// Moves kept rows into free slots: a lane looks after a row (K and V of 64
// features) or half of one (K or V of 128), one bulk copy into shared memory
// and one out of it; a warp's 8 KB of rows come in while the 8 KB before go out.
// Where a round goes and comes from is loaded a round ahead, and the positions
// and weights are written behind its copies: 72 heads that move 4,100 rows each
// of d = 128 take 55 us (5.5 TB/s), 61 before; rows of 128 bytes (d = 64) 42 us
// (3.6 TB/s: a copy costs the engine the same).
template <int HD>
__global__ void __launch_bounds__(128) cache_evict_move_kernel(const __grid_constant__ CacheEvictArgs a)
{
    constexpr int GP = HD == 64 ? 32 : 16;             // rows of a warp's round
    constexpr uint32_t RB = HD * 2;                    // bytes of a row of K or V
    extern __shared__ __align__(128) uint8_t dyn8[];   // [warp][2 rounds][8 KB]
    __shared__ __align__(8) uint64_t bars[4][2];
    const int64_t u = blockIdx.x, bi = u / a.c.h_kv, g = u - bi * a.c.h_kv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < 8) mbar_init(smem_u32(&bars[0][0]) + threadIdx.x * 8, 1);
    fence_mbar_init();
    __syncthreads();
    grid_dep_wait();
    const int32_t n = a.counts[u];
    if (n < 0) return;
    if (blockIdx.y == 0 && g == 0 && threadIdx.x == 0) a.c.lengths[bi] = static_cast<int32_t>(a.keep);
    const int64_t step = static_cast<int64_t>(gridDim.y) * 4 * GP;
    int64_t i0 = (static_cast<int64_t>(blockIdx.y) * 4 + warp) * GP;
    const uint32_t ring = smem_u32(dyn8) + warp * 16384;
    // this lane's part of the rounds on their way: where it goes
    uint16_t *kd[2] = {nullptr, nullptr}, *vd[2] = {nullptr, nullptr};
    // and where the round after them goes and comes from
    int32_t hole = 0, tail = 0;
    auto look = [&](int64_t first) {
        const int64_t i = first + lane % GP;
        if (i < n) {
            hole = a.holes[u * a.m + i];
            tail = a.tails[u * a.m + i];
        }
    };
    auto send = [&](int r, int64_t first) {
        const int64_t i = first + lane % GP;
        bool ok = i < n;
        const bool account = ok && lane < GP;
        const uint32_t dst = hole, src = tail;
        const uint16_t *ks = nullptr, *vs = nullptr;
        int32_t pos = 0;
        float w = 0.f;
        if (ok) {
            if (account) {
                pos = a.c.positions[u * a.c.cap + src];
                w = a.c.weights[u * a.c.cap + src];
            }
            uint32_t sr, dr;
            const int64_t sp = cache_page(a.c, bi, src, sr), dp = cache_page(a.c, bi, dst, dr);
            ok = sp >= 0 && dp >= 0;
            ks = a.c.k + sp * a.c.k_stride[0] + sr * a.c.k_stride[1] + g * a.c.k_stride[2];
            vs = a.c.v + sp * a.c.v_stride[0] + sr * a.c.v_stride[1] + g * a.c.v_stride[2];
            kd[r] = a.c.k + dp * a.c.k_stride[0] + dr * a.c.k_stride[1] + g * a.c.k_stride[2];
            vd[r] = a.c.v + dp * a.c.v_stride[0] + dr * a.c.v_stride[1] + g * a.c.v_stride[2];
        }
        // 64 features: K and V by each lane; 128: K by the lower lanes, V by the upper
        const bool k_mine = ok && (HD == 64 || lane < 16), v_mine = ok && (HD == 64 || lane >= 16);
        if (!k_mine) kd[r] = nullptr;
        if (!v_mine) vd[r] = nullptr;
        const uint32_t bar = smem_u32(&bars[warp][r]);
        const uint32_t copies = __popc(__ballot_sync(0xffffffffu, k_mine)) + __popc(__ballot_sync(0xffffffffu, v_mine));
        if (lane == 0) mbar_arrive_expect_tx(bar, copies * RB);
        __syncwarp();
        const uint32_t at = ring + r * 8192 + (lane % GP) * RB;
        if (k_mine) bulk_load(at, ks, RB, bar);
        if (v_mine) bulk_load(at + 4096, vs, RB, bar);
        look(first + step);
        if (account) {
            a.c.positions[u * a.c.cap + dst] = pos;
            a.c.weights[u * a.c.cap + dst] = w;
        }
    };
    auto store = [&](uint16_t* dst, uint32_t src) {
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(RB) : "memory");
    };
    uint32_t par[2] = {0u, 0u};
    // (test hook: this warp's second round never comes)
    const int64_t never = a.c.stall ? i0 + step : -1;
    look(i0);
    if (i0 < n) send(0, i0);
    int r = 0;
    for (; i0 < n; i0 += step, r ^= 1) {
        // the other half's rows have left it: the next round may come in
        bulk_wait_read0();
        __syncwarp();
        if (i0 + step < n && i0 + step != never) send(r ^ 1, i0 + step);
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[warp][r]), par[r], a.timeout_ns))) {
            // no more rounds; both that are on their way end before the CTA does
            set_status(a.c.status, SDPA_ERR_TIMEOUT);
            mbar_wait(smem_u32(&bars[warp][r]), par[r], a.timeout_ns);
            if (i0 + step < n) mbar_wait(smem_u32(&bars[warp][r ^ 1]), par[r ^ 1], a.timeout_ns);
            break;
        }
        par[r] ^= 1;
        const uint32_t at = ring + r * 8192 + (lane % GP) * RB;
        fence_proxy_async_smem();
        if (kd[r] != nullptr) store(kd[r], at);
        if (vd[r] != nullptr) store(vd[r], at + 4096);
        bulk_commit();
    }
    bulk_wait0();
}

namespace {

constexpr uint32_t kSelMost = 200 * 1024;      // shared memory of a select CTA, at most
constexpr uint32_t kMoveBytes = 65536;
constexpr int64_t kWideSlice = 4096;

// Whether clusters of 16 run on the current device (not every partition of a
// GPU promises them): asked once per device.
template <bool CACHED, int T>
bool clusters_of_16()
{
    static std::atomic<uint64_t> known{0}, yes{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
    const uint64_t bit = uint64_t(1) << dev;
    if (!(known.load(std::memory_order_acquire) & bit)) {
        auto kern = cache_evict_select_kernel<CACHED, T>;
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 16;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(T);
        cfg.dynamicSmemBytes = kSelMost;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int fit = 0;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&fit, kern, &cfg) == cudaSuccess && fit > 0)
            yes.fetch_or(bit, std::memory_order_relaxed);
        cudaGetLastError();
        known.fetch_or(bit, std::memory_order_release);
    }
    return yes.load(std::memory_order_relaxed) & bit;
}

// CTAs of T threads, a cluster of a.cluster for each of `units` heads.
template <bool CACHED, int T>
cudaError_t launch_select(CacheEvictArgs& a, int64_t units, cudaStream_t s)
{
    if (a.cluster == 16 && !clusters_of_16<CACHED, T>()) a.cluster = 8;
    const int64_t most = (a.c.cap + a.cluster - 1) / a.cluster + T;
    // a slice's ranks are kept as far as shared memory goes; a longer one's are computed in each pass
    if (CACHED && most > (kSelMost - kSelFixed) / 4) return launch_select<false, T>(a, units, s);
    auto kern = cache_evict_select_kernel<CACHED, T>;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(units * a.cluster));
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = kSelFixed + (CACHED ? static_cast<uint32_t>((most + 3) / 4 * 16) : 0u);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, kSelMost, allowed);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kern, a);
}

template <int HD>
cudaError_t launch_move(const CacheEvictArgs& a, int64_t units, cudaStream_t s)
{
    auto kern = cache_evict_move_kernel<HD>;
    constexpr int64_t rows = HD == 64 ? 128 : 64;      // of a CTA's round
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(units),
                       static_cast<unsigned>(imax64(1, imin64((a.m + rows - 1) / rows, 152 * 3 / units))));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = kMoveBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, kMoveBytes, allowed);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictArgs& a0, cudaStream_t s)
{
    CacheEvictArgs a = a0;
    const int64_t units = a.c.b * a.c.h_kv;
    if (units == 0) return cudaSuccess;
    if (a.c.cap <= a.keep) {
        // nothing can move: lengths out of range are recorded
        a.cluster = 1;
        return launch_select<false, 512>(a, units, s);
    }
    // CTAs per head: as many as two per SM allow, with 2048 slots each at least (8 heads of 16384 slots: 13.8 us,
    // 18.4 with 1024 at least, 15.3 with 4096; 12 of 16484: 15.8, 18.9, 17.3)
    a.cluster = 1;
    while (a.cluster < 16 && units * a.cluster * 2 <= 304 && a.c.cap / (a.cluster * 2) >= 2048) a.cluster *= 2;
    // Long slices with an SM each get 1024 threads, else two CTAs of 512 share one: slices of 16385 slots (8 heads,
    // clusters of 16) 42 us against 44 to 50, of 32770 (16 heads, 8) 73 against 98, of 4096 19.5 against 20.4, of
    // 2048 16.5 against 15.5.
    const bool wide = units * a.cluster <= 152 && a.c.cap / a.cluster >= kWideSlice;
    const cudaError_t e = wide ? launch_select<true, 1024>(a, units, s) : launch_select<true, 512>(a, units, s);
    if (e != cudaSuccess) return e;
    return a.c.d == 64 ? launch_move<64>(a, units, s) : launch_move<128>(a, units, s);
}

}  // namespace swa
