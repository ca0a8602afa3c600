// cache_weigh.cu -- each cached key's attention weight, summed over given rows
// (sdpa_cache_weigh).
//
// With the rows' LSE known, a key's sum needs no other key: S^T = K Q^T puts
// the keys in the M dimension (128 per tile, a TMEM lane each) and a kv-head's
// rows in N (up to 256 at once), so the thread that owns a lane adds
//   exp2(s_r * scale * log2(e) - LSE_r * log2(e))
// over its lane's columns in registers: one reader and writer per key, no
// atomics, a fixed order. Each group of warps has two accumulators and sums one
// while its other one is computed.
//
// Few rows: bound by reading K once (a 4-stage ring of 128 keys by TMA, 8 at
// d = 64): 55 us at 12 sequences of 16484 keys, 6 kv-heads, 8 rows in bf16,
// d = 128 (5.5 TB/s). Many rows (88 us for 256): by none of its units' rates
// (exponential pipe 29 % busy, tensor pipe 28 %; the exponentials alone would take
// 30 us); its warps wait at barriers first of all, where a key's two threads meet
// behind every tile. The loop over columns exists twice, with and without the
// mask (102 us against 93 with one loop that asked per 32 columns), and is not
// unrolled: both stay within the registers. Weights and positions come into L2
// ahead of their use (93 us against 89).
//
// Roles (640 threads): warp 0 loads K; warp 1 issues the MMAs; warps 4-19 sum,
// and put the rows (Q, LSE, positions) in place, 256 at a time; more rows take
// another round over the part's keys. More than 64 rows: two groups of eight
// warps take every other key tile, two threads a key (64 of an accumulator's
// columns each; with one, 8 warps in all left the SM waiting on latencies: 116
// us against 102 then). Up to 64 rows the second thread would have nothing to
// do, and a tile's chain of waits, not its work, is what a group takes: four
// groups take every fourth tile, a thread a key (16 sequences of 8000 keys, 8
// kv-heads, 8 rows, d = 64: 33 us against 39; 8 rows and d = 128 above: 55
// against 56).
// The key tiles of all (sequence, kv-head) units form one line that the CTAs
// cut evenly. Every wait is bounded (SDPA_ERR_TIMEOUT in the cache's status).
#include <type_traits>

#include "cache_fwd.cuh"

namespace swa {

namespace {

constexpr int kWThreads = 640;
constexpr int kWKeys = 128;
constexpr int kWRows = 256;
constexpr int kWHalf = 128;           // rows of an accumulator
constexpr int kAhead = 6;             // tiles that weights and positions are brought into L2 before their use
constexpr int kWCost = 4;             // a unit's fixed cost in key tiles

template <int HD>
struct WeighCfg {
    static constexpr uint32_t kTile = kWKeys * HD * 2;
    static constexpr uint32_t kBlk = kWKeys * 128;            // a 64-column block of a key tile
    static constexpr uint32_t kQBlk = kWRows * 128;           // and of the rows
    static constexpr int kStages = HD == 128 ? 4 : 8;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = kQ + kWRows * HD * 2;
    static constexpr uint32_t kCst = kK + kStages * kTile;    // float [256]: -LSE * log2(e), -inf for a row that does not count
    static constexpr uint32_t kPos = kCst + kWRows * 4;       // int32 [256]: positions
    static constexpr uint32_t kSum = kPos + kWRows * 4;       // float [2 groups][2 tiles][128]: second threads' sums
    static constexpr uint32_t kBars = kSum + 2048;
    static constexpr uint32_t kMisc = kBars + 384;
    static constexpr uint32_t kBytes = kMisc + 128 + 1024;
    static_assert(kBytes <= 232448, "shared memory above the 227 KB a CTA may opt into");
};

// (accumulators: group * 2 + buffer)
enum WBar : int { wKFull = 0, wKEmpty = 8, wDFull = 16, wDEmpty = 24, wDrain = 32, wNumBars };
static_assert(wNumBars * 8 <= 384, "mbarrier area");

// A chunk of rows and the key tiles [t0, t1) of a segment that it reaches.
__device__ __forceinline__ void reach(int32_t qmin, int32_t qmax, int64_t window, int32_t len, int32_t t0, int32_t t1, int32_t& a,
                                      int32_t& b)
{
    if (qmax < 0) {          // no row counts
        a = b = t0;
        return;
    }
    const int64_t lo = window >= 0 ? imax64(0, qmin - window) : 0;
    const int64_t hi = imin64(qmax, static_cast<int64_t>(len) - 1);
    a = static_cast<int32_t>(imax64(t0, lo / kWKeys));
    b = static_cast<int32_t>(imin64(t1, hi / kWKeys + 1));
    if (b < a) b = a;
}

}  // namespace

// FEW: up to 64 rows; four groups of warps take every fourth key tile each, a
// thread a key, two accumulators of 64 columns each.
template <int HD, bool BF16, bool FEW>
__global__ void __launch_bounds__(kWThreads, 1) cache_weigh_kernel(const __grid_constant__ CacheWeighArgs a)
{
    using C = WeighCfg<HD>;
    constexpr int NS = C::kStages;
    constexpr uint32_t NG = FEW ? 4 : 2;               // groups
    constexpr uint32_t AC = FEW ? 64 : kWHalf;         // columns of an accumulator
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ int64_t sh_sum[kWThreads / 32], sh_at[2];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(sm);
    auto bar = [&](int i) -> uint32_t { return sbase + C::kBars + 8u * i; };
    // [0] tmem base, [1] abort flag, [2] chunks begun, [3] smallest and [4] largest position of the chunk's rows,
    // [5], [6] chunks whose positions warps 0, 1 have read
    uint32_t* misc = reinterpret_cast<uint32_t*>(sm + C::kMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t tmo = static_cast<uint64_t>(a.timeout_ns);

    const int R = a.s_q * a.group;
    const int chunks = (R + kWRows - 1) / kWRows;
    auto tiles_of = [&](int64_t i) -> int32_t {
        bool bad;
        return (cache_length(a.c, i, bad) + kWKeys - 1) / kWKeys;
    };
    // (a sequence without keys keeps its units' cost, so that every sequence has a place in the line)
    const Part part = find_part<kWThreads>(a.c.b, [&](int64_t i) { return (tiles_of(i) + kWCost) * a.c.h_kv; }, sh_sum, sh_at);
    if (part.end == 0) return;

    if (tid == 0) {
        misc[1] = misc[2] = misc[5] = misc[6] = 0;
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar(wKFull + i), 1);
            mbar_init(bar(wKEmpty + i), 1);
        }
        for (uint32_t i = 0; i < 2 * NG; ++i) {
            mbar_init(bar(wDFull + i), 1);
            mbar_init(bar(wDEmpty + i), FEW ? 4 : 8);      // a warp each
        }
        mbar_init(bar(wDrain), 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(sbase + C::kMisc, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    volatile uint32_t* abort_flag = misc + 1;
    volatile int32_t* qrange = reinterpret_cast<volatile int32_t*>(misc + 3);

    auto give_up = [&]() -> bool {
        *abort_flag = 1;
        set_status(a.c.status, SDPA_ERR_TIMEOUT);
        return false;
    };
    auto wait = [&](int b, uint32_t parity) -> bool {
        if (mbar_try_wait(bar(b), parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait(bar(b), parity, tmo)) return true;
        return give_up();
    };
    // until n chunks of rows are in place (word 2; 5, 6: have been seen)
    auto wait_count = [&](uint32_t n, int word = 2) -> bool {
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            uint32_t x;
            asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(x) : "r"(sbase + C::kMisc + 4 * word) : "memory");
            if (x >= n) return true;
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > tmo) return give_up();
        }
    };
    auto put_count = [&](int word, uint32_t n) {
        asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(sbase + C::kMisc + 4 * word), "r"(n) : "memory");
    };
    auto seen = [&](int who, uint32_t n) { put_count(5 + who, n); };
    // Keys that a chunk cannot reach are left out where slots are positions and the rows may be far from some keys.
    const bool skips = a.c.positions == nullptr && (a.window_left >= 0 || chunks > 1);

    // Walks the part: f(sequence, kv-head, its keys, first key tile, number of key tiles) until it returns false.
    auto walk = [&](auto f) {
        int64_t at = part.at, bi = part.bi, rem = part.rem;
        while (at < part.end) {
            bool bad;
            const int32_t len = cache_length(a.c, bi, bad), tiles = (len + kWKeys - 1) / kWKeys;
            const Segment g = segment_at(rem, tiles, kWCost, part.end - at);
            if (g.n > 0 && !f(bi, g.un, len, g.tile0, g.n)) return;
            at += g.line_n;
            rem += g.line_n;
            if (rem == (static_cast<int64_t>(tiles) + kWCost) * a.c.h_kv) {
                ++bi;
                rem = 0;
            }
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------------ K
        uint32_t it = 0, cnt = 0;
        bool ok = true;
        walk([&](int64_t bi, int64_t gk, int32_t len, int32_t tile0, int32_t n) -> bool {
            auto entry_of = [&](int32_t j) -> int32_t {
                if (a.c.page_table == nullptr) return static_cast<int32_t>(bi);
                return cache_entry(a.c, bi, j);
            };
            auto row_of = [&](int32_t j) -> uint32_t {
                return a.c.page_table == nullptr ? j : cache_row(a.c, j);
            };
            const int boxes = a.box_rows ? kWKeys / a.box_rows : 0;
            for (int ch = 0; ch < chunks && ok; ++ch) {
                int32_t ta = tile0, tb = tile0 + n;
                ++cnt;
                if (skips) {
                    if (!(ok = __all_sync(0xffffffffu, wait_count(cnt)))) break;
                    reach(qrange[0], qrange[1], a.window_left, len, tile0, tile0 + n, ta, tb);
                    __syncwarp();
                    if (lane == 0) seen(0, cnt);
                }
                auto box_entry = [&](int32_t t) -> int32_t {
                    const int32_t j = t * kWKeys + lane * a.box_rows;
                    return lane < boxes && t < tb && j < len ? entry_of(j) : -1;
                };
                int32_t entry = box_entry(ta);
                for (int32_t t = ta; t < tb; ++t, ++it) {
                    const uint32_t st = it % NS;
                    const uint32_t stage = sbase + C::kK + st * C::kTile;
                    const int32_t mine = entry;
                    entry = box_entry(t + 1);
                    if (!(ok = __all_sync(0xffffffffu, wait(wKEmpty + st, ((it / NS) & 1) ^ 1)))) break;
                    const int32_t j0 = t * kWKeys;
                    if (boxes > 0) {
                        // boxes without a key, or on a page out of range, stay as they were: their lanes are not used
                        const bool good = mine >= 0 && mine < a.c.n_pages;
                        if (lane < boxes && j0 + lane * a.box_rows < len && !good) set_status(a.c.status, SDPA_ERR_BOUNDS);
                        const uint32_t have = __popc(__ballot_sync(0xffffffffu, good));
                        if (lane == 0) mbar_arrive_expect_tx(bar(wKFull + st), have * a.box_rows * HD * 2);
                        __syncwarp();
                        if (good) {
                            const int row = static_cast<int>(row_of(j0 + lane * a.box_rows));
#pragma unroll
                            for (int cb = 0; cb < HD / 64; ++cb)
                                tma_box(stage + cb * C::kBlk + lane * a.box_rows * 128, &a.tm_k, bar(wKFull + st), cb * 64,
                                        static_cast<int>(gk), row, mine);
                        }
                        continue;
                    }
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const int32_t j = j0 + k * 32 + lane;
                        const uint16_t* p = a.c.k;
                        bool have = j < len;
                        if (have) {
                            const int32_t page = entry_of(j);
                            have = page >= 0 && page < a.c.n_pages;
                            if (!have) set_status(a.c.status, SDPA_ERR_BOUNDS);
                            else p += page * a.c.k_stride[0] + row_of(j) * a.c.k_stride[1] + gk * a.c.k_stride[2];
                        }
                        const uint32_t held = __ballot_sync(0xffffffffu, have);
                        constexpr int CPR = HD / 8, RPI = 32 / CPR;
#pragma unroll 8
                        for (int i = 0; i < 32 / RPI; ++i) {
                            const int r = i * RPI + lane / CPR, c = lane % CPR;
                            const uint64_t q = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(p), r);
                            cp16(stage + swizzled<C::kBlk>(k * 32 + r, c), reinterpret_cast<const uint16_t*>(q) + c * 8,
                                 (held >> r) & 1);
                        }
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(wKFull + st));
                }
            }
            return ok && !a.c.stall;        // (test hook: no second stretch of keys comes)
        });
        // copies in flight end before the CTA does
        for (uint32_t k = 0; k < NS && k < it; ++k) {
            const uint32_t r = it - 1 - k;
            mbar_wait(bar(wKFull + r % NS), (r / NS) & 1, tmo);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        if (elect_one()) {
            uint32_t it = 0, cnt = 0, made0 = 0, made1 = 0;    // accumulators of each group so far
            bool ok = true;
            const uint64_t dk0 = sdesc_sw128(sbase + C::kK, 16, 1024);
            const uint64_t dq0 = sdesc_sw128(sbase + C::kQ, 16, 1024);
            walk([&](int64_t, int64_t, int32_t len, int32_t tile0, int32_t n) -> bool {
                for (int ch = 0; ch < chunks && ok; ++ch) {
                    if (!(ok = wait_count(++cnt))) break;
                    int32_t ta = tile0, tb = tile0 + n;
                    if (skips) {
                        reach(qrange[0], qrange[1], a.window_left, len, tile0, tile0 + n, ta, tb);
                        seen(1, cnt);
                    }
                    const int rows = (min(kWRows, R - ch * kWRows) + 31) & ~31;
                    for (int32_t t = ta; t < tb && ok; ++t, ++it) {
                        const uint32_t st = it % NS, grp = it % NG;
                        if (!(ok = wait(wKFull + st, (it / NS) & 1))) break;
                        const uint64_t dk = sdesc_at(dk0, st * C::kTile);
                        for (int r0 = 0; r0 < rows; r0 += kWHalf) {
                            const uint32_t m = FEW ? it / NG : grp ? made1++ : made0++, b = grp * 2 + (m & 1);
                            if (!(ok = wait(wDEmpty + b, ((m >> 1) & 1) ^ 1))) break;
                            tc_fence_after();
                            const uint32_t idesc = idesc_f16(BF16, 128, 0, false, false) |
                                                   static_cast<uint32_t>(min(kWHalf, rows - r0) >> 3) << 17;
                            const uint64_t dq = sdesc_at(dq0, r0 * 128);
#pragma unroll
                            for (int k = 0; k < HD / 16; ++k)
                                mma_ss(tmem + b * AC, sdesc_at(dk, (k >> 2) * C::kBlk + (k & 3) * 32),
                                       sdesc_at(dq, (k >> 2) * C::kQBlk + (k & 3) * 32), idesc, k > 0);
                            mma_commit(bar(wDFull + b));
                        }
                        mma_commit(bar(wKEmpty + st));
                    }
                }
                return ok;
            });
            // MMAs in flight end before TMEM is freed
            mma_commit(bar(wDrain));
            mbar_wait(bar(wDrain), 0, tmo);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ rows, sums
        const int grp = (warp - 4) >> (FEW ? 2 : 3), second = FEW ? 0 : ((warp - 4) >> 2) & 1;
        const int et = tid - 128;                           // the first 256: a row each
        const int key_lane = ((warp & 3) << 5) + lane;      // key of the tile
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float* cst = reinterpret_cast<const float*>(sm + C::kCst);
        const int32_t* qpos = reinterpret_cast<const int32_t*>(sm + C::kPos);
        uint32_t it = 0, cnt = 0, taken = 0, tile_par = 0;  // taken: this group's accumulators
        bool ok = true;
        // widest distance of a key behind a row
        const uint32_t wide = a.window_left < 0 || a.window_left > INT32_MAX ? INT32_MAX : static_cast<uint32_t>(a.window_left);
        const uint64_t scale2 = pair(__float_as_uint(a.scale_log2), __float_as_uint(a.scale_log2));
        walk([&](int64_t bi, int64_t gk, int32_t len, int32_t tile0, int32_t n) -> bool {
            const int64_t npos = a.c.next_pos ? a.c.next_pos[bi] : len;
            const int64_t unit = (bi * a.c.h_kv + gk) * a.c.cap;
            for (int ch = 0; ch < chunks; ++ch) {
                named_sync(3, 512);         // both groups are done with the last chunk's rows
                const int r = ch * kWRows + et;
                const int rows = (min(kWRows, R - ch * kWRows) + 31) & ~31;
                if (et < kWRows) {
                    int64_t p = -1;
                    float c = -INFINITY;
                    const int tok = r < R ? r / a.group : 0;
                    const int64_t h = gk * a.group + (r - tok * a.group);
                    if (r < R) {
                        p = a.q_pos ? a.q_pos[bi * a.s_q + tok] : npos - a.s_q + tok;
                        const float z = a.lse[(bi * a.h_q + h) * a.s_q + tok];
                        if (p >= 0 && fabsf(z) < INFINITY) c = -z * kLog2e;
                    }
                    const bool live = c != -INFINITY;
                    const int32_t pos = live ? static_cast<int32_t>(imin64(p, INT32_MAX)) : -1;
                    reinterpret_cast<float*>(sm + C::kCst)[et] = c;
                    reinterpret_cast<int32_t*>(sm + C::kPos)[et] = pos;
                    if (et < rows) {
                        const uint16_t* qp = a.q + bi * a.q_stride[0] + tok * a.q_stride[1] + h * a.q_stride[2];
#pragma unroll
                        for (int k = 0; k < HD / 8; ++k) {
                            const uint4 x = live ? ld_nc_v4(qp + k * 8) : make_uint4(0u, 0u, 0u, 0u);
                            *reinterpret_cast<uint4*>(sm + C::kQ + swizzled<C::kQBlk>(et, k)) = x;
                        }
                    }
                    fence_proxy_async_smem();
                }
                named_sync(3, 512);
                // smallest and largest position of the rows that count (each group's warps alike)
                int32_t lo = INT32_MAX, hi = -1;
                for (int i = lane; i < rows; i += 32) {
                    const int32_t p = qpos[i];
                    if (p >= 0) lo = min(lo, p);
                    hi = max(hi, p);
                }
                lo = __reduce_min_sync(0xffffffffu, lo);
                hi = __reduce_max_sync(0xffffffffu, hi);
                ++cnt;
                if (et == 0) {
                    // a chunk without tiles is over at once: its positions stay until both readers have seen them
                    if (skips) ok = ok && wait_count(cnt - 1, 5) && wait_count(cnt - 1, 6);
                    qrange[0] = lo;
                    qrange[1] = hi;
                    put_count(2, cnt);
                }
                int32_t ta = tile0, tb = tile0 + n;
                if (skips) reach(lo, hi, a.window_left, len, tile0, tile0 + n, ta, tb);
                // this thread's key of a tile: its page entry, position and weight are loaded a tile of the group ahead
                struct Mine {
                    int32_t entry, pos;
                    float w;
                };
                auto fetch = [&](int32_t t) -> Mine {
                    Mine k{static_cast<int32_t>(bi), 0, 0.f};
                    const int32_t j = t * kWKeys + key_lane;
                    if (t < tb && j < len) {
                        if (a.c.page_table) k.entry = cache_entry(a.c, bi, j);
                        k.pos = a.c.positions ? a.c.positions[unit + j] : j;
                        k.w = a.c.weights[unit + j];
                        // (a group's tile takes less than memory's latency: later ones come into L2 before)
                        const int32_t later = j + kAhead * kWKeys;
                        if (later < len) {
                            if (!second) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.c.weights + unit + later));
                            if ((FEW || second) && a.c.positions) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.c.positions + unit + later));
                        }
                    }
                    return k;
                };
                const int32_t mine0 = ta + static_cast<int32_t>((grp - it) % NG);   // the group's first tile
                Mine next = fetch(mine0);
                for (int32_t t = ta; t < tb; ++t, ++it) {
                    if (it % NG != static_cast<uint32_t>(grp)) continue;
                    const Mine me = next;
                    next = fetch(t + NG);
                    const int32_t j = t * kWKeys + key_lane;
                    const bool held = j < len && me.entry >= 0 && me.entry < a.c.n_pages;
                    const int32_t kp = held ? me.pos : 0;
                    // does every row that counts admit every key of the warp, or none any?
                    const bool plain = __all_sync(0xffffffffu, !held || (kp <= lo && static_cast<uint32_t>(hi - kp) <= wide));
                    const bool none = __all_sync(0xffffffffu, !held || kp > hi || (kp < lo && static_cast<uint32_t>(lo - kp) > wide));
                    uint64_t s2[4] = {0u, 0u, 0u, 0u};
                    for (int r0 = 0; r0 < rows; r0 += kWHalf) {
                        const uint32_t b = grp * 2 + (taken & 1);
                        ok = ok && wait(wDFull + b, (taken >> 1) & 1);
                        ++taken;
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) continue;
                        tc_fence_after();
                        const uint32_t td = tmem + b * AC + lane_off;
                        const int n32 = min(kWHalf, rows - r0);
                        // this thread's columns, 32 at a time
                        const int c1 = min(n32, 64 * (second + 1));
                        auto columns = [&](auto masked) {
                            constexpr bool M = decltype(masked)::value;
#pragma unroll 1
                            for (int cb = 64 * second; cb < c1; cb += 32) {
                                uint32_t x[32];
                                tmem_ld32(td + cb, x);
                                tmem_ld_wait();
                                loaded(x);
#pragma unroll
                                for (int e = 0; e < 32; e += 4) {
                                    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(cst + r0 + cb + e);
                                    const uint64_t y0 = fma2(pair(x[e], x[e + 1]), scale2, c.x);
                                    const uint64_t y1 = fma2(pair(x[e + 2], x[e + 3]), scale2, c.y);
                                    float p0 = ex2_approx(lo_of(y0)), p1 = ex2_approx(hi_of(y0));
                                    float p2 = ex2_approx(lo_of(y1)), p3 = ex2_approx(hi_of(y1));
                                    if constexpr (M) {
                                        // (a row that does not count is at -1: below every key)
                                        const int4 at = *reinterpret_cast<const int4*>(qpos + r0 + cb + e);
                                        p0 = static_cast<uint32_t>(at.x - kp) > wide ? 0.f : p0;
                                        p1 = static_cast<uint32_t>(at.y - kp) > wide ? 0.f : p1;
                                        p2 = static_cast<uint32_t>(at.z - kp) > wide ? 0.f : p2;
                                        p3 = static_cast<uint32_t>(at.w - kp) > wide ? 0.f : p3;
                                    }
                                    uint64_t& sa = s2[(e >> 1) & 2];
                                    uint64_t& sb = s2[((e >> 1) & 2) + 1];
                                    sa = add2(sa, pair(__float_as_uint(p0), __float_as_uint(p1)));
                                    sb = add2(sb, pair(__float_as_uint(p2), __float_as_uint(p3)));
                                }
                            }
                        };
                        if (plain) columns(std::false_type{});
                        else if (!none) columns(std::true_type{});
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(wDEmpty + b));
                    }
                    const uint64_t sum2 = add2(add2(s2[0], s2[1]), add2(s2[2], s2[3]));
                    float sum = lo_of(sum2) + hi_of(sum2);
                    if constexpr (FEW) {
                        if (held && ok) a.c.weights[unit + j] = me.w + sum;
                    } else {
                        // the key's two threads: the second hands its sum to the first
                        float* slot = reinterpret_cast<float*>(sm + C::kSum) + (grp * 2 + (tile_par & 1)) * kWKeys + key_lane;
                        tile_par ^= 1;
                        if (second) *slot = sum;
                        named_sync(4 + grp * 4 + (warp & 3), 64);
                        if (!second && held && ok) a.c.weights[unit + j] = me.w + (sum + *slot);
                    }
                }
            }
            return true;
        });
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

namespace {

template <int HD, bool BF16, bool FEW>
cudaError_t launch_typed(const CacheWeighArgs& a, cudaStream_t s)
{
    auto kern = cache_weigh_kernel<HD, BF16, FEW>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, WeighCfg<HD>::kBytes, allowed);
    if (e != cudaSuccess) return e;
    kern<<<a.parts, kWThreads, WeighCfg<HD>::kBytes, s>>>(a);
    return cudaGetLastError();
}

template <int HD, bool BF16>
cudaError_t launch_rows(const CacheWeighArgs& a, cudaStream_t s)
{
    return static_cast<int64_t>(a.s_q) * a.group <= 64 ? launch_typed<HD, BF16, true>(a, s) : launch_typed<HD, BF16, false>(a, s);
}

}  // namespace

cudaError_t launch_cache_weigh(const CacheWeighArgs& a, int dtype, cudaStream_t s)
{
    if (a.c.d == 128) return dtype == SDPA_BF16 ? launch_rows<128, true>(a, s) : launch_rows<128, false>(a, s);
    return dtype == SDPA_BF16 ? launch_rows<64, true>(a, s) : launch_rows<64, false>(a, s);
}

}  // namespace swa
