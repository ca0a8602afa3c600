// cache_tile.cu -- the cache forward for many rows per kv-head: tcgen05 tiles.
//
// A unit is a kv-head's block of up to 256 rows. Rows are the M dimension (128
// per tile), keys the N dimension of S = Q K^T and the K dimension of O += P V:
//   S  [128 rows x 64 keys]  TMEM, two buffers for each of two slots
//   P  16-bit, written over its S's columns, the A operand of P V from TMEM
//   O  [128 rows x d]        TMEM, one for each slot
// A slot's next S is computed while its softmax works on this one, and the two
// slots keep the tensor core and the softmax warps busy in turn. With more than
// 128 rows the slots are the unit's two row tiles and share each K/V tile; with
// fewer they take the same rows and every other key tile, and their sums are
// joined at the end. So K and V are read once per 256 rows, and a short row
// block loses no overlap.
//
// Bound by reading K and V up to 128 rows (12 sequences of 16484 keys, 6
// kv-heads, d = 128: 112 us at 128 rows, 5.4 TB/s), then by the softmax groups'
// chain from a tile's S to its P (256 rows 138 us; 512, each half reading K and V
// again, 247 us, 1.26 PFLOP/s): its phases wait on the tensor memory's loads and
// the exponentials in turn, with the tensor core a third of the time idle. Two
// threads a row and 640 threads did not shorten it (256 rows: 161 us against 147
// then), and splitting P as the rows kernel does costs the kernel 3 % at 24 to 128
// rows of even lengths, 11 % of ragged ones, and 16 to 19 % above (512 rows: 283
// us against 238).
//
// Roles (384 threads): warp 0 loads K, warp 1 V into two rings in the 128-byte
// swizzle; warps 2 and 3 issue a slot's MMAs each (one warp for both was the
// bottleneck: its issue of a tile's 12 MMAs takes longer than they run);
// warps 4-7 and 8-11 are the slots' softmax groups, one row per thread. A row's
// reference moves only when a score exceeds it by 2^8 (f16: by 2^15, and then
// lies 2^7 below it, see kBelow), so O is seldom rescaled.
// P is rounded to the I/O dtype, as the prompt's forward does: half a step of a
// P next to a sum that stays in fp32, which leaves O's error within 1.4 times
// that of rounding O alone.
//
// The steps of all units form one line that the persistent CTAs cut evenly, as
// in cache_fwd.cu; partials of cut units go to the same join.
// Every wait is bounded; one that runs out ends the kernel with
// SDPA_ERR_TIMEOUT in the cache's status.
#include <type_traits>

#include "cache_fwd.cuh"

namespace swa {

namespace {

constexpr int kTileThreads = 384;
constexpr int kMmaWarp = 2;            // and 3
constexpr int kSoftWarp0 = 4;
constexpr int kKeys = 64;              // keys of a tile
constexpr uint32_t kQBlk = 128 * 128;  // one 64-column block of a 128-row 16-bit tile
constexpr uint32_t kBlk = kKeys * 128; // the same of a key tile
constexpr int kRing = 16;              // key tiles whose validity and positions are kept

template <int HD>
struct TileCfg {
    static constexpr uint32_t kQTile = 128 * HD * 2;
    static constexpr uint32_t kTile = kKeys * HD * 2;
    static constexpr int kStages = HD == 128 ? 4 : 8;
    static constexpr uint32_t kQ = 0;                           // 2 slots
    static constexpr uint32_t kK = kQ + 2 * kQTile;
    static constexpr uint32_t kV = kK + kStages * kTile;
    static constexpr uint32_t kPos = kV + kStages * kTile;      // int32 [kRing][64]
    static constexpr uint32_t kOk = kPos + kRing * 256;         // uint32 [kRing][2]
    static constexpr uint32_t kMask = kOk + kRing * 8;          // uint64 [64]
    static constexpr uint32_t kMl = kMask + 512;                // float2 [2][128]
    static constexpr uint32_t kBars = kMl + 2048;
    static constexpr uint32_t kMisc = kBars + 448;
    static constexpr uint32_t kBytes = kMisc + 256 + 1024;
    static_assert(kBytes <= 232448, "shared memory above the 227 KB a CTA may opt into");
};

// mbarriers; per-stage and per-slot ones at index + stage or slot (S, P and
// P V: slot * 2 + buffer)
enum TBar : int { tKFull = 0, tKEmpty = 8, tVFull = 16, tVEmpty = 24, tSFull = 32, tPFull = 36, tPvDone = 40, tDrain = 44,
                  tNumBars = 46 };
static_assert(tNumBars * 8 <= 448, "mbarrier area");

template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How a sequence's steps are laid out: per kv-head `na` blocks of 256 rows
// with two row tiles (a step is one key tile), then perhaps one block with one
// row tile (a step is two key tiles), each with its fixed cost before it (by its
// row tiles: Q in, O out).
struct Shape {
    int32_t ta, tb;       // steps of a two-tile block, of a one-tile block
    int64_t per_head;
};

__device__ __forceinline__ Shape shape_of(const SeqView& v, int na, int nb, int32_t cost)
{
    Shape s;
    s.ta = v.tiles;
    s.tb = (v.tiles + 1) >> 1;
    s.per_head = static_cast<int64_t>(na) * (s.ta + 2 * cost) + static_cast<int64_t>(nb) * (s.tb + cost);
    return s;
}

// One stretch of a CTA's part that lies in one unit.
struct Seg {
    int64_t bi, gk;
    int32_t blk;          // row block
    bool two;             // two row tiles
    int32_t step0, steps, of, line_n, cost;   // its steps, how many the unit has, its places in the line, the unit's cost
};

struct Walk {
    int64_t at, end, bi, rem;
    int na, nb;
    SeqView sv;
    Shape sh;
    bool loaded;

    // The next segment with steps; false at the part's end.
    __device__ __forceinline__ bool next(const CacheFwdArgs& a, Seg& g)
    {
        if (at >= end) return false;
        if (!loaded) {
            sv = seq_view(a, bi, kKeys, kKeys);
            sh = shape_of(sv, na, nb, a.unit_cost);
            loaded = true;
        }
        g.bi = bi;
        g.gk = rem / sh.per_head;
        const int64_t r = rem - g.gk * sh.per_head;
        const int64_t a_line = static_cast<int64_t>(na) * (sh.ta + 2 * a.unit_cost);
        g.two = r < a_line;
        g.of = g.two ? sh.ta : sh.tb;
        g.cost = g.two ? 2 * a.unit_cost : a.unit_cost;
        const Segment s = segment_at(g.two ? r : r - a_line, g.of, g.cost, end - at);
        g.blk = g.two ? static_cast<int32_t>(s.un) : na;
        g.step0 = s.tile0;
        g.steps = s.n;
        g.line_n = s.line_n;
        return s.n > 0;       // a part that ends before a unit's first step has no more
    }
    __device__ __forceinline__ void advance(const CacheFwdArgs& a, const Seg& g)
    {
        at += g.line_n;
        rem += g.line_n;
        if (rem == sh.per_head * a.c.h_kv) {
            ++bi;
            rem = 0;
            loaded = false;
        }
    }
};

// Key tiles of a segment: one for each step with two row tiles, two with one
// (the unit's last step may have only one).
__device__ __forceinline__ int32_t seg_tile0(const Seg& g) { return g.two ? g.step0 : 2 * g.step0; }
__device__ __forceinline__ int32_t seg_tiles(const Seg& g, int32_t tiles)
{
    return g.two ? g.steps : min(2 * (g.step0 + g.steps), tiles) - 2 * g.step0;
}
}  // namespace

// POS: a window over keys that have positions. An instance of its own: the
// checks of positions lengthen the loaders' way to a tile (12 sequences of 16484
// keys, 6 kv-heads, 296 rows: 255 us with one instance for both, 223 without the
// checks; d = 64 230 and 193; 16 to 512 rows of one kind of block 1 to 2 %. It is
// the pace, not the reads: 223 and 217 MB from DRAM for 3 of the sequences).
template <int HD, bool BF16, bool POS>
__global__ void __launch_bounds__(kTileThreads, 1) cache_fwd_tile_kernel(const __grid_constant__ CacheTileArgs ta)
{
    const CacheFwdArgs& a = ta.f;
    using C = TileCfg<HD>;
    constexpr int NS = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ int64_t sh_sum[kTileThreads / 32], sh_at[2];
    // the swizzle needs 1024-byte boundaries (kBytes has the slack)
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(sm);
    auto bar = [&](int i) -> uint32_t { return sbase + C::kBars + 8u * i; };
    // [0] tmem base, [1] abort flag, [2] segments begun, [16] on: the masks' numbers of bits, a byte each
    uint32_t* misc = reinterpret_cast<uint32_t*>(sm + C::kMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t tmo = static_cast<uint64_t>(a.timeout_ns);

    const int R = a.s_q * a.group;
    const int blocks = (R + 255) / 256;
    const int nb = (R - 1) % 256 < 128 ? 1 : 0;   // the last block has one row tile
    const int na = blocks - nb;
    Walk walk{};
    walk.na = na;
    walk.nb = nb;
    Part part{1, 0, 0, 0, 0, Line{0}};
    if (a.whole) {
        const int64_t units = a.c.h_kv * blocks;
        part.bi = blockIdx.x / units;
        const int64_t un = blockIdx.x - part.bi * units, gk = un / blocks, blk = un - gk * blocks;
        const Shape s = shape_of(seq_view(a, part.bi, kKeys, kKeys), na, nb, a.unit_cost);
        part.rem = gk * s.per_head + blk * (s.ta + 2 * a.unit_cost) + (blk < na ? 2 : 1) * a.unit_cost;
        part.end = blk < na ? s.ta : s.tb;
    } else {
        part = find_part<kTileThreads>(
            a.c.b, [&](int64_t i) { return a.c.h_kv * shape_of(seq_view(a, i, kKeys, kKeys), na, nb, a.unit_cost).per_head; }, sh_sum, sh_at);
        if (tid == 0 && !a.cut_by_unit) a.cuts[blockIdx.x].bi = -1;
        if (part.end == 0) {
            grid_dep_launch();
            return;
        }
    }
    walk.at = part.at;
    walk.end = part.end;
    walk.bi = part.bi;
    walk.rem = part.rem;

    if (tid == 0) {
        misc[1] = misc[2] = 0;
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar(tKFull + i), 2);
            mbar_init(bar(tKEmpty + i), 2);
            mbar_init(bar(tVFull + i), 2);
            mbar_init(bar(tVEmpty + i), 2);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar(tSFull + s), 2);    // the MMAs' commit, and the issuer's own arrival
            mbar_init(bar(tPFull + s), 4);        // a warp each
            mbar_init(bar(tPvDone + s), 1);
        }
        mbar_init(bar(tDrain), 1);
        mbar_init(bar(tDrain + 1), 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(sbase + C::kMisc, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const uint32_t tm_s0 = tmem, tm_o0 = tmem + 256;     // slot s: S at + 128 s, O at + HD s
    volatile uint32_t* abort_flag = misc + 1;

    auto wait = [&](int b, uint32_t parity) -> bool {
        if (mbar_try_wait(bar(b), parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait(bar(b), parity, tmo)) return true;
        *abort_flag = 1;
        set_status(a.c.status, SDPA_ERR_TIMEOUT);
        return false;
    };
    // until the softmax groups have begun n segments
    auto wait_count = [&](uint32_t n) -> bool {
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            uint32_t x;
            asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(x) : "r"(sbase + C::kMisc + 8) : "memory");
            if (x >= n) return true;
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > tmo) {
                *abort_flag = 1;
                set_status(a.c.status, SDPA_ERR_TIMEOUT);
                return false;
            }
        }
    };
    auto wait_warp = [&](int b, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(b, parity)); };

    if (warp < kMmaWarp) {
        // ------------------------------------------------------------ gather K and V
        // Warp 0 fills the K ring, warp 1 the V ring, each as its stages become
        // free. A tile whose keys are all cached comes by TMA, in boxes that
        // lie within a page (box_rows, a power of two that divides the page size);
        // the last tiles of a unit, and all of them where pages have no such
        // divisor, are gathered 16 bytes at a time, 32 keys a group, zeros in the
        // rows that are not held. A gathered group is handed over (writes made
        // visible to the async proxy, barrier) when LAG later ones are on their
        // way, or while the warp has to wait for a stage. A stage is full after
        // two arrivals, one for each 32 keys.
        const bool is_v = warp == 1;
        constexpr int CPR = HD / 8;           // 16-byte chunks of a row
        constexpr int RPI = 32 / CPR;         // rows that a warp copies at once
        constexpr uint32_t LAG = 5;
        uint64_t queue = 0;                   // stages of the groups on their way, 8 bits each, oldest lowest
        uint32_t pending = 0;
        uint32_t it = 0;                      // key tiles so far
        bool ok = is_v || !a.c.stall;         // (test hook: no K comes)
        const int full0 = is_v ? tVFull : tKFull, empty0 = is_v ? tVEmpty : tKEmpty;
        const uint32_t ring0 = sbase + (is_v ? C::kV : C::kK);
        auto hand_over = [&](uint32_t keep) {     // the groups that are there, all but the last `keep`
            fence_proxy_async_smem();
            __syncwarp();
            for (; pending > keep; --pending, queue >>= 8)
                if (lane == 0) mbar_arrive(bar(full0 + static_cast<int>(queue & 255)));
        };
        auto wait_oldest = [&]() {
            switch (pending) {
                case 6: cp_wait<5>(); break;
                case 5: cp_wait<4>(); break;
                case 4: cp_wait<3>(); break;
                case 3: cp_wait<2>(); break;
                case 2: cp_wait<1>(); break;
                default: cp_wait<0>(); break;
            }
            hand_over(pending > 6 ? 0 : pending - 1);
        };
        auto acquire = [&](int b, uint32_t parity) -> bool {
            for (;;) {
                if (__all_sync(0xffffffffu, mbar_test(bar(b), parity))) return true;
                if (pending == 0) return wait_warp(b, parity);
                wait_oldest();
            }
        };
        const int c = lane % CPR, sub = lane / CPR;
        Seg g;
        while (ok && walk.next(a, g)) {
            const SeqView& sv = walk.sv;
            const int32_t* kpos = POS ? a.c.positions + (g.bi * a.c.h_kv + g.gk) * a.c.cap : nullptr;
            const int32_t t0 = seg_tile0(g), t1 = t0 + seg_tiles(g, sv.tiles) - 1;
            const uint16_t* pool = (is_v ? a.c.v : a.c.k) + g.gk * (is_v ? a.c.v_stride[2] : a.c.k_stride[2]);
            const int64_t st_page = is_v ? a.c.v_stride[0] : a.c.k_stride[0], st_row = is_v ? a.c.v_stride[1] : a.c.k_stride[1];
            const uint16_t* fresh = (is_v ? a.v + g.bi * a.v_stride[0] + g.gk * a.v_stride[2]
                                          : a.k + g.bi * a.k_stride[0] + g.gk * a.k_stride[2]);
            const int64_t st_new = is_v ? a.v_stride[1] : a.k_stride[1];
            auto entry_of = [&](int32_t j) -> int32_t {       // of a held key
                if (a.c.page_table == nullptr) return static_cast<int32_t>(g.bi);
                return cache_entry(a.c, g.bi, j);
            };
            auto row_of = [&](int32_t j) -> uint32_t {
                return a.c.page_table == nullptr ? j : cache_row(a.c, j);
            };
            // new tokens that some row admits: padding may be anything, and would meet a P of 0
            uint32_t used[2] = {0u, 0u};
            int32_t shallow = 64;                 // least bits of a mask whose row admits a key
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                int bits;
                const uint64_t m = admitted_tokens(a, g.bi, sv.nq, w * 32 + lane, bits);
                if (m) shallow = min(shallow, bits);
                used[0] |= __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(m));
                used[1] |= __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(m >> 32));
            }
            // lowest position in any row's window, and without positions the first slot there
            int32_t low = INT32_MIN;
            if (a.window_left >= 0) {
                const int64_t npos = a.c.next_pos ? a.c.next_pos[g.bi] : sv.len;
                low = static_cast<int32_t>(imax64(INT32_MIN, imin64(INT32_MAX,
                    npos + static_cast<int32_t>(__reduce_min_sync(0xffffffffu, shallow)) - 1 - a.window_left)));
            }
            const int32_t first = POS ? 0 : max(sv.first, low);
            const int boxes = ta.box_rows ? kKeys / ta.box_rows : 0;
            // a TMA tile's page of lane's box, a tile ahead
            auto box_entry = [&](int32_t t) -> int32_t {
                const int32_t j = sv.lo + t * kKeys + lane * ta.box_rows;
                return lane < boxes && t <= t1 && j >= first && j < sv.len ? entry_of(j) : 0;
            };
            int32_t entry = box_entry(t0);
            for (int32_t t = t0; t <= t1; ++t, ++it) {
                const uint32_t st = it % NS, par = (it / NS) & 1;
                const int32_t x0 = t * kKeys, j0 = sv.lo + x0;
                const int32_t mine = entry;
                entry = box_entry(t + 1);
                // the positions of the lane's keys (the K warp puts them down for the softmax)
                int32_t pos[2] = {INT32_MAX, INT32_MAX};
                if constexpr (POS) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int32_t j = j0 + k * 32 + lane;
                        pos[k] = j < sv.len ? kpos[j] : j;
                    }
                }
                // (a V that no row's window has may be anything, and would meet a P of 0)
                const bool good = (lane >= boxes || (mine >= 0 && mine < a.c.n_pages)) &&
                                  (!POS || !is_v || (pos[0] >= low && pos[1] >= low));
                const bool by_tma = boxes > 0 && j0 >= first && x0 + kKeys <= sv.new0 && j0 + kKeys <= sv.len &&
                                    __all_sync(0xffffffffu, good);
                if (!(ok = acquire(empty0 + st, par ^ 1))) break;
                const uint32_t stage = ring0 + st * C::kTile;
                if (!is_v && a.window_left >= 0) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        reinterpret_cast<int32_t*>(sm + C::kPos)[(it % kRing) * kKeys + k * 32 + lane] =
                            POS ? pos[k] : j0 + k * 32 + lane;
                    }
                }
                if (by_tma) {
                    if (!is_v && lane < 2) reinterpret_cast<uint32_t*>(sm + C::kOk)[(it % kRing) * 2 + lane] = 0xffffffffu;
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar(full0 + st), C::kTile);
                        mbar_arrive(bar(full0 + st));
                    }
                    __syncwarp();
                    if (lane < boxes) {
                        const CUtensorMap* map = is_v ? &ta.tm_v : &ta.tm_k;
                        const uint32_t dst = stage + lane * ta.box_rows * 128;
                        const int row = static_cast<int>(row_of(j0 + lane * ta.box_rows));
#pragma unroll
                        for (int cb = 0; cb < HD / 64; ++cb)
                            tma_box(dst + cb * kBlk, map, bar(full0 + st), cb * 64, static_cast<int>(g.gk), row, mine);
                    }
                    continue;
                }
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    // this lane's key
                    const int32_t x = x0 + k * 32 + lane, j = sv.lo + x;
                    const uint16_t* p = fresh;
                    bool have = false;
                    if (x < sv.new0) {
                        if (j >= first && j < sv.len && (!POS || (k ? pos[1] : pos[0]) >= low)) {
                            const int32_t page = entry_of(j);
                            have = page >= 0 && page < a.c.n_pages;
                            if (!have) set_status(a.c.status, SDPA_ERR_BOUNDS);
                            else p = pool + page * st_page + row_of(j) * st_row;
                        }
                    } else if (x - sv.new0 < sv.nq) {
                        have = ((x - sv.new0 < 32 ? used[0] : used[1]) >> ((x - sv.new0) & 31)) & 1;
                        p = fresh + (x - sv.new0) * st_new;
                    }
                    const uint32_t held = __ballot_sync(0xffffffffu, have);
                    if (!is_v && lane == 0) reinterpret_cast<uint32_t*>(sm + C::kOk)[(it % kRing) * 2 + k] = held;
#pragma unroll 8
                    for (int i = 0; i < 32 / RPI; ++i) {
                        const int r = i * RPI + sub;
                        const uint64_t q = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(p), r);
                        cp16(stage + swizzled<kBlk>(k * 32 + r, c), reinterpret_cast<const uint16_t*>(q) + c * 8, (held >> r) & 1);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    queue |= static_cast<uint64_t>(st) << (8 * pending);
                    if (++pending > LAG) wait_oldest();
                }
            }
            walk.advance(a, g);
        }
        // copies in flight end before the CTA does, whatever wait has run out
        cp_wait<0>();
        hand_over(0);
        for (uint32_t k = 0; k < NS && k < it; ++k) {
            const uint32_t r = it - 1 - k;
            mbar_wait(bar(full0 + r % NS), (r / NS) & 1, tmo);
        }
        __syncwarp();
    } else if (warp < kSoftWarp0) {
        // ------------------------------------------------------------ MMA issuer of slot `sl`
        constexpr uint32_t kIdS = idesc_f16(BF16, 128, 64, false, false);
        constexpr uint32_t kIdPV = idesc_f16(BF16, 128, HD, false, true);
        const int sl = warp - kMmaWarp;
        uint32_t it0 = 0, seg = 0, done = 0;       // done: this slot's key tiles before the segment
        bool ok = true;
        const uint32_t ts = tm_s0 + sl * 128, to = tm_o0 + sl * HD;
        const uint64_t dk0 = sdesc_sw128(sbase + C::kK, 16, 1024);
        const uint64_t dv0 = sdesc_sw128(sbase + C::kV, kBlk, 1024);
        if (elect_one()) {
        Seg g;
        while (ok && walk.next(a, g)) {
            const int32_t tiles = seg_tiles(g, walk.sv.tiles);
            const bool two = g.two;
            // this slot's key tiles: all, or every other one
            const int32_t first = two ? 0 : sl, step = two ? 1 : 2;
            const int32_t n = tiles > first ? (tiles - first + step - 1) / step : 0;
            const uint64_t dq = sdesc_sw128(sbase + C::kQ + (two ? sl : 0) * C::kQTile, 16, 1024);
            // The softmax groups have read the last segment's O and put this one's rows in place. A count, not a
            // barrier's parity: a slot may have no tile in a segment, and be two phases ahead or behind
            ok = wait_count(seg + 1);
            // S of the slot's i-th tile goes two ahead, into the buffer whose P V was issued last; it is put
            // off while its K is not there and a product can go first
            int32_t si = 0;
            for (int32_t i = 0; i < n && ok; ++i) {
                for (; si < n && si <= i + 1; ++si) {
                    const uint32_t r = it0 + first + si * step, st = r % NS;
                    if (si == i) {
                        if (!(ok = wait(tKFull + st, (r / NS) & 1))) break;
                    } else if (!mbar_test(bar(tKFull + st), (r / NS) & 1)) {
                        break;
                    }
                    const uint32_t b = (done + si) & 1;
                    const uint64_t dk = sdesc_at(dk0, st * C::kTile);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k)
                        mma_ss(ts + b * 64, sdesc_at(dq, (k >> 2) * kQBlk + (k & 3) * 32),
                               sdesc_at(dk, (k >> 2) * kBlk + (k & 3) * 32), kIdS, k > 0);
                    mma_commit(bar(tSFull + sl * 2 + b));
                    mbar_arrive(bar(tSFull + sl * 2 + b));
                    // a K tile has two readers; a lone one counts twice
                    mma_commit(bar(tKEmpty + st));
                    if (!two) mma_commit(bar(tKEmpty + st));
                }
                if (!ok) break;
                const uint32_t r = it0 + first + i * step, st = r % NS, b = (done + i) & 1;
                if (!(ok = wait(tVFull + st, (r / NS) & 1))) break;
                if (!(ok = wait(tPFull + sl * 2 + b, ((done + i) >> 1) & 1))) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_ts(to, ts + b * 64 + k * 8, sdesc_at(dv0, st * C::kTile + k * 2048), kIdPV, i > 0 || k > 0);
                mma_commit(bar(tPvDone + sl * 2 + b));
                mma_commit(bar(tVEmpty + st));
                if (!two) mma_commit(bar(tVEmpty + st));
            }
            done += n;
            it0 += tiles;
            ++seg;
            walk.advance(a, g);
        }
        // MMAs in flight end before TMEM is freed, whatever wait has run out
        mma_commit(bar(tDrain + sl));
        mbar_wait(bar(tDrain + sl), 0, tmo);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        const int sl = (warp - kSoftWarp0) >> 2;
        const int r = tid - (kSoftWarp0 + 4 * sl) * 32;     // index in the group
        // a warp reads the quarter of the TMEM lanes of its number modulo 4
        const int row = ((warp & 3) << 5) + lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tm_s = tm_s0 + sl * 128 + lane_off, tm_o = tm_o0 + sl * HD + lane_off;
        float2* ml = reinterpret_cast<float2*>(sm + C::kMl);
        uint64_t* masks = reinterpret_cast<uint64_t*>(sm + C::kMask);     // new tokens that each one's rows admit
        uint8_t* bits = reinterpret_cast<uint8_t*>(misc + 16);            // and its mask's number of bits
        const uint64_t scale2 = pair(__float_as_uint(a.scale_log2), __float_as_uint(a.scale_log2));
        uint32_t it0 = 0, cnt = 0;            // ring index at the segment's start; this slot's key tiles so far
        bool ok = true;
        const int64_t part0 = walk.at;
        uint32_t segs = 0;
        Seg g;
        while (walk.next(a, g)) {
            const SeqView& sv = walk.sv;
            const int32_t tiles = seg_tiles(g, sv.tiles), t0 = seg_tile0(g);
            named_sync(3, 256);               // the last segment's masks and statistics have been read
            if (sl == 0 && r < 64) {
                int n;
                masks[r] = admitted_tokens(a, g.bi, sv.nq, r, n);
                bits[r] = static_cast<uint8_t>(n);
            }
            if (sl == 0 && r == 0 && !a.whole)
                name_cut(a, part, walk.at == part0, walk.at + g.line_n - g.step0 - g.steps, g.cost, g.bi,
                         g.gk * blocks + g.blk, a.c.h_kv * blocks, g.step0, g.steps, g.of);
            // this thread's row
            const int rr = g.blk * 256 + (g.two ? sl * 128 : 0) + row;
            const int tok = rr < R ? rr / a.group : 0;
            const int64_t h = g.gk * a.group + (rr - tok * a.group);
            if (g.two || sl == 0) {
                const bool real = rr < R && tok < sv.nq;
                const uint16_t* qp = a.q + g.bi * a.q_stride[0] + tok * a.q_stride[1] + h * a.q_stride[2];
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) {
                    const uint4 x = real ? ld_nc_v4(qp + c * 8) : make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(sm + C::kQ + sl * C::kQTile + swizzled<kQBlk>(row, c)) = x;
                }
                fence_proxy_async_smem();
            }
            named_sync(3, 256);
            if (sl == 0 && r == 0)
                asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(sbase + C::kMisc + 8), "r"(++segs) : "memory");
            const uint64_t mask = rr < R ? masks[tok] : 0;
            const int64_t npos = a.c.next_pos ? a.c.next_pos[g.bi] : sv.len;
            int32_t low = INT32_MIN;
            if (a.window_left >= 0)
                low = static_cast<int32_t>(imax64(INT32_MIN, imin64(INT32_MAX, npos + bits[tok] - 1 - a.window_left)));
            const bool windowed = a.window_left >= 0;

            float m = -INFINITY, l = 0.f;
            const uint32_t cnt0 = cnt;
            for (int32_t tt = g.two ? 0 : sl; tt < tiles; tt += g.two ? 1 : 2) {
                const uint32_t my = cnt++, pb = sl * 2 + (my & 1);
                ok = ok && wait(tSFull + pb, (my >> 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
                tc_fence_after();
                const uint32_t ts = tm_s + (my & 1) * 64;
                uint32_t v[64];
                tmem_ld32(ts, *reinterpret_cast<uint32_t(*)[32]>(v));
                tmem_ld32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
                const uint32_t ring = (it0 + tt) % kRing;
                const int32_t x0 = (t0 + tt) * kKeys;
                const uint32_t* held = reinterpret_cast<const uint32_t*>(sm + C::kOk) + ring * 2;
                // every key is cached, held and in the window of all of the warp's rows
                const bool plain = x0 + kKeys <= sv.new0 && (held[0] & held[1]) == 0xffffffffu && !POS &&
                                   !__any_sync(0xffffffffu, windowed && mask != 0 && sv.lo + x0 < low);
                uint32_t see[2] = {0xffffffffu, 0xffffffffu};
                if (!plain) {
                    const int32_t* pos = reinterpret_cast<const int32_t*>(sm + C::kPos) + ring * kKeys;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        uint32_t s = held[w];
                        const int32_t xw = x0 + w * 32;
                        if (mask == 0) s = 0;
                        if (xw < sv.new0 ? windowed : false) {
#pragma unroll 1
                            for (int e = 0; e < 32; ++e)
                                if (xw + e < sv.new0 && pos[w * 32 + e] < low) s &= ~(1u << e);
                        }
                        if (xw + 31 >= sv.new0) {
                            // the mask's bits from the word's first new token on, behind cached keys
                            const int32_t u = xw - sv.new0;
                            s &= u >= 64 ? 0u : u >= 0 ? static_cast<uint32_t>(mask >> u)
                                                       : static_cast<uint32_t>(mask << -u) | ((1u << -u) - 1);
                        }
                        see[w] = s;
                    }
                }
                tmem_ld_wait();
                loaded(*reinterpret_cast<uint32_t(*)[32]>(v));
                loaded(*reinterpret_cast<uint32_t(*)[32]>(v + 32));
                if (!plain) {
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (!((see[e >> 5] >> (e & 31)) & 1)) v[e] = 0xff800000u;   // -inf
                }
                float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 64; e += 2)
                    x[(e >> 1) & 3] = max3(x[(e >> 1) & 3], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * a.scale_log2;
                const bool up = top > m + kMoves<BF16>;
                if (__any_sync(0xffffffffu, up)) {
                    const float f = !up ? 1.f : m == -INFINITY ? 0.f : ex2_approx(m - (top - kBelow<BF16>));
                    l *= f;
                    m = up ? top - kBelow<BF16> : m;
                    if (my != cnt0) {
                        // O holds the P V of this slot's earlier keys: they are done before it changes
                        ok = __all_sync(0xffffffffu, wait(tPvDone + (pb ^ 1), ((my - 1) >> 1) & 1));
                        tc_fence_after();
                        if (ok) {
#pragma unroll 1
                            for (int cb = 0; cb < HD / 16; ++cb) {
                                uint32_t o16[16];
                                tmem_ld16(tm_o + cb * 16, o16);
                                tmem_ld_wait();
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    uint32_t w8[8];
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        w8[e] = __float_as_uint(__uint_as_float(o16[8 * q + e]) * f);
                                    tmem_st8(tm_o + cb * 16 + 8 * q, w8);
                                }
                            }
                            tmem_st_wait();
                        }
                    }
                }
                // P over the first columns of its S
                const float mr = m == -INFINITY ? 0.f : m;
                const uint64_t mr2 = pair(__float_as_uint(-mr), __float_as_uint(-mr));
                uint64_t ps[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t w8[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // a masked score is -inf, its P is 0
                        const uint64_t y = fma2(pair(v[16 * q + 2 * e], v[16 * q + 2 * e + 1]), scale2, mr2);
                        const float p0 = ex2_approx(lo_of(y)), p1 = ex2_approx(hi_of(y));
                        ps[e & 3] = add2(ps[e & 3], pair(__float_as_uint(p0), __float_as_uint(p1)));
                        w8[e] = pack2<BF16>(p0, p1);
                    }
                    tmem_st8(ts + 8 * q, w8);
                }
                const uint64_t pt = add2(add2(ps[0], ps[1]), add2(ps[2], ps[3]));
                l += lo_of(pt) + hi_of(pt);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(tPFull + pb));
            }
            // the slot's last P V is done
            if (cnt != cnt0) {
                ok = ok && wait(tPvDone + sl * 2 + ((cnt - 1) & 1), ((cnt - 1) >> 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
            }
            tc_fence_after();
            if (mask == 0) {
                m = -INFINITY;
                l = 0.f;
            }
            ml[sl * 128 + row] = make_float2(m, l);
            tc_fence_before();
            named_sync(3, 256);
            tc_fence_after();
            // two row tiles: each slot its rows; one: both slots the same rows,
            // each half of the features, from both slots' sums
            const bool whole = g.steps == g.of;
            const int64_t slot = blockIdx.x * int64_t(2) + (walk.at == part0 ? 0 : 1);
            const int urow = (g.two ? sl * 128 : 0) + row;         // row in the unit
            float top = m, sum = l, f0 = 1.f, f1 = 0.f;
            if (!g.two) {
                const float2 x = ml[row], y = ml[128 + row];
                top = fmaxf(x.x, y.x);
                f0 = x.x == -INFINITY ? 0.f : ex2_approx(x.x - top);
                f1 = tiles < 2 || y.x == -INFINITY ? 0.f : ex2_approx(y.x - top);
                sum = f0 * x.y + f1 * y.y;
            }
            const int cb0 = g.two ? 0 : sl * (HD / 64), cb1 = g.two ? HD / 32 : cb0 + HD / 64;
            // (rows behind the last one, empty, as far as the join reads)
            const int stored = whole ? R : (R + kPartialRows - 1) / kPartialRows * kPartialRows;
            const bool dead = top == -INFINITY;          // (no key, or NaN scores: store_row sees it by the sum)
            if (ok) {
#pragma unroll 1
                for (int cb = cb0; cb < cb1; ++cb) {
                    uint32_t v[32];
                    float x[32];
                    __syncwarp();       // rows behind the last one have left the last turn early
                    tmem_ld32((g.two ? tm_o : tm_o0 + lane_off) + cb * 32, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = dead || f0 == 0.f ? 0.f : f0 * __uint_as_float(v[e]);
                    if (!g.two && tiles > 1) {
                        tmem_ld32(tm_o0 + HD + lane_off + cb * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!dead && f1 != 0.f) x[e] += f1 * __uint_as_float(v[e]);
                    }
                    if (rr >= stored) continue;
                    if (!whole) {
                        float* po = a.part_o + (slot * 256 + urow) * HD + cb * 32;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(po + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                        if (cb == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * 256 + urow) * 2) = make_float2(top, sum);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float y[8];
#pragma unroll
                            for (int q = 0; q < 8; ++q) y[q] = x[e + q];
                            store_row<BF16, 8>(a, g.bi, tok, h, cb * 32 + e, tok < sv.nq, top, sum, y);
                        }
                    }
                }
            }
            tc_fence_before();
            it0 += tiles;
            walk.advance(a, g);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (!a.whole) grid_dep_launch();
}

namespace {

template <int HD, bool BF16, bool POS>
cudaError_t launch_tile_pos(const CacheTileArgs& a, cudaStream_t s)
{
    auto kern = cache_fwd_tile_kernel<HD, BF16, POS>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, TileCfg<HD>::kBytes, allowed);
    if (e != cudaSuccess) return e;
    kern<<<a.f.parts, kTileThreads, TileCfg<HD>::kBytes, s>>>(a);
    return cudaGetLastError();
}

template <int HD, bool BF16>
cudaError_t launch_tile_typed(const CacheTileArgs& a, cudaStream_t s)
{
    return a.f.c.positions != nullptr && a.f.window_left >= 0 ? launch_tile_pos<HD, BF16, true>(a, s)
                                                              : launch_tile_pos<HD, BF16, false>(a, s);
}

}  // namespace

cudaError_t launch_cache_fwd_tiles(const CacheTileArgs& a, int dtype, cudaStream_t s)
{
    if (a.f.c.d == 128)
        return dtype == SDPA_BF16 ? launch_tile_typed<128, true>(a, s) : launch_tile_typed<128, false>(a, s);
    return dtype == SDPA_BF16 ? launch_tile_typed<64, true>(a, s) : launch_tile_typed<64, false>(a, s);
}

}  // namespace swa
