// cache_tile.cuh -- the cache forward for many rows per kv-head: tcgen05 tiles.
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
#pragma once

#include <type_traits>

#include "cache4.cuh"
#include "cache_fwd.cuh"

namespace swa {

namespace {

// Threads: with a cache in 4 bits four warps more
template <bool Q4>
constexpr int kTileThreads = Q4 ? 512 : 384;
constexpr int kMmaWarp = 2;            // and 3
constexpr int kSoftWarp0 = 4;
constexpr int kKeys = 64;              // keys of a tile
constexpr uint32_t kQBlk = 128 * 128;  // one 64-column block of a 128-row 16-bit tile
constexpr uint32_t kBlk = kKeys * 128; // the same of a key tile
constexpr int kRing = 16;              // key tiles whose validity and positions are kept
constexpr int kRawStages = 4;          // 4 bits: key tiles that are on their way as they are held

template <int HD, bool Q4>
struct TileCfg {
    static constexpr uint32_t kQTile = 128 * HD * 2;
    static constexpr uint32_t kTile = kKeys * HD * 2;
    static constexpr int kStages = Q4 ? (HD == 128 ? 3 : 6) : HD == 128 ? 4 : 8;
    static constexpr uint32_t kRaw1 = 4 * Group4<HD>::kBytes;      // 4 bits: a key tile as it is held
    static constexpr uint32_t kQ = 0;                           // 2 slots
    static constexpr uint32_t kK = kQ + 2 * kQTile;
    static constexpr uint32_t kV = kK + kStages * kTile;
    static constexpr uint32_t kRaw = kV + kStages * kTile;       // K's ring, V's ring, which of their keys count
    static constexpr uint32_t kRawOk = kRaw + (Q4 ? 2 * kRawStages * kRaw1 : 0);
    static constexpr uint32_t kPos = kRawOk + (Q4 ? 2 * kRawStages * 8 : 0);      // int32 [kRing][64]
    static constexpr uint32_t kOk = kPos + kRing * 256;         // uint32 [kRing][2]
    static constexpr uint32_t kMask = kOk + kRing * 8;          // uint64 [64]
    static constexpr uint32_t kMl = kMask + 512;                // float2 [2][128]
    static constexpr uint32_t kBars = kMl + 2048;
    static constexpr uint32_t kMisc = kBars + 512;
    static constexpr uint32_t kBytes = kMisc + 256 + 1024;
    static_assert(kBytes <= 232448, "shared memory above the 227 KB a CTA may opt into");
};

// mbarriers; per-stage and per-slot ones at index + stage or slot (S, P and
// P V: slot * 2 + buffer)
enum TBar : int { tKFull = 0, tKEmpty = 8, tVFull = 16, tVEmpty = 24, tSFull = 32, tPFull = 36, tPvDone = 40, tDrain = 44,
                  tNumBars = 46, tRawKFull = 46, tRawKEmpty = 50, tRawVFull = 54, tRawVEmpty = 58, tNumBars4 = 62 };
static_assert(kRawStages <= 4, "mbarriers of the raw stages");
static_assert(tNumBars4 * 8 <= 512, "mbarrier area");

template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How a sequence's steps are laid out: per kv-head `na` blocks of 256 rows
// with two row tiles (a step is one key tile), then perhaps one block with one
// row tile (a step is two key tiles; over a cache in 4 bits one, as its cost is the values'
// way out of it), each with its fixed cost before it (by its row tiles: Q in, O out).
struct Shape {
    int32_t ta, tb;       // steps of a two-tile block, of a one-tile block
    int64_t per_head;
};

template <int HD, bool Q4>
struct Walk;

template <int HD, bool Q4>
__device__ __forceinline__ Shape shape_of(const SeqView& v, int na, int nb, int32_t cost)
{
    using W = Walk<HD, Q4>;
    Shape s;
    s.ta = v.tiles;
    s.tb = Q4 ? v.tiles : (v.tiles + 1) >> 1;
    s.per_head = static_cast<int64_t>(na) * ((s.ta + 2 * cost) * W::kTwo) + static_cast<int64_t>(nb) * ((s.tb + cost) * W::kOne);
    return s;
}

// One stretch of a CTA's part that lies in one unit.
struct Seg {
    int64_t bi, gk;
    int32_t blk;          // row block
    bool two;             // two row tiles
    int32_t step0, steps, of, line_n, cost;   // its steps, how many the unit has, its places in the line, the unit's cost
};

template <bool Q4>
__device__ __forceinline__ SeqView tile_view(const CacheFwdArgs& a, int64_t bi)
{
    if constexpr (Q4) return seq_view4(a, bi, kKeys, kKeys);
    else return seq_view(a, bi, kKeys, kKeys);
}

// A CTA's way through its part of the line.
template <int HD, bool Q4>
struct Walk {
    static constexpr int kTwo = 1, kOne = 1;      // places of a step with two row tiles, with one
    int64_t at, end, bi, rem;
    int na, nb;
    SeqView sv;
    Shape sh;
    bool loaded;

    __device__ __forceinline__ void begin(const CacheFwdArgs&, const Part& p, int na_, int nb_)
    {
        na = na_;
        nb = nb_;
        at = p.at;
        end = p.end;
        bi = p.bi;
        rem = p.rem;
    }
    // Changes from segment to segment; the place of a segment's unit's tile 0.
    __device__ __forceinline__ int64_t mark() const { return at; }
    __device__ __forceinline__ int64_t tile0_place(const Part&, const Seg& g) const { return at + g.line_n - g.step0 - g.steps; }
    // The next segment with steps; false at the part's end.
    __device__ __forceinline__ bool next(const CacheFwdArgs& a, Seg& g)
    {
        if (at >= end) return false;
        if (!loaded) {
            sv = tile_view<Q4>(a, bi);
            sh = shape_of<HD, Q4>(sv, na, nb, a.unit_cost);
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

// Over a cache in 4 bits, d = 64: a step with one row tile takes 3/4 of the time of one
// with two, and so of the places. It steps from unit to unit, without divisions: fewer
// instructions in each role. 12 sequences of 16484 keys, 6 kv-heads, 296 rows 232 us, 272
// with even places, 300 by the form above; d = 128 by this form 2 % more (24 rows 14 %),
// and the places as they are are even there.
template <>
struct Walk<64, true> {
    static constexpr int kTwo = 4, kOne = 3;
    int64_t left;                 // places
    int32_t bi, gk, blk, y;       // y: the place among the unit's
    int na, nb;
    SeqView sv;
    bool loaded;

    static __device__ __forceinline__ int32_t places(bool two) { return two ? kTwo : kOne; }

    __device__ __forceinline__ void begin(const CacheFwdArgs& a, const Part& p, int na_, int nb_)
    {
        na = na_;
        nb = nb_;
        left = p.end - p.at;
        bi = static_cast<int32_t>(p.bi);
        sv = tile_view<true>(a, bi);
        loaded = true;
        const Shape sh = shape_of<64, true>(sv, na, nb, a.unit_cost);
        gk = static_cast<int32_t>(quotient(p.rem, sh.per_head));
        const int64_t r = p.rem - gk * sh.per_head;
        const int32_t each = (sh.ta + 2 * a.unit_cost) * kTwo;
        blk = static_cast<int32_t>(imin64(na, quotient(r, each)));
        y = static_cast<int32_t>(r - static_cast<int64_t>(blk) * each);
    }
    __device__ __forceinline__ int64_t mark() const { return left; }
    __device__ __forceinline__ int64_t tile0_place(const Part& p, const Seg& g) const
    {
        return p.end - left - y + g.cost * places(g.two);
    }
    __device__ __forceinline__ bool next(const CacheFwdArgs& a, Seg& g)
    {
        if (left <= 0) return false;
        if (!loaded) {
            sv = tile_view<true>(a, bi);
            loaded = true;
        }
        g.bi = bi;
        g.gk = gk;
        g.blk = blk;
        g.two = blk < na;
        g.of = sv.tiles;
        g.cost = (g.two ? 2 : 1) * a.unit_cost;
        const int32_t w = places(g.two);
        g.line_n = static_cast<int32_t>(imin64((g.of + g.cost) * w - y, left));
        g.step0 = max(0, y / w - g.cost);
        g.steps = max(0, (y + g.line_n) / w - g.cost) - g.step0;
        return g.steps > 0;
    }
    __device__ __forceinline__ void advance(const CacheFwdArgs& a, const Seg& g)
    {
        left -= g.line_n;
        if (left <= 0) return;
        y = 0;                    // (only a part's end is inside a unit)
        if (++blk < na + nb) return;
        blk = 0;
        if (++gk < a.c.h_kv) return;
        gk = 0;
        ++bi;
        loaded = false;
    }
};

// Key tiles of a segment: one for each step with two row tiles, two with one
// (the unit's last step may have only one).
template <bool Q4>
__device__ __forceinline__ int32_t seg_tile0(const Seg& g) { return Q4 || g.two ? g.step0 : 2 * g.step0; }
template <bool Q4>
__device__ __forceinline__ int32_t seg_tiles(const Seg& g, int32_t tiles)
{
    return Q4 || g.two ? g.steps : min(2 * (g.step0 + g.steps), tiles) - 2 * g.step0;
}

// ---- a cache in 4 bits
//
// K and V tiles are made in shared memory, as f16, out of the codes: two warps bring
// them as they are held, two turn K's and two V's (a warp 32 keys of each tile). Q is
// f16 as well (see cache4_fwd.cu). 12 sequences of 16484 keys, 6 kv-heads, d = 128: 24
// rows 131 us, 128 rows 133, 256 rows 177, 296 rows 302; of 16 bits 109, 114, 142, 237.
// d = 64: 128 rows 105 and 84, 296 rows 233 and 204.
//
// Below 128 rows the turning warps' chain is the bound (about 2000 cycles a tile: wait,
// load, 200 operations, store, fence), above it that of the softmax groups beside it.
// What costs most there is instructions: with K's and V's turning as functions of their
// own (more code between the same loops, fewer registers spilled) 296 rows took 370 to
// 520 us, with all warps' registers set behind one branch (and softmax spilling) 381.
// Setting them takes whole warpgroups: warps 0-3 and 12-15 the lower number, 4-11 the
// higher. A softmax of 32 columns at a time: 334 us.
//
// A tile's columns (keys of S, and of P and V) are in the order in which V's values come out of their groups in runs of
// 16 bytes: of each 32 keys, column 8 t + 4 q + e is key 16 q + 4 t + e. V lies transposed, its row 8 i + rho(g) is
// feature i of lane row g's run of d / 8, rho(g) chosen so that the lanes of a store meet no bank twice.

__device__ __forceinline__ int lane_row4(int g) { return ((g & 1) << 2) | (g >> 1); }

// Bits of 32 keys in their own order -> in the columns'.
__device__ __forceinline__ uint32_t column_order4(uint32_t x)
{
    auto spread = [](uint32_t y) -> uint32_t {
        y = (y | y << 8) & 0x00ff00ffu;
        return (y | y << 4) & 0x0f0f0f0fu;
    };
    return spread(x & 0xffffu) | spread(x >> 16) << 4;
}

// Waits of a whole warp: bounded, and given up with the CTA.
__device__ __forceinline__ bool wait_warp4(const CacheFwdArgs& a, uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag)
{
    bool ok = mbar_try_wait(bar, parity);
    if (!ok && !*abort_flag) {
        ok = mbar_wait(bar, parity, static_cast<uint64_t>(a.timeout_ns));
        if (!ok) {
            *abort_flag = 1;
            set_status(a.c.status, SDPA_ERR_TIMEOUT);
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// Brings the tiles of K (is_v: V) of cached keys as they are held into a ring of raw stages, by bulk copies of as many
// keys as a page and a tile allow, and says which keys count. It runs ahead over the ends of units.
template <int HD, bool POS>
__device__ __forceinline__ void tile_load4(const CacheTileArgs& ta, Walk<HD, true> walk, uint8_t* sm, bool is_v, int lane)
{
    const CacheFwdArgs& a = ta.f;
    using C = TileCfg<HD, true>;
    const uint32_t sbase = smem_u32(sm);
    auto bar = [&](int i) -> uint32_t { return sbase + C::kBars + 8u * i; };
    volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(sm + C::kMisc) + 1;
    const int full0 = is_v ? tRawVFull : tRawKFull, empty0 = is_v ? tRawVEmpty : tRawKEmpty;
    const uint32_t raw0 = sbase + C::kRaw + (is_v ? kRawStages * C::kRaw1 : 0);
    uint32_t* const oks0 = reinterpret_cast<uint32_t*>(sm + C::kRawOk) + (is_v ? kRawStages * 2 : 0);
    const int ck = ta.box_rows, nu = kKeys / ck;                // keys of a copy, copies of a tile
    const uint32_t bytes = ck / 16 * Group4<HD>::kBytes;
    uint32_t sent = 0;
    bool ok = is_v || !a.c.stall;                               // (test hook: no K comes)
    Seg g;
    while (ok && walk.next(a, g)) {
        const SeqView& sv = walk.sv;
        const int32_t* kpos = POS ? a.c.positions + (g.bi * a.c.h_kv + g.gk) * a.c.cap : nullptr;
        const int32_t t0 = seg_tile0<true>(g);
        const int32_t cached = min(t0 + seg_tiles<true>(g, sv.tiles), sv.new0 / kKeys);   // the segment's tiles of cached keys end here
        const uint8_t* pool = reinterpret_cast<const uint8_t*>(is_v ? a.c.v : a.c.k) + g.gk * (is_v ? a.c.v_stride[2] : a.c.k_stride[2]);
        const int64_t st_page = is_v ? a.c.v_stride[0] : a.c.k_stride[0];
        // the lowest position in any row's window
        int32_t low = INT32_MIN;
        if (a.window_left >= 0) {
            int32_t shallow = 64;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                int bits;
                if (admitted_tokens(a, g.bi, sv.nq, w * 32 + lane, bits)) shallow = min(shallow, bits);
            }
            const int64_t npos = a.c.next_pos ? a.c.next_pos[g.bi] : sv.len;
            low = static_cast<int32_t>(imax64(INT32_MIN, imin64(INT32_MAX,
                npos + static_cast<int32_t>(__reduce_min_sync(0xffffffffu, shallow)) - 1 - a.window_left)));
        }
        // the page of lane's copy of tile t, a tile ahead
        auto fetch_entry = [&](int32_t t) -> int32_t {
            if (a.c.page_table == nullptr) return static_cast<int32_t>(g.bi);
            const int32_t j = sv.lo + t * kKeys + lane * ck;
            return lane < nu && t < cached && j < sv.len ? cache_entry(a.c, g.bi, j) : 0;
        };
        int32_t entry = fetch_entry(t0);
#pragma unroll 1
        for (int32_t t = t0; t < cached; ++t, ++sent) {
            const int32_t mine = entry;
            entry = fetch_entry(t + 1);
            const uint32_t rs = sent % kRawStages;
            const int32_t j0 = sv.lo + t * kKeys;
            const bool paged = mine >= 0 && mine < a.c.n_pages;
            // lanes whose copies have all their keys in reach, and on a page
            const int32_t ju = j0 + lane * ck;
            const bool whole = !POS && lane < nu && paged && ju + ck <= sv.len && (a.window_left < 0 || ju >= low);
            uint32_t oks[2] = {0xffffffffu, 0xffffffffu};
            if ((__ballot_sync(0xffffffffu, whole || lane >= nu)) != 0xffffffffu) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int32_t x = w * 32 + lane, j = j0 + x;
                    const bool there = __shfl_sync(0xffffffffu, paged ? 1 : 0, x / ck) != 0;
                    bool in = j < sv.len;
                    if (in && a.window_left >= 0) in = (POS ? kpos[j] : j) >= low;
                    if (in && !there) set_status(a.c.status, SDPA_ERR_BOUNDS);
                    oks[w] = __ballot_sync(0xffffffffu, in && there);
                }
            }
            const int first = lane * ck;
            const uint32_t part = ck == 64 ? oks[0] | oks[1] : ck == 32 ? oks[lane & 1] : (oks[(lane >> 1) & 1] >> (first & 31)) & 0xffffu;
            const bool go = lane < nu && part != 0;
            const uint32_t copies = __popc(__ballot_sync(0xffffffffu, go));
            if (!(ok = wait_warp4(a, bar(empty0 + rs), ((sent / kRawStages) & 1) ^ 1, abort_flag))) break;
            if (lane == 0) {
                oks0[rs * 2] = oks[0];
                oks0[rs * 2 + 1] = oks[1];
                mbar_arrive_expect_tx(bar(full0 + rs), copies * bytes);
            }
            __syncwarp();
            if (go) {
                const uint32_t row = a.c.page_table == nullptr ? ju : cache_row(a.c, ju);
                bulk_load(raw0 + rs * C::kRaw1 + lane * bytes, pool + mine * st_page + static_cast<int64_t>(row >> 4) * Group4<HD>::kBytes,
                          bytes, bar(full0 + rs));
            }
        }
        walk.advance(a, g);
    }
    // copies in flight end before the CTA does, whatever wait has run out
    for (uint32_t k = 0; k < kRawStages && k < sent; ++k) {
        const uint32_t r = sent - 1 - k;
        mbar_wait(bar(full0 + r % kRawStages), (r / kRawStages) & 1, static_cast<uint64_t>(a.timeout_ns));
    }
    __syncwarp();
}

// Turns 32 keys (half p) of every tile of K (is_v: V) into f16 in the 128-byte swizzle. The new tokens' tile comes from
// their 16-bit form.
template <int HD, bool BF16, bool POS>
__device__ __forceinline__ void tile_convert4(const CacheTileArgs& ta, Walk<HD, true> walk, uint8_t* sm, bool is_v, int p, int lane)
{
    const CacheFwdArgs& a = ta.f;
    using C = TileCfg<HD, true>;
    constexpr int NS = C::kStages, KW = HD / 32;
    const uint32_t sbase = smem_u32(sm);
    auto bar = [&](int i) -> uint32_t { return sbase + C::kBars + 8u * i; };
    volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(sm + C::kMisc) + 1;
    const int full0 = is_v ? tVFull : tKFull, empty0 = is_v ? tVEmpty : tKEmpty;
    const int raw_full0 = is_v ? tRawVFull : tRawKFull, raw_empty0 = is_v ? tRawVEmpty : tRawKEmpty;
    const uint32_t ring0 = is_v ? C::kV : C::kK, raw0 = C::kRaw + (is_v ? kRawStages * C::kRaw1 : 0) + p * (C::kRaw1 / 2);
    const uint32_t* const oks0 = reinterpret_cast<const uint32_t*>(sm + C::kRawOk) + (is_v ? kRawStages * 2 : 0) + p;
    const int lg = lane >> 2, lt = lane & 3;
    uint32_t it = 0, got = 0;                                   // tiles so far, those of cached keys
    bool ok = true;
    Seg g;
    while (ok && walk.next(a, g)) {
        const SeqView& sv = walk.sv;
        const int32_t t0 = seg_tile0<true>(g), t1 = t0 + seg_tiles<true>(g, sv.tiles) - 1;
#pragma unroll 1
        for (int32_t t = t0; t <= t1; ++t, ++it) {
            const uint32_t st = it % NS, rs = got % kRawStages;
            const int32_t w0 = t * kKeys + p * 32 - sv.new0;        // new tokens: the first of the 32
            const bool fresh = w0 >= 0;
            if (!(ok = wait_warp4(a, bar(empty0 + st), ((it / NS) & 1) ^ 1, abort_flag))) break;
            if (!fresh && !(ok = wait_warp4(a, bar(raw_full0 + rs), (got / kRawStages) & 1, abort_flag))) break;
            uint8_t* stage = sm + ring0 + st * C::kTile;
            uint32_t oks;
            if (!fresh) {
                oks = oks0[rs * 2];
            } else {
                // new tokens that some row admits: the others may be anything, and would meet a P of 0
                uint32_t used = 0;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    int bits;
                    const uint64_t m = admitted_tokens(a, g.bi, sv.nq, w * 32 + lane, bits);
                    used |= __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(p ? m >> 32 : m));
                }
                oks = used;
            }
            if (!is_v) {
                if (lane == 0) reinterpret_cast<uint32_t*>(sm + C::kOk)[(it % kRing) * 2 + p] = oks;
                if (a.window_left >= 0) {
                    const int32_t j = sv.lo + t * kKeys + p * 32 + lane;
                    const int32_t* kpos = POS ? a.c.positions + (g.bi * a.c.h_kv + g.gk) * a.c.cap : nullptr;
                    reinterpret_cast<int32_t*>(sm + C::kPos)[(it % kRing) * kKeys + p * 32 + lane] = POS && j < sv.len ? kpos[j] : j;
                }
            }
            if (!fresh) {
                const uint8_t* raw = sm + raw0 + rs * C::kRaw1;
                uint32_t w[2][2][KW], sc[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint8_t* grp = raw + q * Group4<HD>::kBytes;
                    const Words4<HD> x = words4<HD>(grp, lane);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                        for (int k = 0; k < KW; ++k) w[q][hh][k] = x.w[hh][k];
                    sc[q] = is_v ? v_scales4<HD>(grp, lane) : k_scales4<HD>(grp, lane);
                }
                if (!is_v) {
                    // rows of keys: the lane has a quarter of the features of two keys of each group. Lanes two quarters
                    // apart would write to the same banks: they take their words in another order
                    const uint32_t turn = HD == 128 && lt >= 2 ? 2 : 0;
                    // 16-byte piece c of row r: a row's 8 pieces are exchanged by c ^ (r & 7); of r & 7, q and hh are bits 2 and 1
                    uint8_t* const dst = stage + (HD == 128 ? lt >> 1 : 0) * kBlk + (p * 4 + (lg >> 1)) * 1024 + (lg & 1) * 128;
                    const uint32_t c0 = (HD == 128 ? (lt & 1) * 4 : lt * 2) ^ turn ^ (lg & 1);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            Scale4 s[2];
                            if constexpr (HD == 128) {
                                const uint32_t x = turn ? __byte_perm(sc[q], 0u, 0x2301) : sc[q];
                                s[0] = hh ? scale4<0x2424>(x) : scale4<0x0404>(x);
                                s[1] = hh ? scale4<0x3434>(x) : scale4<0x1414>(x);
                            } else {
                                s[0] = s[1] = hh ? scale4<0x1414>(sc[q]) : scale4<0x0404>(sc[q]);
                            }
#pragma unroll
                            for (int k = 0; k < KW; ++k) {
                                const uint32_t x = HD == 128 && turn ? w[q][hh][(k + 2) & 3] : w[q][hh][k];
                                uint32_t f[4];
                                values4(x, s[k >> 1], f);
                                *reinterpret_cast<uint4*>(dst + (q * 4 + hh * 2) * 128 + ((c0 ^ k ^ (q * 4 + hh * 2)) << 4)) =
                                    make_uint4(f[0], f[1], f[2], f[3]);
                            }
                        }
                } else {
                    // rows of features: the lane has a run of features of 4 keys of each group
                    uint8_t* const dst = stage + lane_row4(lg) * 128 + (((p * 4 + lt) ^ lane_row4(lg)) << 4);
                    Scale4 s[2][2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t x = sc[q];
                        // what stands in the place of a key that does not count meets a P of 0: its scale has to be 0
                        if (oks != 0xffffffffu) x &= (((oks >> (q * 16 + 4 * lt)) & 15) * 0x00204081u & 0x01010101u) * 255u;
                        s[q][0] = scale4<0x1404>(x), s[q][1] = scale4<0x3424>(x);
                    }
#pragma unroll
                    for (int k = 0; k < KW; ++k) {
                        uint32_t f[2][2][4];
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int hh = 0; hh < 2; ++hh) values4(w[q][hh][k], s[q][hh], f[q][hh]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4*>(dst + (4 * k + j) * 1024) = make_uint4(f[0][0][j], f[0][1][j], f[1][0][j], f[1][1][j]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(raw_empty0 + rs));
                ++got;
            } else if (!is_v) {
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    const int x = (q >> 1) * 16 + 4 * (lg >> 1) + (lg & 1) + 2 * (q & 1);
                    const int row = p * 32 + (lg >> 1) * 8 + (q >> 1) * 4 + (lg & 1) + 2 * (q & 1);
                    const bool in = (oks >> x) & 1;
                    const uint16_t* kn = a.k + g.bi * a.k_stride[0] + (w0 + x) * a.k_stride[1] + g.gk * a.k_stride[2] + lt * (HD / 4);
#pragma unroll 1
                    for (int k = 0; k < KW; ++k) {
                        const uint4 y = in ? ld_nc_v4(kn + k * 8) : make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4*>(stage + swizzled<kBlk>(row, lt * KW + k)) =
                            make_uint4(to_f16x2<BF16>(y.x), to_f16x2<BF16>(y.y), to_f16x2<BF16>(y.z), to_f16x2<BF16>(y.w));
                    }
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < HD / 64; ++c) {
                    uint32_t v[8][4];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int x = (k >> 2) * 16 + 4 * lt + (k & 3);
                        const uint16_t* vn = a.v + g.bi * a.v_stride[0] + (w0 + x) * a.v_stride[1] + g.gk * a.v_stride[2] + lg * (HD / 8);
                        const uint4 y = (oks >> x) & 1 ? ld_nc_v4(vn + c * 8) : make_uint4(0u, 0u, 0u, 0u);
                        v[k][0] = to_f16x2<BF16>(y.x), v[k][1] = to_f16x2<BF16>(y.y);
                        v[k][2] = to_f16x2<BF16>(y.z), v[k][3] = to_f16x2<BF16>(y.w);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t sel = z ? 0x7632 : 0x5410;
                            *reinterpret_cast<uint4*>(stage + swizzled<kBlk>((8 * c + 2 * j + z) * 8 + lane_row4(lg), p * 4 + lt)) =
                                make_uint4(__byte_perm(v[0][j], v[1][j], sel), __byte_perm(v[2][j], v[3][j], sel),
                                           __byte_perm(v[4][j], v[5][j], sel), __byte_perm(v[6][j], v[7][j], sel));
                        }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(full0 + st));
        }
        walk.advance(a, g);
    }
}

}  // namespace

// POS: a window over keys that have positions. An instance of its own: the
// checks of positions lengthen the loaders' way to a tile (12 sequences of 16484
// keys, 6 kv-heads, 296 rows: 255 us with one instance for both, 223 without the
// checks; d = 64 230 and 193; 16 to 512 rows of one kind of block 1 to 2 %. It is
// the pace, not the reads: 223 and 217 MB from DRAM for 3 of the sequences).
template <int HD, bool BF16, bool POS, bool Q4>
__global__ void __launch_bounds__(kTileThreads<Q4>, 1) cache_fwd_tile_kernel(const __grid_constant__ CacheTileArgs ta)
{
    const CacheFwdArgs& a = ta.f;
    using C = TileCfg<HD, Q4>;
    constexpr bool MB = BF16 && !Q4;      // the products' type: values of 4 bits are f16
    constexpr int NS = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ int64_t sh_sum[kTileThreads<Q4> / 32], sh_at[2];
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
    using W = Walk<HD, Q4>;
    Part part{1, 0, 0, 0, 0, Line{0}};
    if (a.whole) {
        const int64_t units = a.c.h_kv * blocks;
        part.bi = blockIdx.x / units;
        const int64_t un = blockIdx.x - part.bi * units, gk = un / blocks, blk = un - gk * blocks;
        const Shape s = shape_of<HD, Q4>(tile_view<Q4>(a, part.bi), na, nb, a.unit_cost);
        const int w = blk < na ? W::kTwo : W::kOne;
        part.rem = gk * s.per_head + blk * (s.ta + 2 * a.unit_cost) * W::kTwo + (blk < na ? 2 : 1) * a.unit_cost * w;
        part.end = static_cast<int64_t>(blk < na ? s.ta : s.tb) * w;
    } else {
        part = find_part<kTileThreads<Q4>, W::kTwo>(
            a.c.b, [&](int64_t i) { return a.c.h_kv * shape_of<HD, Q4>(tile_view<Q4>(a, i), na, nb, a.unit_cost).per_head; }, sh_sum, sh_at);
        if (tid == 0 && !a.cut_by_unit) a.cuts[blockIdx.x].bi = -1;
        if (part.end == 0) {
            grid_dep_launch();
            return;
        }
    }
    W walk{};
    walk.begin(a, part, na, nb);

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
        if constexpr (Q4)
            for (int i = 0; i < kRawStages; ++i) {
                mbar_init(bar(tRawKFull + i), 1);
                mbar_init(bar(tRawKEmpty + i), 2);
                mbar_init(bar(tRawVFull + i), 1);
                mbar_init(bar(tRawVEmpty + i), 2);
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

    // (4 bits: the softmax groups' registers come out of the other warpgroups', 512 x 128 in all: 2 x 152 + 2 x 104. Every
    // warp of a warpgroup runs the same instruction, and it stands in the branch whose registers it sets: behind a branch
    // that joins again the compiler has to take the lower number for all)
    if (warp < kSoftWarp0 || warp >= kSoftWarp0 + 8) {
    if constexpr (Q4) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (Q4 && (warp < kMmaWarp || warp >= kSoftWarp0 + 8)) {
        if constexpr (Q4) {
            // warps 12 and 13 load; 0 and 1 turn K, 14 and 15 V: each of the four schedulers has one of these beside the softmax
            if (warp == kSoftWarp0 + 8 || warp == kSoftWarp0 + 9) tile_load4<HD, POS>(ta, walk, sm, warp & 1, lane);
            else tile_convert4<HD, BF16, POS>(ta, walk, sm, warp >= kSoftWarp0, warp & 1, lane);
        }
    } else if (warp < kMmaWarp) {
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
            const int32_t t0 = seg_tile0<Q4>(g), t1 = t0 + seg_tiles<Q4>(g, sv.tiles) - 1;
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
    } else {
        // ------------------------------------------------------------ MMA issuer of slot `sl`
        constexpr uint32_t kIdS = idesc_f16(MB, 128, 64, false, false);
        constexpr uint32_t kIdPV = idesc_f16(MB, 128, HD, false, !Q4);      // (4 bits: V lies transposed)
        const int sl = warp - kMmaWarp;
        uint32_t it0 = 0, seg = 0, done = 0;       // done: this slot's key tiles before the segment
        bool ok = true;
        const uint32_t ts = tm_s0 + sl * 128, to = tm_o0 + sl * HD;
        const uint64_t dk0 = sdesc_sw128(sbase + C::kK, 16, 1024);
        const uint64_t dv0 = sdesc_sw128(sbase + C::kV, Q4 ? 16 : kBlk, 1024);
        constexpr uint32_t kVStep = Q4 ? 32 : 2048;      // from 16 keys of V to the next
        if (elect_one()) {
        Seg g;
        while (ok && walk.next(a, g)) {
            const int32_t tiles = seg_tiles<Q4>(g, walk.sv.tiles);
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
                    mma_ts(to, ts + b * 64 + k * 8, sdesc_at(dv0, st * C::kTile + k * kVStep), kIdPV, i > 0 || k > 0);
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
    }
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        if constexpr (Q4) asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        const int sl = (warp - kSoftWarp0) >> 2;
        const int r = tid - (kSoftWarp0 + 4 * sl) * 32;     // index in the group
        // a warp reads the quarter of the TMEM lanes of its number modulo 4
        const int row = ((warp & 3) << 5) + lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tm_s = tm_s0 + sl * 128 + lane_off, tm_o = tm_o0 + sl * HD + lane_off;
        float2* ml = reinterpret_cast<float2*>(sm + C::kMl);
        uint64_t* masks = reinterpret_cast<uint64_t*>(sm + C::kMask);     // new tokens that each one's rows admit
        uint8_t* bits = reinterpret_cast<uint8_t*>(misc + 16);            // and its mask's number of bits
        uint32_t it0 = 0, cnt = 0;            // ring index at the segment's start; this slot's key tiles so far
        bool ok = true;
        const int64_t part0 = walk.mark();
        uint32_t segs = 0;
        Seg g;
        while (walk.next(a, g)) {
            const SeqView& sv = walk.sv;
            const int32_t tiles = seg_tiles<Q4>(g, sv.tiles), t0 = seg_tile0<Q4>(g);
            named_sync(3, 256);               // the last segment's masks and statistics have been read
            if (sl == 0 && r < 64) {
                int n;
                masks[r] = admitted_tokens(a, g.bi, sv.nq, r, n);
                bits[r] = static_cast<uint8_t>(n);
            }
            if (sl == 0 && r == 0 && !a.whole)
                name_cut(a, part, walk.mark() == part0, walk.tile0_place(part, g), g.cost, g.bi, g.gk * blocks + g.blk,
                         a.c.h_kv * blocks, g.step0, g.steps, g.of, g.two ? W::kTwo : W::kOne);
            // this thread's row
            const int rr = g.blk * 256 + (g.two ? sl * 128 : 0) + row;
            const int tok = rr < R ? rr / a.group : 0;
            const int64_t h = g.gk * a.group + (rr - tok * a.group);
            const bool real = rr < R && tok < sv.nq;
            const uint16_t* qp = a.q + g.bi * a.q_stride[0] + tok * a.q_stride[1] + h * a.q_stride[2];
            float row_scale = a.scale_log2;
            if constexpr (Q4 && BF16) {
                // a bf16 row goes to f16 by the power of two that puts its largest magnitude between 2^14 and 2^15
                uint32_t most = 0;
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) {
                    const uint4 x = real ? ld_nc_v4(qp + c * 8) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) most = max(most, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
                }
                const QScale4 q = q_scale4(most);
                row_scale = fmaxf(a.scale_log2 * q.back, 1e-38f);     // (not 0: masked scores are -inf)
                if (g.two || sl == 0)
#pragma unroll
                    for (int c = 0; c < HD / 8; ++c) {
                        const uint4 x = real ? ld_nc_v4(qp + c * 8) : make_uint4(0u, 0u, 0u, 0u);
                        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = unpack2<true>(w[k]);
                            w[k] = pack2<false>(f.x * q.mul, f.y * q.mul);
                        }
                        *reinterpret_cast<uint4*>(sm + C::kQ + sl * C::kQTile + swizzled<kQBlk>(row, c)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
            } else if (g.two || sl == 0) {
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) {
                    const uint4 x = real ? ld_nc_v4(qp + c * 8) : make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(sm + C::kQ + sl * C::kQTile + swizzled<kQBlk>(row, c)) = x;
                }
            }
            fence_proxy_async_smem();
            const uint64_t scale2 = pair(__float_as_uint(row_scale), __float_as_uint(row_scale));
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
                        see[w] = Q4 ? column_order4(s) : s;
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
                const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * row_scale;
                const bool up = top > m + kMoves<MB>;
                if (__any_sync(0xffffffffu, up)) {
                    const float f = !up ? 1.f : m == -INFINITY ? 0.f : ex2_approx(m - (top - kBelow<MB>));
                    l *= f;
                    m = up ? top - kBelow<MB> : m;
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
                        w8[e] = pack2<MB>(p0, p1);
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
            const int64_t slot = blockIdx.x * int64_t(2) + (walk.mark() == part0 ? 0 : 1);
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
                    if constexpr (Q4) {
                        // column n of a V that lies transposed: feature (n / 8) of the run of lane row n % 8
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int f = k * (HD / 8) + cb * 4, n = lane_row4(k);
                            const float y[4] = {x[n], x[8 + n], x[16 + n], x[24 + n]};
                            if (!whole) {
                                *reinterpret_cast<float4*>(a.part_o + (slot * 256 + urow) * HD + f) = make_float4(y[0], y[1], y[2], y[3]);
                                if (f == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * 256 + urow) * 2) = make_float2(top, sum);
                            } else {
                                store_row<BF16, 4>(a, g.bi, tok, h, f, tok < sv.nq, top, sum, y);
                            }
                        }
                    } else if (!whole) {
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

template <int HD, bool BF16, bool POS, bool Q4>
cudaError_t launch_tile_pos(const CacheTileArgs& a, cudaStream_t s)
{
    auto kern = cache_fwd_tile_kernel<HD, BF16, POS, Q4>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, TileCfg<HD, Q4>::kBytes, allowed);
    if (e != cudaSuccess) return e;
    if constexpr (Q4) {
        // the warpgroups' registers add up to those of 128 a thread: a kernel built with fewer would wait for more
        static std::atomic<int> regs{0};
        if (regs.load(std::memory_order_relaxed) == 0) {
            cudaFuncAttributes attr;
            const cudaError_t q = cudaFuncGetAttributes(&attr, kern);
            if (q != cudaSuccess) return q;
            regs.store(attr.numRegs, std::memory_order_relaxed);
        }
        if (regs.load(std::memory_order_relaxed) < 128) return cudaErrorLaunchOutOfResources;
    }
    kern<<<a.f.parts, kTileThreads<Q4>, TileCfg<HD, Q4>::kBytes, s>>>(a);
    return cudaGetLastError();
}

template <bool Q4>
cudaError_t launch_tiles_typed(const CacheTileArgs& a, int dtype, cudaStream_t s)
{
    const bool pos = a.f.c.positions != nullptr && a.f.window_left >= 0;
    if (a.f.c.d == 128) {
        if (dtype == SDPA_BF16) return pos ? launch_tile_pos<128, true, true, Q4>(a, s) : launch_tile_pos<128, true, false, Q4>(a, s);
        return pos ? launch_tile_pos<128, false, true, Q4>(a, s) : launch_tile_pos<128, false, false, Q4>(a, s);
    }
    if (dtype == SDPA_BF16) return pos ? launch_tile_pos<64, true, true, Q4>(a, s) : launch_tile_pos<64, true, false, Q4>(a, s);
    return pos ? launch_tile_pos<64, false, true, Q4>(a, s) : launch_tile_pos<64, false, false, Q4>(a, s);
}

}  // namespace

}  // namespace swa
