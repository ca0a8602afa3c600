// cache_fwd.cuh -- what the cache forward's kernels share: the sequence as its
// rows and keys, the line of tiles that is cut between CTAs, and the last step
// of a row.
#pragma once

#include "cache.cuh"
#include "ptx.cuh"

namespace swa {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t x)
{
    if constexpr (BF16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    const __half2 h = *reinterpret_cast<const __half2*>(&x);
    return __half22float2(h);
}

// Two fp32 values in one 64-bit register, and the packed arithmetic on them.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ float lo_of(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float hi_of(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

__device__ __forceinline__ float max3(float x, float y, float z)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// 16-byte chunk of a row of a swizzled tile whose 64-column blocks are BLK bytes.
template <uint32_t BLK>
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t chunk)
{
    return (chunk >> 3) * BLK + (row >> 3) * 1024 + (row & 7) * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// A box of 64 features (from c0) x the map's rows of one head of a page.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int head, int row,
                                        int page)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(head), "r"(row), "r"(page)
        : "memory");
}

// 16 bytes to shared memory; zeros (nothing read) if not `have`.
__device__ __forceinline__ void cp16(uint32_t dst, const uint16_t* src, bool have)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}

// The MMAs below are issued by one elected thread (elect.sync tells the
// compiler that the branch holds one): back to back 64 cycles each at N = 128,
// 48 (A from shared memory) or 32 (from TMEM) at N = 64, against 87, 71 and 52
// with the whole warp running the code and a predicate on the instruction.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

// After tmem_ld_wait: the values of a load that other work was put behind are
// used from here on (the compiler may not move that use before the wait).
__device__ __forceinline__ void loaded(uint32_t (&r)[32])
{
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                     "+r"(r[i + 6]), "+r"(r[i + 7])
                     :
                     : "memory");
}

// Whether the phase with the given parity has completed, without suspending the
// thread (try_wait may hold it for a while).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Arrives once on `bar` when this thread's MMAs so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// How far, in powers of two, a row's reference lies below the score that set it, and how far above the reference a
// score may lie before it moves. f16 has no exponent below 2^-24: with its largest P at 2^7 to 2^15 (of 65504), keys
// down to 2^-31 of the heaviest keep a P, of 2^-21 all 11 bits of it (a reference at the score itself: 2^-24 and 2^-14).
// bf16 has fp32's exponents.
template <bool BF16>
constexpr float kBelow = BF16 ? 0.f : 7.f;
template <bool BF16>
constexpr float kMoves = 8.f + kBelow<BF16>;

// One sequence as the rows and keys of this call see it.
struct SeqView {
    int32_t len, nq;    // cached keys, new tokens
    int32_t first;      // first cached key in the window of a row at next_pos (the loads know the rows' own depths)
    int32_t lo;         // the same, rounded down to `align`
    int32_t new0;       // place of new token 0 in the line of keys (lo ... ), a multiple of 16 from lo
    int32_t tiles;
};

// tk keys a tile; align is a power of two, at least 16.
__device__ __forceinline__ SeqView seq_view(const CacheFwdArgs& a, int64_t bi, int tk, int align = 16)
{
    SeqView v;
    bool bad;
    v.len = cache_length(a.c, bi, bad);
    v.nq = a.s_q;
    if (a.seq_q_lens) {
        v.nq = a.seq_q_lens[bi];
        if (v.nq < 0 || v.nq > a.s_q) {
            set_status(a.c.status, SDPA_ERR_BAD_LENGTHS);
            v.nq = v.nq < 0 ? 0 : a.s_q;
        }
    }
    // without positions the window of a row at next_pos starts at len - W
    v.first = 0;
    if (a.window_left >= 0 && a.c.positions == nullptr) v.first = static_cast<int32_t>(imax64(0, v.len - a.window_left));
    v.lo = v.first & ~(align - 1);
    const int64_t cached = ((static_cast<int64_t>(v.len) + 15) & ~int64_t(15)) - v.lo;
    v.new0 = static_cast<int32_t>(cached);
    v.tiles = static_cast<int32_t>((cached + ((max(v.nq, 1) + 15) & ~15) + tk - 1) / tk);
    return v;
}

// The same of a cache in 4 bits: the line starts at a multiple of gk keys, and so
// do the new tokens behind it (at most gk of them).
__device__ __forceinline__ SeqView seq_view4(const CacheFwdArgs& a, int64_t bi, int tk, int gk)
{
    SeqView v = seq_view(a, bi, tk, gk);
    v.new0 = static_cast<int32_t>(((static_cast<int64_t>(v.len) + gk - 1) & ~static_cast<int64_t>(gk - 1)) - v.lo);
    v.tiles = (v.new0 + gk + tk - 1) / tk;
    return v;
}

// New token r's mask as it is given (r < nq), without the bits from nq on.
__device__ __forceinline__ uint64_t given_mask(const CacheFwdArgs& a, int64_t bi, int32_t nq, int r)
{
    const uint64_t in = nq == 64 ? ~0ull : (1ull << nq) - 1;
    return in & (a.tree ? static_cast<uint64_t>(a.tree[bi * a.s_q + r]) : (2ull << r) - 1);
}

// The new tokens that row r admits, and (`bits`) the number of its mask's bits,
// which is its position + 1 behind next_pos: none without its own bit, and none
// out of the window (a row only looks for those if it is deeper than the window).
__device__ __forceinline__ uint64_t admitted_tokens(const CacheFwdArgs& a, int64_t bi, int32_t nq, int r, int& bits)
{
    bits = 0;
    if (r >= nq) return 0;
    uint64_t m = given_mask(a, bi, nq, r);
    bits = __popcll(m);
    if (!((m >> r) & 1)) return 0;
    if (a.window_left >= 0 && bits > a.window_left)
        for (uint64_t rest = m; rest; rest &= rest - 1) {
            const int u = __ffsll(static_cast<long long>(rest)) - 1;
            if (bits - __popcll(given_mask(a, bi, nq, u)) > a.window_left) m &= ~(1ull << u);
        }
    return m;
}

// A cut unit leaves partials of its rows up to a multiple of this (the join's
// warps take as many).
constexpr int kPartialRows = 4;

// x / y of numbers that are not negative; in 32 bits where they fit (a division in 64 bits is a routine of some 100 cycles,
// and a kernel's start has several in a row).
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y)
{
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}

// The line of tiles: all sequences' units, cut evenly between the parts.
struct Line {
    int64_t total;
    __device__ __forceinline__ int64_t start(int64_t c, int64_t parts) const { return quotient(c * total, parts); }
    // the part that holds tile t
    __device__ __forceinline__ int64_t part_of(int64_t t, int64_t parts) const { return quotient((t + 1) * parts - 1, total); }
};

__device__ __forceinline__ int64_t warp_sum64(int64_t x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Sum of per-thread values over the CTA (every thread calls it).
template <int THREADS>
__device__ __forceinline__ int64_t block_sum64(int64_t x, int64_t* sh)
{
    x = warp_sum64(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    int64_t s = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) s += sh[i];
    return s;
}

// A CTA's part of the line: its tiles [at, end) (end 0: none), the sequence bi
// that holds the first one, and that tile's place among the sequence's.
struct Part {
    int64_t parts, at, end, bi, rem;
    Line line;
};

// Cuts the line of all sequences' tiles (tiles_of(i), each more than 0) into
// one part per CTA, fewer if there are fewer tiles; a part has LEAST places at
// least. Every thread calls it; sh has a place per warp, sh_at two.
template <int THREADS, int LEAST = 1, class F>
__device__ __forceinline__ Part find_part(int64_t b, F tiles_of, int64_t* sh, int64_t* sh_at)
{
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Part p{};
    const int64_t mine = tid < b ? tiles_of(tid) : 0;      // (of the first THREADS sequences, for both passes)
    int64_t s = mine;
    for (int64_t i = tid + THREADS; i < b; i += THREADS) s += tiles_of(i);
    p.line.total = block_sum64<THREADS>(s, sh);
    p.parts = imin64(gridDim.x, p.line.total / LEAST);
    if (blockIdx.x >= p.parts) return p;
    p.at = p.line.start(blockIdx.x, p.parts);
    p.end = p.line.start(blockIdx.x + 1, p.parts);
    int64_t before = 0;
    for (int64_t base = 0; base < b; base += THREADS) {
        const int64_t i = base + tid;
        const int64_t n = base == 0 ? mine : i < b ? tiles_of(i) : 0;
        int64_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        __syncthreads();
        if (lane == 31) sh[warp] = incl;
        __syncthreads();
        int64_t off = before;
        for (int w = 0; w < warp; ++w) off += sh[w];
        if (off + incl - n <= p.at && p.at < off + incl) {
            sh_at[0] = i;
            sh_at[1] = p.at - (off + incl - n);
        }
#pragma unroll
        for (int w = 0; w < W; ++w) before += sh[w];
        if (before > p.at) break;
    }
    __syncthreads();
    p.bi = sh_at[0];
    p.rem = sh_at[1];
    return p;
}

// A unit's place in the line: `cost` tiles' worth of its fixed cost (rows in,
// pipeline filled and drained, O out), then its tiles. A part that ends within
// the first has none of the unit's tiles. A segment: what a part has of a unit.
struct Segment {
    int64_t un;                 // the unit's number in its sequence
    int32_t tile0, n, line_n;   // first tile, tiles (0: none), places in the line
};

__device__ __forceinline__ Segment segment_at(int64_t rem, int32_t tiles, int32_t cost, int64_t left)
{
    Segment g;
    g.un = quotient(rem, tiles + cost);
    const int32_t y = static_cast<int32_t>(rem - g.un * (tiles + cost));
    g.tile0 = max(0, y - cost);
    g.line_n = static_cast<int32_t>(imin64(tiles + cost - y, left));
    g.n = max(0, y + g.line_n - cost) - g.tile0;
    return g;
}

// Names the join's work for a segment of g.n > 0 tiles of unit `un` (of
// `tiles`) of sequence bi; `pos0` is the place of the unit's tile 0 in the line
// (one thread calls it, for each segment of a part). `units`: per sequence. A
// tile may take w places; the part with the last of them has it.
__device__ __forceinline__ void name_cut(const CacheFwdArgs& a, const Part& p, bool first_of_part, int64_t pos0, int32_t cost,
                                         int64_t bi, int64_t un, int64_t units, int32_t tile0, int32_t n, int32_t tiles,
                                         int32_t w = 1)
{
    if (a.cut_by_unit ? tile0 != 0 : !first_of_part || tile0 == 0) return;
    CacheFwdCut cut{-1, 0, 0, 0, 0};
    const int64_t first = p.line.part_of(pos0 + w - 1, p.parts);
    if (n != tiles)
        cut = CacheFwdCut{bi, un, static_cast<int32_t>(first), static_cast<int32_t>(p.line.part_of(pos0 + int64_t(tiles) * w - 1, p.parts)),
                          p.line.start(first, p.parts) >= pos0 - cost * w ? 0 : 1};
    if (a.cut_by_unit) a.cuts[bi * units + un] = cut;
    // by part (a part's entry holds no cut at first): the one right behind the unit's first part names it
    else if (first + 1 == blockIdx.x) a.cuts[blockIdx.x] = cut;
}

// Finishes E features (from c) of a row: O and, with its first feature, LSE.
// `ref` is the reference of the row's exponentials (log2), -inf for no key. The
// maxima pass over NaN: of a row with NaN scores (a NaN in its q) the sum tells.
template <bool BF16, int E>
__device__ __forceinline__ void store_row(const CacheFwdArgs& a, int64_t bi, int tok, int64_t h, int c, bool in_rows,
                                          float ref, float sum, const float (&x)[E])
{
    const float top = sum == sum ? ref : sum;
    const bool sunk = a.sink != nullptr && in_rows;
    float mf = top, lt = sum;
    if (sunk) {
        const float sk = a.sink[h] * kLog2e;
        mf = fmaxf(top, sk);
        // (a sink of +inf is its own reference, and all of the sum)
        lt = (top == -INFINITY ? 0.f : sum * ex2_approx(top - mf)) + (sk == mf ? 1.f : ex2_approx(sk - mf));
    }
    const float mul = top == -INFINITY ? 0.f : ex2_approx(top - mf) / lt;
    uint16_t* o = a.o + bi * a.o_stride[0] + tok * a.o_stride[1] + h * a.o_stride[2] + c;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) w[e] = pack2<BF16>(x[2 * e] * mul, x[2 * e + 1] * mul);
    if constexpr (E == 8) *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (E == 4) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(o) = w[0];
    if (c == 0) {
        // a row without a key: the sink itself, or -inf
        const float lse = top == -INFINITY ? (sunk ? a.sink[h] : -INFINITY) : (mf + log2f(lt)) * kLn2;
        a.lse[(bi * a.h_q + h) * a.s_q + tok] = lse;
    }
}

}  // namespace swa
