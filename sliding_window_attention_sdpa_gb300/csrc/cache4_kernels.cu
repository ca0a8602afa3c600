// cache4_kernels.cu -- rows into a cache held in 4 bits, and cached rows of either
// kind out of it.
#include "cache4.cuh"
#include "cache_append.cuh"

namespace swa {

namespace {

// 8 features of a block of 16 whose other half the neighbouring lane (^ 1) has, as codes c + 8 (see code4_2); the
// block's scale byte.
template <bool BF16>
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint32_t (&c)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    // the largest magnitude, a NaN if there is one
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        if constexpr (BF16) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
        else asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
    }
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t most = BF16 ? m << 16 : __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(m))));
    float inv;
    bool wide;
    const uint32_t scale = scale_byte4(most, inv, wide);
    uint64_t inv2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(inv2) : "f"(inv));
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = to_float<BF16>(static_cast<uint16_t>(w[i]));
        f[2 * i + 1] = to_float<BF16>(static_cast<uint16_t>(w[i] >> 16));
    }
    if (__any_sync(0xffffffffu, wide)) {
        // (8 s and 7 s are exact; where s is 0 the codes are anyway)
        const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(scale << 7)));
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(f[i], -8.f * s), 7.f * s);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t x2;
        asm("mov.b64 %0, {%1, %2};" : "=l"(x2) : "f"(f[2 * i]), "f"(f[2 * i + 1]));
        x2 = code4_2(x2, inv2);
        c[2 * i] = static_cast<uint32_t>(x2);
        c[2 * i + 1] = static_cast<uint32_t>(x2 >> 32);
    }
    return scale;
}

}  // namespace

// A warp takes 2 (d = 64: 4) adjacent slots, a lane 8 features of K and of V, head
// after head. Bound by its operations, some 125 for 16 values, with 73 % of the issue
// slots busy: prompts of 16 sequences (68,000 rows of 8 kv-heads, d = 128) 84 us, of
// 52 for their bytes. Two heads' loads are on their way, with 4 CTAs on an SM: one head
// takes 12 us more, four with 2 CTAs 20; looking rows up for each head took 123.
template <int HD, bool BF16>
__global__ void __launch_bounds__(256, 4) cache4_append_kernel(const CacheAppendArgs a)
{
    constexpr uint32_t LK = HD / 8, KP = 32 / LK;      // lanes of a key, keys of a warp
    const int64_t bi = blockIdx.x;
    const AppendPlan p = append_plan(a, bi);
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    // this CTA's slots, from a multiple of 16
    const int64_t lo = (p.len & ~15) + static_cast<int64_t>(blockIdx.y) * a.rows_per_cta;
    const int64_t s0 = imax64(lo, p.len), s1 = imin64(lo + a.rows_per_cta, static_cast<int64_t>(p.len) + imax64(p.n, 0));
    if (p.n > 0 && s0 < s1) {
        const uint32_t h_kv = static_cast<uint32_t>(a.c.h_kv), c = lane % LK, sub = lane / LK;
        const uint32_t first = static_cast<uint32_t>(s0) / KP, sets = static_cast<uint32_t>(s1 - 1) / KP - first + 1;
        const int64_t b0 = a.thd ? 0 : bi;
        // a warp takes all heads of its slots (which are looked up once then), a share of them where there are few slots
        // (48 sequences of 1 to 5 rows, 8 heads of d = 64, 6.2 us, 9.4 without shares)
        const uint32_t splits = max(1u, min(h_kv, warps / sets)), per = (h_kv + splits - 1) / splits;
        constexpr int U = 2;                            // heads whose loads are on their way together
        for (uint32_t u = warp; u < sets * splits; u += warps) {
            const uint32_t set = u / splits, h0 = (u - set * splits) * per, h1 = min(h0 + per, h_kv);
            const uint32_t slot = (first + set) * KP + sub;
            const bool in = slot >= s0 && slot < s1;
            const bool both = __shfl_xor_sync(0xffffffffu, in ? 1 : 0, LK) != 0 && in;
            const uint16_t *kp = nullptr, *vp = nullptr;
            uint8_t *kg = nullptr, *vg = nullptr;       // the slot's group of head 0
            uint32_t row = 0;
            if (in) {
                const int32_t i = static_cast<int32_t>(slot) - p.len;
                const int64_t src = p.src0 + (a.index ? a.index[bi * a.n + i] : i);
                kp = a.k + b0 * a.k_stride[0] + src * a.k_stride[1] + c * 8;
                vp = a.v + b0 * a.v_stride[0] + src * a.v_stride[1] + c * 8;
                const int64_t page = cache_page(a.c, bi, slot, row);
                const int64_t at = static_cast<int64_t>(row >> 4) * Group4<HD>::kBytes;
                kg = reinterpret_cast<uint8_t*>(a.c.k) + page * a.c.k_stride[0] + at;
                vg = reinterpret_cast<uint8_t*>(a.c.v) + page * a.c.v_stride[0] + at;
            }
            const uint32_t x = row & 15;
            const bool odd = slot & 1;
            // an even slot's lane writes both keys' first half words, the odd slot's the second ones; an even piece's lane the
            // scale of K's block, the odd piece's that of V's
            uint8_t* kw_to = kg + k4_word<HD>(x, c);
            uint8_t* vw_to = vg + (both ? v4_half<HD>(x & ~1u, 2 * c + (odd ? 1 : 0)) : v4_half<HD>(x, 2 * c));
            uint8_t* s_to = c & 1 ? vg + v4_scale<HD>(x, c >> 1) : kg + k4_scale<HD>(x, c >> 1);
            if (in) {
                kp += h0 * a.k_stride[2];
                vp += h0 * a.v_stride[2];
                kw_to += h0 * a.c.k_stride[2];
                vw_to += h0 * a.c.v_stride[2];
                s_to += h0 * (c & 1 ? a.c.v_stride[2] : a.c.k_stride[2]);
            }
            const int64_t s_step = c & 1 ? a.c.v_stride[2] : a.c.k_stride[2];
#pragma unroll 1
            for (uint32_t h = h0; h < h1; h += U) {
                uint4 kx[U], vx[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const bool load = in && h + k < h1;
                    kx[k] = load ? ld_nc_v4(kp) : make_uint4(0u, 0u, 0u, 0u);
                    vx[k] = load ? ld_nc_v4(vp) : make_uint4(0u, 0u, 0u, 0u);
                    kp += a.k_stride[2];
                    vp += a.v_stride[2];
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    if (h + k >= h1) break;
                    uint32_t q[8];
                    const uint32_t ks = quantise8<BF16>(kx[k], q);
                    const uint32_t even4[4] = {q[0], q[2], q[4], q[6]}, odd4[4] = {q[1], q[3], q[5], q[7]};
                    const uint32_t kw = pack_word4(even4, odd4);
                    const uint32_t vs = quantise8<BF16>(vx[k], q);
                    const uint32_t lo4[4] = {q[0], q[1], q[2], q[3]}, hi4[4] = {q[4], q[5], q[6], q[7]};
                    const uint32_t vw = pack_word4(lo4, hi4);       // both half words of this key
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, vw, LK);
                    if (in) {
                        *reinterpret_cast<uint32_t*>(kw_to) = kw;
                        if (both) {
                            *reinterpret_cast<uint32_t*>(vw_to) = odd ? __byte_perm(other, vw, 0x7632) : __byte_perm(vw, other, 0x5410);
                        } else {
                            *reinterpret_cast<uint16_t*>(vw_to) = static_cast<uint16_t>(vw);
                            *reinterpret_cast<uint16_t*>(vw_to + 4) = static_cast<uint16_t>(vw >> 16);
                        }
                        *s_to = static_cast<uint8_t>(c & 1 ? vs : ks);
                    }
                    kw_to += a.c.k_stride[2];
                    vw_to += a.c.v_stride[2];
                    s_to += s_step;
                }
            }
        }
        const uint32_t nr = static_cast<uint32_t>(s1 - s0);
        for (uint32_t u = threadIdx.x; u < nr * h_kv; u += blockDim.x) {
            const uint32_t g = u / nr;
            const int64_t slot = s0 + (u - g * nr), at = (bi * a.c.h_kv + g) * a.c.cap + slot;
            if (a.c.positions) a.c.positions[at] = a.c.next_pos[bi] + static_cast<int32_t>(slot - p.len);
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

cudaError_t launch_cache4_append(const CacheAppendArgs& a0, int dtype, cudaStream_t s)
{
    CacheAppendArgs a = a0;
    const int64_t most = a.index ? a.n : a.s;
    if (a.c.b == 0) return cudaSuccess;
    const int64_t per_row = a.c.h_kv * (a.c.d / 8);
    int64_t rows = most * per_row <= 4096 ? most + 15 : 2048 / per_row;
    rows = imax64(imax64(rows, most / 2048), (most + 15) / 65535 + 1);
    rows = (rows + 15) & ~int64_t(15);
    a.rows_per_cta = static_cast<int32_t>(rows);
    const dim3 grid(static_cast<unsigned>(a.c.b), static_cast<unsigned>(imax64(1, (most + 15 + rows - 1) / rows)));
    const bool bf16 = dtype == SDPA_BF16;
    if (a.c.d == 64) (bf16 ? cache4_append_kernel<64, true> : cache4_append_kernel<64, false>)<<<grid, 256, 0, s>>>(a);
    else (bf16 ? cache4_append_kernel<128, true> : cache4_append_kernel<128, false>)<<<grid, 256, 0, s>>>(a);
    if (grid.y > 1) return launch_cache_advance(a, s);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- read

namespace {

// The sequence of an output row, kept for the rows that follow: its first output row and the one behind its last, and
// of row `first` + j the slot start + j for j < n.
struct ReadSeq {
    int64_t bi, first, end, start, n;
};

__device__ __forceinline__ ReadSeq read_seq(const CacheReadArgs& a, int64_t r)
{
    ReadSeq x;
    if (a.offsets) {
        // the last sequence that begins at or in front of the row
        int64_t lo = 0, hi = a.c.b;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (a.offsets[mid] <= r) lo = mid; else hi = mid;
        }
        x.bi = lo;
        x.first = a.offsets[lo];
        x.end = a.offsets[lo + 1];
        if (r < x.first || r >= x.end) {        // (a row of no sequence: looked up alone)
            set_status(a.c.status, SDPA_ERR_BAD_LENGTHS);
            x.first = r;
            x.end = r + 1;
            x.n = 0;
            return x;
        }
    } else {
        x.bi = r / a.s;
        x.first = x.bi * a.s;
        x.end = x.first + a.s;
    }
    bool bad;
    const int64_t len = cache_length(a.c, x.bi, bad), room = x.end - x.first;
    x.start = a.start ? a.start[x.bi] : 0;
    x.n = a.counts ? a.counts[x.bi] : room;
    if (x.start < 0 || x.start > len || x.n < 0 || x.n > room) set_status(a.c.status, SDPA_ERR_BAD_LENGTHS);
    x.n = x.start < 0 ? 0 : imin64(x.n, len - x.start);
    return x;
}

}  // namespace

// A warp takes 2 (d = 64: 4) adjacent output rows, all heads or a share of them, a
// lane 8 features of K and of V. Bound by writing, mostly: 12 sequences of 16484 rows
// of 6 kv-heads, d = 128 in f16 141 us, 5.5 TB/s of its bytes.
template <int HD, bool BF16, bool Q4>
__global__ void __launch_bounds__(256, 4) cache_read_kernel(const __grid_constant__ CacheReadArgs a)
{
    constexpr uint32_t LK = HD / 8, KP = 32 / LK;
    constexpr int U = 3;                                // heads whose loads are on their way together
    const uint32_t lane = threadIdx.x & 31, c = lane % LK, sub = lane / LK;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int32_t h_kv = static_cast<int32_t>(a.c.h_kv);
    const int64_t units = (a.rows + KP - 1) / KP * a.splits;
    // a warp's units follow one another: the look-ups of a sequence and of a page serve many rows
    const int64_t u0 = warp * a.per_warp, u1 = imin64(units, u0 + a.per_warp);
    ReadSeq x;
    x.first = x.end = 0;
    int64_t page = -1, page0 = -1;                      // of slots [page0, page0 + page_size)
    if (blockIdx.x == 0 && a.offsets) {
        // (rows of no sequence are found below; here offsets that do not ascend from 0 to the end)
        bool ok = a.offsets[0] == 0 && a.offsets[a.c.b] == a.rows;
        for (int64_t i = threadIdx.x; i < a.c.b; i += blockDim.x) ok = ok && a.offsets[i] <= a.offsets[i + 1];
        if (!ok) set_status(a.c.status, SDPA_ERR_BAD_LENGTHS);
    }
    for (int64_t u = u0; u < u1; ++u) {
        const int64_t set = a.splits == 1 ? u : u / a.splits, r = set * KP + sub;
        const int32_t h0 = static_cast<int32_t>(u - set * a.splits) * a.per_split, h1 = min(h0 + a.per_split, h_kv);
        if (r >= a.rows) continue;
        if (r < x.first || r >= x.end) {
            x = read_seq(a, r);
            page0 = -1;
        }
        const bool held = r - x.first < x.n;            // (else zeros)
        const int64_t slot = x.start + r - x.first;
        if (held && (page0 < 0 || slot < page0 || slot >= page0 + a.c.page_size)) {
            uint32_t at;
            page = cache_page(a.c, x.bi, static_cast<uint32_t>(slot), at);
            page0 = slot - at;
        }
        const bool there = held && page >= 0;
        const uint32_t row = held ? static_cast<uint32_t>(slot - page0) : 0;
        const int64_t b0 = a.offsets ? 0 : x.bi, j = a.offsets ? r : r - x.first;
        uint16_t* ko = a.k + b0 * a.k_stride[0] + j * a.k_stride[1] + c * 8;
        uint16_t* vo = a.v + b0 * a.v_stride[0] + j * a.v_stride[1] + c * 8;
        if constexpr (Q4) {
            const uint32_t i = row & 15;
            const int64_t at = static_cast<int64_t>(row >> 4) * Group4<HD>::kBytes;
            const uint8_t* kp = reinterpret_cast<const uint8_t*>(a.c.k) + page * a.c.k_stride[0] + at;
            const uint8_t* vp = reinterpret_cast<const uint8_t*>(a.c.v) + page * a.c.v_stride[0] + at;
            const uint32_t kw_at = k4_word<HD>(i, c), ks_at = k4_scale<HD>(i, c >> 1);
            const uint32_t vw_at = v4_half<HD>(i, 2 * c) & ~3u, vs_at = v4_scale<HD>(i, c >> 1);
#pragma unroll 1
            for (int32_t h = h0; h < h1; h += U) {
                uint32_t kw[U], ks[U], vs[U];
                uint2 vw[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    kw[k] = ks[k] = vs[k] = 0u;
                    vw[k] = make_uint2(0u, 0u);
                    if (there && h + k < h1) {
                        const uint8_t* kg = kp + (h + k) * a.c.k_stride[2];
                        const uint8_t* vg = vp + (h + k) * a.c.v_stride[2];
                        kw[k] = *reinterpret_cast<const uint32_t*>(kg + kw_at);
                        vw[k] = *reinterpret_cast<const uint2*>(vg + vw_at);
                        ks[k] = kg[ks_at];
                        vs[k] = vg[vs_at];
                    }
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    if (h + k >= h1) break;
                    // V: this key's half words, whose features go to the low and the high half of a register
                    const uint32_t two = __byte_perm(vw[k].x, vw[k].y, i & 1 ? 0x7632 : 0x5410);
                    uint32_t f[4], g[4];
                    if constexpr (BF16) {
                        auto scale = [](uint32_t b, uint32_t& n24) -> uint32_t {
                            const __nv_bfloat162 s = __float2bfloat162_rn(__half2float(__ushort_as_half(static_cast<uint16_t>(b << 7))));
                            const __nv_bfloat162 n = __hmul2(s, __float2bfloat162_rn(-24.f));
                            n24 = *reinterpret_cast<const uint32_t*>(&n);
                            return *reinterpret_cast<const uint32_t*>(&s);
                        };
                        uint32_t n24;
                        uint32_t s = scale(ks[k], n24);
                        values4_bf16(kw[k], s, n24, f);
                        s = scale(vs[k], n24);
                        values4_bf16(two, s, n24, g);
                    } else {
                        values4(kw[k], scale4<0x0404>(ks[k]), f);
                        values4(two, scale4<0x0404>(vs[k]), g);
                    }
                    *reinterpret_cast<uint4*>(ko + (h + k) * a.k_stride[2]) = make_uint4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<uint4*>(vo + (h + k) * a.v_stride[2]) =
                        make_uint4(__byte_perm(g[0], g[1], 0x5410), __byte_perm(g[2], g[3], 0x5410),
                                   __byte_perm(g[0], g[1], 0x7632), __byte_perm(g[2], g[3], 0x7632));
                }
            }
        } else {
            const uint16_t* kp = a.c.k + page * a.c.k_stride[0] + row * a.c.k_stride[1] + c * 8;
            const uint16_t* vp = a.c.v + page * a.c.v_stride[0] + row * a.c.v_stride[1] + c * 8;
#pragma unroll 1
            for (int32_t h = h0; h < h1; h += U) {
                uint4 kx[U], vx[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const bool in = there && h + k < h1;
                    kx[k] = in ? ld_nc_v4(kp + (h + k) * a.c.k_stride[2]) : make_uint4(0u, 0u, 0u, 0u);
                    vx[k] = in ? ld_nc_v4(vp + (h + k) * a.c.v_stride[2]) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    if (h + k >= h1) break;
                    *reinterpret_cast<uint4*>(ko + (h + k) * a.k_stride[2]) = kx[k];
                    *reinterpret_cast<uint4*>(vo + (h + k) * a.v_stride[2]) = vx[k];
                }
            }
        }
    }
}

namespace {

template <int HD, bool BF16, bool Q4>
cudaError_t launch_read(const CacheReadArgs& a0, cudaStream_t s)
{
    CacheReadArgs a = a0;
    constexpr int64_t KP = 256 / HD;
    // a warp takes all heads of its rows (which are looked up once then), a share of them where there are fewer rows than
    // warps that fit (4 x 128 rows, 8 heads of d = 64, 5.6 us, 10.3 without shares)
    const int64_t sets = (a.rows + KP - 1) / KP, most = 152 * 48;
    const int64_t splits = imax64(1, imin64(a.c.h_kv, most / sets));
    a.per_split = static_cast<int32_t>((a.c.h_kv + splits - 1) / splits);
    a.splits = static_cast<int32_t>((a.c.h_kv + a.per_split - 1) / a.per_split);
    // (a warp's sets follow one another, 4 of them: 12 x 16484 rows of 6 heads 142 us; 16 of them 167, one 149)
    const int64_t units = sets * a.splits;
    a.per_warp = imax64(1, imin64(4, units / most));
    const int64_t ctas = ((units + a.per_warp - 1) / a.per_warp + 7) / 8;
    cache_read_kernel<HD, BF16, Q4><<<static_cast<unsigned>(ctas), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_read(const CacheReadArgs& a, int dtype, cudaStream_t s)
{
    if (a.c.bits != 4) return a.c.d == 64 ? launch_read<64, false, false>(a, s) : launch_read<128, false, false>(a, s);
    if (dtype == SDPA_BF16) return a.c.d == 64 ? launch_read<64, true, true>(a, s) : launch_read<128, true, true>(a, s);
    return a.c.d == 64 ? launch_read<64, false, true>(a, s) : launch_read<128, false, true>(a, s);
}

}  // namespace swa
