// cache4_kernels.cu -- rows into a cache held in 4 bits, and cached rows of either
// kind out of it.
#include "cache4.cuh"
#include "cache_append.cuh"

namespace swa {

namespace {

// The 8 features of a 16-byte piece as fp32.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = to_float<BF16>(static_cast<uint16_t>(w[i]));
        f[2 * i + 1] = to_float<BF16>(static_cast<uint16_t>(w[i] >> 16));
    }
}

// 8 features of a block of 16 whose other half the neighbouring lane (^ 1) has, as codes c + 8; the block's scale byte.
template <bool BF16>
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint32_t (&c)[8])
{
    float f[8];
    unpack8<BF16>(x, f);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(f[i]) & 0x7fffffffu);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    float inv;
    const uint32_t scale = scale_byte4(most, inv);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = code4(f[i], inv);
    return scale;
}

}  // namespace

// A warp takes 2 (d = 64: 4) adjacent slots of a head at a time, a lane 8 features
// of K and of V.
template <int HD, bool BF16>
__global__ void __launch_bounds__(256) cache4_append_kernel(const CacheAppendArgs a)
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
        for (uint32_t u = warp; u < sets * h_kv; u += warps) {
            const uint32_t set = u / h_kv, g = u - set * h_kv;
            const uint32_t slot = (first + set) * KP + sub;
            const bool in = slot >= s0 && slot < s1;
            uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
            uint8_t *kg = nullptr, *vg = nullptr;       // the slot's group
            uint32_t row = 0;
            if (in) {
                const int32_t i = static_cast<int32_t>(slot) - p.len;
                const int64_t src = p.src0 + (a.index ? a.index[bi * a.n + i] : i);
                kx = ld_nc_v4(a.k + b0 * a.k_stride[0] + src * a.k_stride[1] + g * a.k_stride[2] + c * 8);
                vx = ld_nc_v4(a.v + b0 * a.v_stride[0] + src * a.v_stride[1] + g * a.v_stride[2] + c * 8);
                const int64_t page = cache_page(a.c, bi, slot, row);
                const int64_t at = static_cast<int64_t>(row >> 4) * Group4<HD>::kBytes;
                kg = reinterpret_cast<uint8_t*>(a.c.k) + page * a.c.k_stride[0] + g * a.c.k_stride[2] + at;
                vg = reinterpret_cast<uint8_t*>(a.c.v) + page * a.c.v_stride[0] + g * a.c.v_stride[2] + at;
            }
            const uint32_t x = row & 15;
            uint32_t q[8];
            const uint32_t ks = quantise8<BF16>(kx, q);
            const uint32_t kw = pack_half4(q[0], q[2], q[4], q[6]) | pack_half4(q[1], q[3], q[5], q[7]) << 16;
            const uint32_t vs = quantise8<BF16>(vx, q);
            const uint32_t v0 = pack_half4(q[0], q[1], q[2], q[3]), v1 = pack_half4(q[4], q[5], q[6], q[7]);
            // an even slot's lane writes both keys' first half words, the odd slot's the second ones
            const bool odd = slot & 1;
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, LK);
            const bool both = __shfl_xor_sync(0xffffffffu, in ? 1 : 0, LK) != 0 && in;
            if (!in) continue;
            *reinterpret_cast<uint32_t*>(kg + k4_word<HD>(x, c)) = kw;
            if (both) {
                *reinterpret_cast<uint32_t*>(vg + v4_half<HD>(x & ~1u, 2 * c + (odd ? 1 : 0))) =
                    odd ? other | v1 << 16 : v0 | other << 16;
            } else {
                *reinterpret_cast<uint16_t*>(vg + v4_half<HD>(x, 2 * c)) = static_cast<uint16_t>(v0);
                *reinterpret_cast<uint16_t*>(vg + v4_half<HD>(x, 2 * c + 1)) = static_cast<uint16_t>(v1);
            }
            if (c & 1) vg[v4_scale<HD>(x, c >> 1)] = static_cast<uint8_t>(vs);
            else kg[k4_scale<HD>(x, c >> 1)] = static_cast<uint8_t>(ks);
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

// Where an output row's key is: its sequence and slot, or slot -1 (zeros).
struct ReadRow {
    int64_t bi, slot;
};

__device__ __forceinline__ ReadRow read_row(const CacheReadArgs& a, int64_t r)
{
    ReadRow x;
    int64_t j, room;
    if (a.offsets) {
        // the last sequence that begins at or in front of the row
        int64_t lo = 0, hi = a.c.b;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (a.offsets[mid] <= r) lo = mid; else hi = mid;
        }
        x.bi = lo;
        j = r - a.offsets[lo];
        room = static_cast<int64_t>(a.offsets[lo + 1]) - a.offsets[lo];
        if (j < 0 || j >= room) {
            set_status(a.c.status, SDPA_ERR_BAD_LENGTHS);
            x.slot = -1;
            return x;
        }
    } else {
        x.bi = r / a.s;
        j = r - x.bi * a.s;
        room = a.s;
    }
    bool bad;
    const int64_t len = cache_length(a.c, x.bi, bad);
    const int64_t start = a.start ? a.start[x.bi] : 0, n = a.counts ? a.counts[x.bi] : room;
    if (start < 0 || start > len || n < 0 || n > room) set_status(a.c.status, SDPA_ERR_BAD_LENGTHS);
    x.slot = start >= 0 && j < n && start + j < len ? start + j : -1;
    return x;
}

}  // namespace

// A warp takes 2 (d = 64: 4) adjacent output rows of a head, a lane 8 features
// of K and of V.
template <int HD, bool BF16, bool Q4>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheReadArgs a)
{
    constexpr uint32_t LK = HD / 8, KP = 32 / LK;
    const uint32_t lane = threadIdx.x & 31, c = lane % LK, sub = lane / LK;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int64_t units = (a.rows + KP - 1) / KP * a.c.h_kv;
    if (blockIdx.x == 0 && a.offsets) {
        // (rows of no sequence are found below; here offsets that do not ascend from 0 to the end)
        bool ok = a.offsets[0] == 0 && a.offsets[a.c.b] == a.rows;
        for (int64_t i = threadIdx.x; i < a.c.b; i += blockDim.x) ok = ok && a.offsets[i] <= a.offsets[i + 1];
        if (!ok) set_status(a.c.status, SDPA_ERR_BAD_LENGTHS);
    }
    for (int64_t u = warp; u < units; u += warps) {
        const int64_t set = u / a.c.h_kv, g = u - set * a.c.h_kv, r = set * KP + sub;
        if (r >= a.rows) continue;
        const ReadRow x = read_row(a, r);
        uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
        uint32_t row = 0;
        const int64_t page = x.slot < 0 ? -1 : cache_page(a.c, x.bi, static_cast<uint32_t>(x.slot), row);
        if (page >= 0) {
            if constexpr (Q4) {
                const int64_t at = static_cast<int64_t>(row >> 4) * Group4<HD>::kBytes;
                const uint8_t* kg = reinterpret_cast<const uint8_t*>(a.c.k) + page * a.c.k_stride[0] + g * a.c.k_stride[2] + at;
                const uint8_t* vg = reinterpret_cast<const uint8_t*>(a.c.v) + page * a.c.v_stride[0] + g * a.c.v_stride[2] + at;
                const uint32_t i = row & 15;
                const uint32_t kw = *reinterpret_cast<const uint32_t*>(kg + k4_word<HD>(i, c));
                const uint2 vw = *reinterpret_cast<const uint2*>(vg + (v4_half<HD>(i, 2 * c) & ~3u));
                const uint32_t ks = kg[k4_scale<HD>(i, c >> 1)], vs = vg[v4_scale<HD>(i, c >> 1)];
                uint32_t f[4];
                values4(kw, scale4<0x0404>(ks), f);
                kx = make_uint4(f[0], f[1], f[2], f[3]);
                // V: this key's halves, paired feature by feature
                const uint32_t two = __byte_perm(vw.x, vw.y, i & 1 ? 0x7632 : 0x5410);
                values4(two, scale4<0x0404>(vs), f);
                vx = make_uint4(__byte_perm(f[0], f[1], 0x5410), __byte_perm(f[2], f[3], 0x5410),
                                __byte_perm(f[0], f[1], 0x7632), __byte_perm(f[2], f[3], 0x7632));
                if constexpr (BF16) {
                    auto conv = [](uint32_t h) -> uint32_t {
                        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h));
                        uint32_t z;
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(z) : "f"(y.y), "f"(y.x));
                        return z;
                    };
                    kx = make_uint4(conv(kx.x), conv(kx.y), conv(kx.z), conv(kx.w));
                    vx = make_uint4(conv(vx.x), conv(vx.y), conv(vx.z), conv(vx.w));
                }
            } else {
                kx = ld_nc_v4(a.c.k + page * a.c.k_stride[0] + row * a.c.k_stride[1] + g * a.c.k_stride[2] + c * 8);
                vx = ld_nc_v4(a.c.v + page * a.c.v_stride[0] + row * a.c.v_stride[1] + g * a.c.v_stride[2] + c * 8);
            }
        }
        const int64_t b0 = a.offsets ? 0 : r / a.s, j = a.offsets ? r : r - b0 * a.s;
        *reinterpret_cast<uint4*>(a.k + b0 * a.k_stride[0] + j * a.k_stride[1] + g * a.k_stride[2] + c * 8) = kx;
        *reinterpret_cast<uint4*>(a.v + b0 * a.v_stride[0] + j * a.v_stride[1] + g * a.v_stride[2] + c * 8) = vx;
    }
}

namespace {

template <int HD, bool BF16, bool Q4>
cudaError_t launch_read(const CacheReadArgs& a, cudaStream_t s)
{
    constexpr int64_t KP = 256 / HD;
    const int64_t units = (a.rows + KP - 1) / KP * a.c.h_kv;
    const int64_t ctas = imin64((units + 7) / 8, 152 * 8);
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
