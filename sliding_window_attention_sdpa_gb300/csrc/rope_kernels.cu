// rope_kernels.cu -- each head's RMS norm and position rotation in one pass, and
// its backward pass.
//
// Both are bound by reading their inputs and writing their outputs once. A warp
// takes a token's queries or keys (few tokens: a share of the heads): it computes
// the token's cosines and sines, which all heads have in common, puts them into its
// shared memory and keeps those of its lanes' features in registers; then head
// after head, 8 features (16 bytes) a lane, 2 heads at a time (d = 64: 4).
//
// Rotation: feature f becomes y_f cos + y_partner (+-) sin, with the sign kept
// in the lane's sine and (1, 0) for features that are not rotated. The partner of
// neighbouring pairs is in the lane itself; that of halves is in another lane at the
// same place if rot is a multiple of 16, else it is found through shared memory.
//
// Angles: a frequency is held as its 64-bit fraction of a turn a position, so that
// the product with a 32-bit position modulo 2^64 is the angle's fraction of a turn,
// exact to 2^-24 of one for every position and both signs (|freq| up to 2^50): fp32
// products are off by whole radians far into a text.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "../../include/sdpa_bwd.h"
#include "rope_internal.h"
#include "seq.cuh"

namespace swa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

// CTAs on an SM: more leave too few registers for two batches (backward with 3: 413 us against 288 for 38 k packed rows of
// 54 heads), fewer too few loads on their way
template <bool BWD>
constexpr int kRopeOcc = BWD ? 2 : 3;

enum RopeMode { kNeighbours, kHalves, kAnyHalves };

// Two fp32 values in one 64-bit register, and packed arithmetic on them.
__device__ __forceinline__ uint64_t pair2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lo2(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float hi2(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint64_t unpack2(uint32_t w)
{
    if constexpr (BF16) return pair2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pair2(y.x, y.y);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(uint64_t x)
{
    uint32_t w;
    if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi2(x)), "f"(lo2(x)));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi2(x)), "f"(lo2(x)));
    return w;
}

// Sum over the LK lanes of a head, the same in each.
template <int LK>
__device__ __forceinline__ float head_sum(float x)
{
#pragma unroll
    for (int o = 1; o < LK; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

}  // namespace

template <int HD, bool BF16, RopeMode MODE, bool NORM, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, kRopeOcc<BWD>) rope_kernel(const __grid_constant__ RopeArgs a)
{
    constexpr int LK = HD / 8, HP = 32 / LK;       // lanes of a head, heads at a time
    constexpr int U = 2;                           // of those in a batch: one is on its way while one is worked on
    constexpr int PAIRS = HD / 64;                 // pairs of a lane when angles are computed
    __shared__ __align__(16) float2 sh_turn[kRopeWarps][HD / 2];
    __shared__ __align__(16) float sh_w[2][NORM ? HD : 1];       // weights
    __shared__ uint64_t sh_frac[HD / 2];
    __shared__ float sh_row[MODE == kAnyHalves ? kRopeWarps : 1][MODE == kAnyHalves ? HP : 1][HD];
    __shared__ float sh_dw[BWD && NORM ? kRopeWarps : 1][2][HD];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = lane % LK, sub = lane / LK, f0 = c * 8;
    const int half = a.rot / 2;

    // a pair's fraction of a turn a position, times 2^64 (once for the CTA: arithmetic in 64 bits is slow, and 33 k packed
    // rows of 54 heads took 173 us, not 170, with each warp for itself)
    if (tid < half) {
        // f / (2 pi) as a product and what it lost (1 / (2 pi) in two doubles): one double's last place, times a position of
        // 2^31, is 2^-24 of a turn at f = 1 and more above
        constexpr double kInv = 0x1.45f306dc9c883p-3, kInvLow = -0x1.6b01ec5417056p-57;
        const double f = a.freq[tid], x = f * kInv, low = fma(f, kInv, -x) + f * kInvLow;
        // (signed remainders of the nearest whole number: exact, where that of a small negative x from the one below, 1 - |x|, is
        // rounded at 2^-54, 2^-23 of a turn at 2^31 positions)
        sh_frac[tid] = static_cast<uint64_t>(__double2ll_rn((x - rint(x)) * 0x1p64)) + static_cast<uint64_t>(__double2ll_rn((low - rint(low)) * 0x1p64));
    }
    // the lane's features of the weights' gradient, of the tensor in hand (queries first, then keys)
    uint64_t dw[4];
    auto flush = [&](int n) {
        if constexpr (BWD && NORM) {
            // lanes with the same features
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x = e & 1 ? hi2(dw[e / 2]) : lo2(dw[e / 2]);
#pragma unroll
                for (int o = LK; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (sub == 0) sh_dw[warp][n][f0 + e] = x;
            }
        }
    };
    if constexpr (NORM)
        for (int i = tid; i < 2 * HD; i += kRopeThreads) {
            const int f = i % HD;
            const void* wt = a.t[i / HD].weight;
            float v = 0.f;
            if (wt == nullptr) continue;
            if (a.weight_f32) v = static_cast<const float*>(wt)[f];
            else if constexpr (BF16) v = __bfloat162float(static_cast<const __nv_bfloat16*>(wt)[f]);
            else v = __half2float(static_cast<const __half*>(wt)[f]);
            sh_w[i / HD][f] = v + a.weight_offset;
        }
    int axis[PAIRS];           // of the lane's pairs
#pragma unroll
    for (int i = 0; i < PAIRS; ++i)
        axis[i] = a.axis && lane + 32 * i < half ? min(max(a.axis[lane + 32 * i], 0), a.n_axes - 1) : 0;
    __syncthreads();
    uint64_t turn[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) turn[i] = lane + 32 * i < half ? sh_frac[lane + 32 * i] : 0;

    const int64_t units_q = a.rows * a.splits[0], units = units_q + a.rows * a.splits[1];
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRopeWarps;
    auto row_of = [&](int64_t u) -> int64_t {
        const int32_t sp = a.splits[u >= units_q ? 1 : 0];
        const int64_t un = u >= units_q ? u - units_q : u;
        return sp == 1 ? un : un >> 32 ? un / sp : static_cast<uint32_t>(un) / static_cast<uint32_t>(sp);
    };
    // positions of the lane's pairs, a unit ahead
    int32_t pos[PAIRS];
    auto fetch_pos = [&](int64_t u) {
        if (u >= units) return;
        const int64_t row = row_of(u);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i)
            if (lane + 32 * i < half) pos[i] = a.positions[axis[i] * a.rows + row];
    };
    int64_t u = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
    fetch_pos(u);
    // the units of one tensor (a function each, so that its addresses and strides are constants)
    auto tensor = [&](auto which, int64_t end) {
    constexpr int now = decltype(which)::value;
    const RopeTensor& t = a.t[now];
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[e] = 0;
#pragma unroll 1
    for (; u < end; u += stride) {
        const int64_t un = u - (now ? units_q : 0), row = row_of(u);
        const int first = static_cast<int>(un - row * a.splits[now]) * a.per_split, last = min(first + a.per_split, t.heads);
        const int64_t bi = a.s == a.rows ? 0 : static_cast<uint32_t>(row) / static_cast<uint32_t>(a.s), j = row - bi * a.s;
        const bool real = a.seq_lens == nullptr || j < a.seq_lens[bi];
        if (!real) {
            // padding: zeros, and nothing read
            fetch_pos(u + stride);
            uint16_t* op = t.o + bi * t.o_stride[0] + j * t.o_stride[1] + f0;
            for (int h = first + sub; h < last; h += HP) *reinterpret_cast<uint4*>(op + h * t.o_stride[2]) = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        // ---- the heads' loads: a batch of U sets is on its way while the one before is worked on, the first one during the
        // token's turns
        const int64_t head0 = first + sub;
        [[maybe_unused]] const uint16_t* xp = t.x + bi * t.x_stride[0] + j * t.x_stride[1] + head0 * t.x_stride[2] + f0;
        [[maybe_unused]] const uint16_t* gp = t.g + bi * t.g_stride[0] + j * t.g_stride[1] + head0 * t.g_stride[2] + f0;
        uint16_t* op = t.o + bi * t.o_stride[0] + j * t.o_stride[1] + head0 * t.o_stride[2] + f0;
        uint4 xa[U], ga[U], xb[U], gb[U];
        auto load = [&](int h, uint4 (&xr)[U], uint4 (&gr)[U]) {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const bool in = h + k * HP + sub < last;
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                if constexpr (!BWD || NORM) {
                    xr[k] = in ? *reinterpret_cast<const uint4*>(xp) : z;
                    xp += HP * t.x_stride[2];
                }
                if constexpr (BWD) {
                    gr[k] = in ? *reinterpret_cast<const uint4*>(gp) : z;
                    gp += HP * t.g_stride[2];
                }
            }
        };
        load(first, xa, ga);
        // ---- the token's turns
        uint64_t cs[4], sn[4];
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const int p = lane + 32 * i;
            if (p < half) {
                const int32_t part = static_cast<int32_t>((static_cast<uint64_t>(static_cast<int64_t>(pos[i])) * turn[i]) >> 32);
                float s, co;
                sincospif(static_cast<float>(part) * 0x1p-31f, &s, &co);
                sh_turn[warp][p] = make_float2(co * a.rot_scale, s * a.rot_scale);
            }
        }
        __syncwarp();
        [[maybe_unused]] const bool on = f0 < a.rot;                     // (halves of a multiple of 8: the lane's features are alike)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // features f and f + 1: cosines, and sines with the sign of the turn (or of the turn back)
            const int f = f0 + 2 * e;
            cs[e] = pair2(1.f, 1.f);
            sn[e] = 0;
            if constexpr (MODE == kNeighbours) {
                if (f < a.rot) {
                    const float2 x = sh_turn[warp][f >> 1];
                    cs[e] = pair2(x.x, x.x);
                    sn[e] = BWD ? pair2(x.y, -x.y) : pair2(-x.y, x.y);
                }
            } else if constexpr (MODE == kHalves) {
                if (on) {
                    const bool hi = f0 >= half;
                    const float4 x = *reinterpret_cast<const float4*>(&sh_turn[warp][hi ? f - half : f]);
                    cs[e] = pair2(x.x, x.z);
                    sn[e] = hi != BWD ? pair2(x.y, x.w) : pair2(-x.y, -x.w);
                }
            } else {
                float c2[2] = {1.f, 1.f}, s2[2] = {0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (f + k < a.rot) {
                        const bool hi = f + k >= half;
                        const float2 x = sh_turn[warp][hi ? f + k - half : f + k];
                        c2[k] = x.x;
                        s2[k] = hi != BWD ? x.y : -x.y;
                    }
                cs[e] = pair2(c2[0], c2[1]);
                sn[e] = pair2(s2[0], s2[1]);
            }
            if constexpr (NORM && !BWD) {
                // (with the weights of the features and of their partners)
                auto partner = [&](int k) -> int {
                    return k >= a.rot ? k : MODE == kNeighbours ? k ^ 1 : k < half ? k + half : k - half;
                };
                const float2 w = *reinterpret_cast<const float2*>(&sh_w[now][f]);
                cs[e] = mul2(cs[e], pair2(w.x, w.y));
                sn[e] = mul2(sn[e], pair2(sh_w[now][partner(f)], sh_w[now][partner(f + 1)]));
            }
        }
        [[maybe_unused]] uint64_t w[4];
        if constexpr (NORM && BWD)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = *reinterpret_cast<const float2*>(&sh_w[now][f0 + 2 * e]);
                w[e] = pair2(x.x, x.y);
            }
        __syncwarp();
        fetch_pos(u + stride);
        // the lane that has the partners (halves: rot / 16 lanes on or back)
        [[maybe_unused]] const int with = MODE == kHalves && on ? (f0 < half ? lane + half / 8 : lane - half / 8) : lane;
        [[maybe_unused]] const bool part = a.rot < HD;
        // the partners' values; 0 where there is none, so that nothing of another feature comes in
        auto partners = [&](const uint4& raw, const uint64_t (&y)[4], uint64_t (&p)[4]) {
            if constexpr (MODE == kNeighbours) {
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = part && f0 + 2 * e >= a.rot ? 0 : pair2(hi2(y[e]), lo2(y[e]));
            } else if constexpr (MODE == kHalves) {
                const uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t z = __shfl_sync(0xffffffffu, v[e], with);
                    p[e] = unpack2<BF16>(part && !on ? 0u : z);
                }
            } else {
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sh_row[warp][sub][f0 + 2 * e] = lo2(y[e]);
                    sh_row[warp][sub][f0 + 2 * e + 1] = hi2(y[e]);
                }
                __syncwarp();
                auto at = [&](int f) -> float { return f < a.rot ? sh_row[warp][sub][f < half ? f + half : f - half] : 0.f; };
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = pair2(at(f0 + 2 * e), at(f0 + 2 * e + 1));
            }
        };
        auto work = [&](int h, const uint4 (&xr)[U], const uint4 (&gr)[U]) {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (h + k * HP >= last) break;
                [[maybe_unused]] const uint32_t xw[4] = {xr[k].x, xr[k].y, xr[k].z, xr[k].w};
                [[maybe_unused]] const uint32_t gw[4] = {gr[k].x, gr[k].y, gr[k].z, gr[k].w};
                [[maybe_unused]] uint64_t x[4], y[4], p[4];
                [[maybe_unused]] float r = 1.f;
                if constexpr (!BWD || NORM)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = unpack2<BF16>(xw[e]);
                if constexpr (NORM) {
                    uint64_t ss = mul2(x[0], x[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) ss = fma2(x[e], x[e], ss);
                    r = rsqrtf(fmaf(head_sum<LK>(lo2(ss) + hi2(ss)), 1.f / HD, a.eps));
                }
                [[maybe_unused]] const uint64_t r2 = pair2(r, r);
                if constexpr (!BWD) {
                    // y = r (x w cos + x' w' sin): the weights are in the cosines and sines
                    partners(xr[k], x, p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = fma2(p[e], sn[e], mul2(x[e], cs[e]));
                        if constexpr (NORM) y[e] = mul2(y[e], r2);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = unpack2<BF16>(gw[e]);
                    partners(gr[k], y, p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = fma2(p[e], sn[e], mul2(y[e], cs[e]));
                    if constexpr (NORM) {
                        // y = u r w; dx = y - x r^2 mean(y x)
                        uint64_t dot = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            y[e] = mul2(y[e], r2);
                            dw[e] = fma2(y[e], x[e], dw[e]);
                            y[e] = mul2(y[e], w[e]);
                            dot = fma2(y[e], x[e], dot);
                        }
                        // (of a head of zeros r^2 may be beyond fp32, if eps is below 2^-128)
                        const float sum = head_sum<LK>(lo2(dot) + hi2(dot)), z = sum == 0.f ? 0.f : sum * (1.f / HD) * -(r * r);
                        const uint64_t z2 = pair2(z, z);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = fma2(x[e], z2, y[e]);
                    }
                }
                if (h + k * HP + sub < last)
                    *reinterpret_cast<uint4*>(op) =
                        make_uint4(pack2<BF16>(y[0]), pack2<BF16>(y[1]), pack2<BF16>(y[2]), pack2<BF16>(y[3]));
                op += HP * t.o_stride[2];
            }
        };
#pragma unroll 1
        for (int h = first; h < last; h += 2 * HP * U) {
            load(h + HP * U, xb, gb);
            work(h, xa, ga);
            load(h + 2 * HP * U, xa, ga);
            work(h + HP * U, xb, gb);
        }
    }
    flush(now);
    };
    tensor(std::integral_constant<int, 0>{}, units_q);
    tensor(std::integral_constant<int, 1>{}, units);
    if constexpr (BWD && NORM) {
        // the CTA's sums: its warps', in order
        __syncthreads();
        for (int i = tid; i < 2 * HD; i += kRopeThreads) {
            float x = 0.f;
#pragma unroll
            for (int k = 0; k < kRopeWarps; ++k) x += (&sh_dw[k][0][0])[i];
            a.partial[static_cast<int64_t>(blockIdx.x) * 2 * HD + i] = x;
        }
        grid_dep_launch();
    }
}

// The CTAs' sums of a weight gradient, in order: a CTA takes 32 features, a warp
// every eighth partial.
template <int HD>
__global__ void __launch_bounds__(256) rope_sum_kernel(const __grid_constant__ RopeArgs a)
{
    __shared__ float sh[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = blockIdx.x * 32 + lane, n = i / HD;
    grid_dep_wait();
    float x = 0.f;
#pragma unroll 8
    for (int k = warp; k < a.ctas; k += 8) x += a.partial[static_cast<int64_t>(k) * 2 * HD + i];
    sh[warp][lane] = x;
    __syncthreads();
    if (warp > 0 || a.t[n].heads == 0) return;
    x = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) x += sh[k][lane];
    a.t[n].dw[i - n * HD] = x;
}

void rope_plan(RopeArgs& a, bool backward)
{
    const int resident = 152 * (backward ? kRopeOcc<true> : kRopeOcc<false>);
    const int hp = 256 / a.d;
    // a warp for a token's queries and one for its keys, unless there are fewer of those than warps: then heads are shared
    // out (48 + 6 heads of d = 128, one token 6.4 us, 12 for a warp that has all; 64 tokens 7.0 and 12.8)
    const int64_t warps = static_cast<int64_t>(resident) * kRopeWarps;
    const int64_t sets = (static_cast<int64_t>(a.t[0].heads) + hp - 1) / hp + (static_cast<int64_t>(a.t[1].heads) + hp - 1) / hp;
    const int64_t shares = a.rows > 0 ? imax64(1, imin64(warps / a.rows, sets)) : 1;
    const int64_t most = (a.t[0].heads > a.t[1].heads ? a.t[0].heads : a.t[1].heads) + hp - 1;
    a.per_split = static_cast<int32_t>(imin64(most / hp, (sets + shares - 1) / shares) * hp);
    if (shares <= 2) a.per_split = static_cast<int32_t>(most / hp * hp);
    int64_t units = 0;
    for (int n = 0; n < 2; ++n) {
        a.splits[n] = (a.t[n].heads + a.per_split - 1) / a.per_split;
        units += a.rows * a.splits[n];
    }
    a.ctas = static_cast<int32_t>(imax64(1, imin64(resident, (units + kRopeWarps - 1) / kRopeWarps)));
}

namespace {

template <int HD, bool BF16, RopeMode MODE, bool NORM>
cudaError_t launch_norm(const RopeArgs& a, bool backward, cudaStream_t s)
{
    if (!backward) {
        rope_kernel<HD, BF16, MODE, NORM, false><<<a.ctas, kRopeThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    rope_kernel<HD, BF16, MODE, NORM, true><<<a.ctas, kRopeThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !NORM) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * HD / 32);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_sum_kernel<HD>, a);
}

template <int HD, bool BF16>
cudaError_t launch_mode(const RopeArgs& a, bool backward, cudaStream_t s)
{
    const bool norm = a.t[0].weight != nullptr;
    if (a.interleaved || a.rot == 0)
        return norm ? launch_norm<HD, BF16, kNeighbours, true>(a, backward, s) : launch_norm<HD, BF16, kNeighbours, false>(a, backward, s);
    // a lane's partner features are another lane's own 8 (16 x 4096 tokens, all of d = 128 turned, 170 us; through shared
    // memory, as for halves that end inside 8 features, 335; 35,000 rows of 54 heads, 92 of 128 features so 231, all of them 171)
    if (a.rot % 16 == 0)
        return norm ? launch_norm<HD, BF16, kHalves, true>(a, backward, s) : launch_norm<HD, BF16, kHalves, false>(a, backward, s);
    return norm ? launch_norm<HD, BF16, kAnyHalves, true>(a, backward, s) : launch_norm<HD, BF16, kAnyHalves, false>(a, backward, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, bool backward, cudaStream_t s)
{
    if (a.d == 64) return dtype == SDPA_BF16 ? launch_mode<64, true>(a, backward, s) : launch_mode<64, false>(a, backward, s);
    return dtype == SDPA_BF16 ? launch_mode<128, true>(a, backward, s) : launch_mode<128, false>(a, backward, s);
}

}  // namespace swa
