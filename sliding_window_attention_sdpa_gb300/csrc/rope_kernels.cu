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
// exact to 2^-24 of one for every position: fp32 products are off by whole radians
// far into a text.
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

enum RopeMode { kNeighbours, kHalves, kAnyHalves };

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = y.x;
            f[2 * i + 1] = y.y;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
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

#ifndef V_FU
#define V_FU 4
#define V_FO 3
#define V_BU 2
#define V_BO 2
#endif
template <int HD, bool BF16, RopeMode MODE, bool NORM, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, BWD ? V_BO : V_FO) rope_kernel(const __grid_constant__ RopeArgs a)
{
    constexpr int LK = HD / 8, HP = 32 / LK;       // lanes of a head, heads at a time
    constexpr int U = BWD ? V_BU : V_FU;           // of those on their way together
    constexpr int PAIRS = HD / 64;                 // pairs of a lane when angles are computed
    __shared__ float2 sh_turn[kRopeWarps][HD / 2];
    __shared__ float sh_row[MODE == kAnyHalves ? kRopeWarps : 1][MODE == kAnyHalves ? HP : 1][HD];
    __shared__ float sh_dw[BWD && NORM ? kRopeWarps : 1][2][HD];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = lane % LK, sub = lane / LK, f0 = c * 8;
    const int half = a.rot / 2;

    uint64_t turn[PAIRS];      // of the lane's pairs: a position's fraction of a turn, times 2^64
    int axis[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        const int p = lane + 32 * i;
        turn[i] = 0;
        axis[i] = 0;
        if (p < half) {
            const double x = static_cast<double>(a.freq[p]) * 0.15915494309189533577;     // 1 / (2 pi)
            turn[i] = __double2ull_rn((x - floor(x)) * 18446744073709551616.0);
            if (a.axis) axis[i] = min(max(a.axis[p], 0), a.n_axes - 1);
        }
    }
    // the lane's features of the weights, and of their gradient's sum, of the tensor in hand (queries first, then keys)
    float w[8], dw[8];
    int n = -1;
    auto flush = [&]() {
        if constexpr (BWD && NORM) {
            // lanes with the same features
#pragma unroll
            for (int e = 0; e < 8; ++e) {
#pragma unroll
                for (int o = LK; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
                if (sub == 0) sh_dw[warp][n][f0 + e] = dw[e];
            }
        }
    };
    if constexpr (BWD && NORM)
        for (int i = tid; i < kRopeWarps * 2 * HD; i += kRopeThreads) (&sh_dw[0][0][0])[i] = 0.f;
    __syncthreads();

    const int64_t units_q = a.rows * a.splits[0], units = units_q + a.rows * a.splits[1];
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp; u < units; u += static_cast<int64_t>(gridDim.x) * kRopeWarps) {
        const int now = u >= units_q ? 1 : 0;
        const RopeTensor& t = a.t[now];
        if (now != n) {
            if (n >= 0) flush();
            n = now;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[e] = 0.f;
                w[e] = 1.f;
                if constexpr (NORM) {
                    float v;
                    if (a.weight_f32) v = static_cast<const float*>(t.weight)[f0 + e];
                    else if constexpr (BF16) v = __bfloat162float(static_cast<const __nv_bfloat16*>(t.weight)[f0 + e]);
                    else v = __half2float(static_cast<const __half*>(t.weight)[f0 + e]);
                    w[e] = v + a.weight_offset;
                }
            }
        }
        const int64_t un = now ? u - units_q : u, row = a.splits[now] == 1 ? un : un / a.splits[now];
        const int first = static_cast<int>(un - row * a.splits[now]) * a.per_split, last = min(first + a.per_split, t.heads);
        const int64_t bi = a.s == a.rows ? 0 : row / a.s, j = row - bi * a.s;
        const bool real = a.seq_lens == nullptr || j < a.seq_lens[bi];
        // ---- the token's turns
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const int p = lane + 32 * i;
            if (p < half) {
                const int64_t pos = a.positions[axis[i] * a.rows + row];
                const int32_t part = static_cast<int32_t>((static_cast<uint64_t>(pos) * turn[i]) >> 32);
                float s, co;
                sincospif(static_cast<float>(part) * 0x1p-31f, &s, &co);
                sh_turn[warp][p] = make_float2(co * a.rot_scale, s * a.rot_scale);
            }
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int f = f0 + e;
            cs[e] = 1.f;
            sn[e] = 0.f;
            if (f < a.rot) {
                const bool hi = MODE == kNeighbours ? (e & 1) : f >= half;
                const float2 x = sh_turn[warp][MODE == kNeighbours ? f >> 1 : hi ? f - half : f];
                cs[e] = x.x;
                // the sign of the turn, and of the turn back
                sn[e] = hi != BWD ? x.y : -x.y;
            }
        }
        __syncwarp();
        // the lane that has the partners (halves: rot / 16 lanes on or back)
        const int with = MODE == kHalves ? (f0 < half ? lane + half / 8 : f0 < a.rot ? lane - half / 8 : lane) : lane;
        auto turned = [&](float (&y)[8]) {
            float p[8];
            if constexpr (MODE == kNeighbours) {
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = y[e ^ 1];
            } else if constexpr (MODE == kHalves) {
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = __shfl_sync(0xffffffffu, y[e], with);
            } else {
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) sh_row[warp][sub][f0 + e] = y[e];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int f = f0 + e;
                    p[e] = f < a.rot ? sh_row[warp][sub][f < half ? f + half : f - half] : 0.f;
                }
            }
            // (what is not rotated stays as it is, whatever its partner is)
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = f0 + e < a.rot ? fmaf(y[e], cs[e], p[e] * sn[e]) : y[e];
        };
        // ---- the heads
        const uint16_t* xp = t.x + bi * t.x_stride[0] + j * t.x_stride[1] + f0;
        const uint16_t* gp = t.g + bi * t.g_stride[0] + j * t.g_stride[1] + f0;
        uint16_t* op = t.o + bi * t.o_stride[0] + j * t.o_stride[1] + f0;
#pragma unroll 1
        for (int h = first; h < last; h += HP * U) {
            uint4 xr[U], gr[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int hh = h + k * HP + sub;
                const bool in = real && hh < last;
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                xr[k] = (!BWD || NORM) && in ? *reinterpret_cast<const uint4*>(xp + hh * t.x_stride[2]) : z;
                gr[k] = BWD && in ? *reinterpret_cast<const uint4*>(gp + hh * t.g_stride[2]) : z;
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int hh = h + k * HP + sub;
                if (h + k * HP >= last) break;
                float x[8], y[8], r = 1.f;
                unpack8<BF16>(xr[k], x);
                if constexpr (NORM) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                    r = rsqrtf(fmaf(head_sum<LK>(ss), 1.f / HD, a.eps));
                }
                if constexpr (!BWD) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = NORM ? x[e] * r * w[e] : x[e];
                    turned(y);
                } else {
                    unpack8<BF16>(gr[k], y);
                    turned(y);
                    if constexpr (NORM) {
                        float dot = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x[e] *= r;
                            dw[e] = fmaf(y[e], x[e], dw[e]);
                            y[e] *= w[e];
                            dot = fmaf(y[e], x[e], dot);
                        }
                        dot = head_sum<LK>(dot) * (1.f / HD);
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = r * fmaf(-x[e], dot, y[e]);
                    }
                }
                if (hh < last)
                    *reinterpret_cast<uint4*>(op + hh * t.o_stride[2]) = real ? pack8<BF16>(y) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
    if constexpr (BWD && NORM) {
        // the CTA's sums: its warps', in order
        if (n >= 0) flush();
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
    const int resident = 152 * (backward ? V_BO : V_FO);
    const int hp = 256 / a.d;
    // a warp for a token's queries and one for its keys, unless there are fewer of those than warps: then heads are shared out
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
