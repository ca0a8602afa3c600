// cache4_fwd.cu -- attention of a few new tokens per sequence over a cache held in 4
// bits and over each other: up to 16 rows of a kv-head in a unit.
//
// Rows, units, the line of tiles and its cut into parts are those of cache_fwd.cu. A
// step of a CTA is 256 keys, 64 for each of four warps; a fifth warp brings it, 64
// keys (or as many as a page has in one run) a bulk copy, into a ring of two or more
// steps. The new tokens, in their 16-bit form, are the unit's last 64 keys; one warp
// takes them from global memory.
//
// The values come out of the codes as f16, exactly (cache4.cuh), straight into the
// operand registers of m16n8k16:
//   S^T = K Q^T     M = 16 keys, N = 8 rows
//   O^T += V^T P^T  M = 16 features, N = 8 rows, K = 16 keys
// with the k indexes of both products mapped to features and keys as the groups hold
// them. Q and the new tokens are f16 as well: a bf16 row of Q is first multiplied by the
// power of two that puts its largest magnitude between 2^14 and 2^15 (what then lies
// below f16's last place is 2^-39 of that), and its scores by the inverse.
// P is f16 for either type, with references as cache_fwd.cu has them for f16; for f16
// output its remainder is a second product. For bf16 output it is left out: f16's half
// step is an eighth of O's own, and adds in squares (errors against 64 bits relative to
// O's norm: 0.0016 to 0.0017, those of an fp32 form rounded once).
//
// Reading is 9/16 byte a feature, 25 us for 12 sequences of 16484 keys of 6 kv-heads, d =
// 128 (8 rows: 47 us, 3.6 TB/s). Without the arithmetic the same kernel takes 42 us: 6 us
// pass before the first keys are there, 6 in the join's launch and the join. With it,
// no unit is near its rate (ALU 39 %, fma 28 %, matrix unit 20 %, DRAM 47 % of the time), and
// warps wait for operations that have just been issued. A ring for each warp instead
// (three steps, no fifth warp: the copies' issue takes a warp some 600 cycles a step)
// was as fast there, and took 55 us against 44 for 64 ragged sequences; twice as many
// warps with half the step, 30 % more instructions, 50 us against 47.
#include <type_traits>

#include "cache4.cuh"
#include "cache_fwd.cuh"

namespace swa {

namespace {

constexpr int kWarps4 = 4;                          // that compute; one more brings the keys
constexpr int kThreads4 = 32 * (kWarps4 + 1);
constexpr int kStep4 = 64, kGroups4 = kStep4 / 16;  // keys, groups of a warp's step
constexpr int kTile4 = kWarps4 * kStep4;            // keys of a CTA's step

template <int HD, int NT>
struct Rows4Cfg {
    static constexpr int kOcc = 2;
    static constexpr int kSub = HD == 128 && NT == 2 ? 2 : 4;            // groups whose scores are in registers together
    static constexpr uint32_t kHalf = kGroups4 * Group4<HD>::kBytes;     // a warp's K of a step
    static constexpr uint32_t kStage = 2 * kWarps4 * kHalf;              // the CTA's K, then its V
    static constexpr int kStages = static_cast<int>(110 * 1024 / kStage);
    static constexpr uint32_t kBytes = kStages * kStage;
};

__device__ __forceinline__ uint32_t movm_trans4(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a sum of 0 to begin with.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

}  // namespace

template <int HD, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads4, Rows4Cfg<HD, NT>::kOcc) cache4_fwd_rows_kernel(const __grid_constant__ CacheTileArgs qa)
{
    const CacheFwdArgs& a = qa.f;
    using C = Rows4Cfg<HD, NT>;
    constexpr int ST = C::kStages;
    constexpr bool SPLIT = !BF16;
    constexpr int GK = kStep4, KG = kGroups4, TK = kTile4, OKW = GK / 32;
    constexpr int KW = HD / 32;        // words of a lane, key and tensor
    constexpr int MT = HD / 16;        // feature tiles of O^T
    constexpr int ROWS = 8 * NT;
    constexpr int PAD = HD + 4;
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ __align__(8) uint64_t sh_full[ST], sh_empty[ST];
    float (*sh_o)[ROWS][PAD] = reinterpret_cast<float (*)[ROWS][PAD]>(dyn);     // at a unit's end
    static_assert(4 * ROWS * PAD * 4 <= C::kBytes, "the warps' O in the rings' place");
    __shared__ uint32_t sh_ok[ST][TK / 32];            // per stage: which keys count,
    __shared__ uint32_t sh_all[ST];                    // and whether all of them do
    __shared__ float sh_m[4][ROWS], sh_l[4][ROWS];
    __shared__ uint64_t sh_mask[64];       // new tokens that each one's rows admit
    __shared__ int32_t sh_bits[64];        // and its mask's number of bits
    __shared__ uint32_t sh_used[2];        // new tokens that some row admits
    __shared__ int64_t sh_sum[kThreads4 / 32], sh_at[2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int kappa = 4 * (g >> 1) + (g & 1);
    const int R = a.s_q * a.group;
    const int blocks = (R + ROWS - 1) / ROWS;
    const int64_t units = a.c.h_kv * blocks;      // per sequence
    auto view = [&](int64_t i) -> SeqView { return seq_view4(a, i, TK, GK); };

    __shared__ Part sh_part;
    __shared__ int64_t sh_done, sh_count;      // places of the part in the line: done, all
    {
        Part part{1, 0, 0, 0, 0, Line{0}};
        if (a.whole) {
            part.bi = blockIdx.x / units;
            part.end = view(part.bi).tiles;
            part.rem = (blockIdx.x - part.bi * units) * (part.end + a.unit_cost) + a.unit_cost;
        } else {
            part = find_part<kThreads4>(a.c.b, [&](int64_t i) { return (view(i).tiles + a.unit_cost) * units; }, sh_sum, sh_at);
            if (tid == 0 && !a.cut_by_unit) a.cuts[blockIdx.x].bi = -1;
            if (part.end == 0) {
                grid_dep_launch();
                return;
            }
        }
        if (tid == 0) {
            sh_part = part;
            sh_done = 0;
            sh_count = part.end - part.at;
        }
        __syncthreads();
    }

    if (tid < ST) {
        mbar_init(smem_u32(&sh_full[tid]), 1);
        mbar_init(smem_u32(&sh_empty[tid]), kWarps4);
    }
    fence_mbar_init();
    __syncthreads();
    const uint32_t full = smem_u32(&sh_full[0]), empty = smem_u32(&sh_empty[0]);
    uint32_t stage = 0, par = 0;      // the ring's stage to fill or to read, and its phase
    bool good = true;         // no wait has run out
    int64_t cur = -1;
    for (;;) {
        const int64_t bi = sh_part.bi, rem = sh_part.rem;
        const SeqView sv = view(bi);
        const Segment seg = segment_at(rem, sv.tiles, a.unit_cost, sh_count - sh_done);
        const int64_t un = seg.un;
        const int32_t tile0 = seg.tile0, nt = seg.n;
        if (nt == 0) break;                                 // the part ends before the unit's first tile
        const int64_t gk = blocks == 1 ? un : un / blocks;  // kv-head
        const int r0 = static_cast<int>(un - gk * blocks) * ROWS;
        const int64_t npos = a.c.next_pos ? a.c.next_pos[bi] : sv.len;
        const int32_t* kpos = a.c.positions && a.window_left >= 0 ? a.c.positions + (bi * a.c.h_kv + gk) * a.c.cap : nullptr;

        // a step is TK cached keys of the CTA, GK of each warp; the new tokens are the unit's last GK
        const int32_t cached = max(0, min(nt, (sv.new0 - tile0 * TK + TK - 1) / TK));    // steps with cached keys
        if (warp == kWarps4) {
            // ---- brings the steps: bulk copies of as many keys as a page and a warp's step allow, lane u K's copy u, lane
            // nu + u V's. Keys in front of every row's window are not fetched
            int32_t low_min = INT32_MIN;
            if (a.window_left >= 0) {
                int32_t shallow = 64;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    int bits;
                    if (admitted_tokens(a, bi, sv.nq, w * 32 + lane, bits)) shallow = min(shallow, bits);
                }
                low_min = static_cast<int32_t>(imax64(INT32_MIN, imin64(INT32_MAX,
                    npos + static_cast<int32_t>(__reduce_min_sync(0xffffffffu, shallow)) - 1 - a.window_left)));
            }
            const int ck = qa.box_rows, nu = TK / ck;           // keys of a copy, copies of a step's K (16 at most)
            const uint32_t bytes = ck / 16 * Group4<HD>::kBytes;
            const bool is_v = lane >= nu;
            const int mine = lane < 2 * nu ? lane % nu : 0;
            const int64_t st_page = is_v ? a.c.v_stride[0] : a.c.k_stride[0];
            const uint8_t* pool = reinterpret_cast<const uint8_t*>(is_v ? a.c.v : a.c.k) + gk * (is_v ? a.c.v_stride[2] : a.c.k_stride[2]);
            const uint32_t dst = smem_u32(dyn) + (is_v ? C::kStage / 2 : 0u) + mine * bytes;
            // the page of the lane's copy of a step
            auto fetch_entry = [&](int32_t s) -> int32_t {
                if (a.c.page_table == nullptr) return static_cast<int32_t>(bi);
                const int32_t j = sv.lo + (tile0 + s) * TK + mine * ck;
                return s < cached && j < sv.len ? cache_entry(a.c, bi, j) : 0;
            };
            // (the ring holds the last unit's O: its reads are done, and known to the copy engine)
            fence_proxy_async_smem();
            int32_t entry = fetch_entry(0);
            int32_t sent = 0;
#pragma unroll 1
            for (; sent < cached && good; ++sent) {
                const uint32_t bar = full + stage * 8;
                const int32_t j0 = sv.lo + (tile0 + sent) * TK, j = j0 + mine * ck;
                const bool paged = entry >= 0 && entry < a.c.n_pages;
                bool go = lane < 2 * nu;
                uint32_t copies = 2 * nu;
                good = __all_sync(0xffffffffu, mbar_wait(empty + stage * 8, par ^ 1, a.timeout_ns));
                if (!good) {
                    set_status(a.c.status, SDPA_ERR_TIMEOUT);
                    break;
                }
                // (every key of every copy is there and in reach, mostly)
                const bool all = __all_sync(0xffffffffu, paged && j + ck <= sv.len && kpos == nullptr && j >= low_min);
                if (!all) {
                    uint32_t any = 0;
#pragma unroll 1
                    for (int w = 0; w < TK / 32; ++w) {
                        const int32_t x = w * 32 + lane, jx = j0 + x;
                        const bool there = __shfl_sync(0xffffffffu, paged ? 1 : 0, x / ck) != 0;
                        bool in = jx < sv.len;
                        if (in && a.window_left >= 0) in = (kpos ? kpos[jx] : jx) >= low_min;
                        if (in && !there) set_status(a.c.status, SDPA_ERR_BOUNDS);
                        const uint32_t oks = __ballot_sync(0xffffffffu, in && there);
                        if (lane == 0) sh_ok[stage][w] = oks;
                        const int first = mine * ck - w * 32;                // the copy's keys in this word
                        if (ck >= 32 ? first <= 0 && first + ck > 0 : first >= 0 && first < 32)
                            any |= ck >= 32 ? oks : (oks >> first) & 0xffffu;
                    }
                    go = go && any != 0;
                    copies = __popc(__ballot_sync(0xffffffffu, go));
                }
                if (lane == 0) {
                    sh_all[stage] = all;
                    mbar_arrive_expect_tx(bar, copies * bytes);
                }
                __syncwarp();
                if (go && !(a.c.stall && sent == min(1, cached - 1))) {       // (test hook: a step that never comes)
                    const uint32_t row = a.c.page_table == nullptr ? j : cache_row(a.c, j);
                    bulk_load(dst + stage * C::kStage, pool + entry * st_page + static_cast<int64_t>(row >> 4) * Group4<HD>::kBytes, bytes,
                              bar);
                }
                entry = fetch_entry(sent + 1);
                if (++stage == ST) stage = 0, par ^= 1;
            }
            if (lane == 0 && !a.whole)
                name_cut(a, sh_part, sh_done == 0, sh_part.at + sh_done + seg.line_n - tile0 - nt, a.unit_cost, bi, un, units, tile0,
                         nt, sv.tiles);
            // what is on its way ends before the unit does, whatever wait has run out
            uint32_t q = stage, ph = par;
            for (int32_t r = 0; r < ST && r < sent; ++r) {
                if (q-- == 0) q = ST - 1, ph ^= 1;
                if (!mbar_wait(full + q * 8, ph, a.timeout_ns)) good = false;
            }
            good = __all_sync(0xffffffffu, good);
        } else {
            if (cur != bi) {
                if (tid < 64) {
                    int bits;
                    sh_mask[tid] = admitted_tokens(a, bi, sv.nq, tid, bits);
                    sh_bits[tid] = bits;
                }
                if (tid < 2) sh_used[tid] = 0;
                named_sync(1, 32 * kWarps4);
                if (warp < 2) {
                    const uint64_t m = sh_mask[tid];
                    const uint32_t lo32 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(m));
                    const uint32_t hi32 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(m >> 32));
                    if (lane == 0) {
                        atomicOr(&sh_used[0], lo32);
                        atomicOr(&sh_used[1], hi32);
                    }
                }
                named_sync(1, 32 * kWarps4);
                cur = bi;
            }
            auto step_x = [&](int32_t s) -> int32_t { return (tile0 + s) * TK + warp * GK; };
            // ---- rows: masks and windows (rows 2t, 2t + 1)
            int row_tok[NT][2];           // the row's token, -1: admits nothing
            int32_t row_low[NT][2];       // lowest position in the row's window
            int32_t low_max = INT32_MIN;  // the highest of them (this CTA's rows)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int rr = r0 + n * 8 + 2 * t + e;
                    const int tk = rr < R ? rr / a.group : 0;
                    const uint64_t m = rr < R ? sh_mask[tk] : 0;
                    row_tok[n][e] = m ? tk : -1;
                    row_low[n][e] = INT32_MIN;
                    if (a.window_left >= 0)
                        row_low[n][e] = static_cast<int32_t>(
                            imax64(INT32_MIN, imin64(INT32_MAX, npos + sh_bits[tk] - 1 - a.window_left)));
                    if (m) low_max = max(low_max, row_low[n][e]);
                }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) low_max = max(low_max, __shfl_xor_sync(0xffffffffu, low_max, o));

            // ---- Q in f16 (row g of each 8) and its factors (rows 2t, 2t + 1), while the first keys are on their way
            uint32_t q[NT][KW][4];
            float row_scale[NT][2];       // the row's scores to powers of two
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = r0 + n * 8 + g;
                const int tok = r / a.group;
                const bool real = r < R && tok < sv.nq;
                const uint16_t* qp = a.q + bi * a.q_stride[0] + tok * a.q_stride[1] +
                                     (gk * a.group + (r - tok * a.group)) * a.q_stride[2] + t * (HD / 4);
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    const uint4 x = real ? ld_nc_v4(qp + w * 8) : make_uint4(0u, 0u, 0u, 0u);
                    q[n][w][0] = x.x, q[n][w][1] = x.y, q[n][w][2] = x.z, q[n][w][3] = x.w;
                }
                float back = 1.f;
                if constexpr (BF16) {
                    uint32_t most = 0;
#pragma unroll
                    for (int w = 0; w < KW; ++w)
#pragma unroll
                        for (int j = 0; j < 4; ++j) most = max(most, max(q[n][w][j] & 0x7fffu, (q[n][w][j] >> 16) & 0x7fffu));
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    const QScale4 scale = q_scale4(most);
                    back = scale.back;
#pragma unroll
                    for (int w = 0; w < KW; ++w)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = unpack2<true>(q[n][w][j]);
                            q[n][w][j] = pack2<false>(f.x * scale.mul, f.y * scale.mul);
                        }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // (not 0: masked scores are -inf)
                    row_scale[n][e] = fmaxf(a.scale_log2 * __shfl_sync(0xffffffffu, back, (2 * t + e) * 4), 1e-38f);
                }
            }

            float o[NT][MT][4];
            float m[NT][2], l[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.f;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
            }

            // The softmax of G groups' masked scores: references, sums, and P^T as the second product's operands (hi, and
            // with SPLIT the remainders lo).
            auto softmax = [&](auto& sc, auto& hi, auto& lo) {
                constexpr int G = std::extent<std::remove_reference_t<decltype(sc)>, 1>::value;
                float mx[NT][2];
                bool up = false;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mx[n][0] = mx[n][1] = -INFINITY;
#pragma unroll
                    for (int u = 0; u < G; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[n][e & 1] = fmaxf(mx[n][e & 1], sc[n][u][e]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[n][e] *= row_scale[n][e];
                        up = up || mx[n][e] > m[n][e] + kMoves<false>;
                    }
                }
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float al[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = mx[n][e];
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
                            x = fmaxf(x - kBelow<false>, m[n][e]);
                            al[e] = m[n][e] == -INFINITY ? 0.f : ex2_approx(m[n][e] - x);
                            m[n][e] = x;
                            l[n][e] *= al[e];
                        }
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[n][i][e] *= al[e & 1];
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int u = 0; u < G; ++u) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // a masked score is -inf, its P is 0 (a row's reference is finite here, or 0)
                            p[e] = ex2_approx(fmaf(sc[n][u][e], row_scale[n][e & 1], m[n][e & 1] == -INFINITY ? 0.f : -m[n][e & 1]));
                            l[n][e & 1] += p[e];
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            hi[n][u][h] = pack2<false>(p[2 * h], p[2 * h + 1]);
                            if constexpr (SPLIT) {
                                const float2 f = unpack2<false>(hi[n][u][h]);
                                lo[n][u][h] = movm_trans4(pack2<false>(p[2 * h] - f.x, p[2 * h + 1] - f.y));
                            }
                            hi[n][u][h] = movm_trans4(hi[n][u][h]);
                        }
                    }
            };

#pragma unroll 1
            for (int32_t s = 0; s < cached; ++s) {
                const uint32_t st = stage;
                const uint8_t* step = dyn + st * C::kStage + warp * C::kHalf;
                if (good) {
                    good = __all_sync(0xffffffffu, mbar_wait(full + st * 8, par, a.timeout_ns));
                    if (!good) set_status(a.c.status, SDPA_ERR_TIMEOUT);
                }
                if (++stage == ST) stage = 0, par ^= 1;
                if (!good) continue;
                const int32_t x0 = step_x(s);
                const bool all = sh_all[st] != 0;
                uint32_t ok[OKW];
#pragma unroll
                for (int w = 0; w < OKW; ++w) ok[w] = all ? 0xffffffffu : sh_ok[st][warp * OKW + w];
                if (all || (ok[0] | ok[1]) != 0) {
                    constexpr int KS = C::kSub;
                    auto okw = [&](int u) -> uint32_t { return u < 2 ? ok[0] : ok[1]; };
                    static_assert(OKW == 2, "");
#pragma unroll 1
                    for (int u0 = 0; u0 < KG; u0 += KS) {
                        // S^T
                        float sc[NT][KS][4];
#pragma unroll
                        for (int u = 0; u < KS; ++u) {
                            const uint8_t* grp = step + (u0 + u) * Group4<HD>::kBytes;
                            const Words4<HD> kw = words4<HD>(grp, lane);
                            const uint32_t x = k_scales4<HD>(grp, lane);
                            Scale4 ks[2][HD / 64];
                            ks[0][0] = scale4<0x0404>(x);
                            if constexpr (HD == 128) {
                                ks[0][1] = scale4<0x1414>(x);
                                ks[1][0] = scale4<0x2424>(x), ks[1][1] = scale4<0x3434>(x);
                            } else {
                                ks[1][0] = scale4<0x1414>(x);
                            }
#pragma unroll
                            for (int w = 0; w < KW; ++w) {
                                uint32_t k0[4], k1[4];
                                values4(kw.w[0][w], ks[0][w / 2], k0);
                                values4(kw.w[1][w], ks[1][w / 2], k1);
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    if (w == 0) mma_f16_first(sc[n][u], k0[0], k1[0], k0[1], k1[1], q[n][w][0], q[n][w][1]);
                                    else mma_f16(sc[n][u], k0[0], k1[0], k0[1], k1[1], q[n][w][0], q[n][w][1]);
                                    mma_f16(sc[n][u], k0[2], k1[2], k0[3], k1[3], q[n][w][2], q[n][w][3]);
                                }
                            }
                        }
                        // masks (a step whose keys are all there and in every row's window needs none; rows that admit nothing
                        // are left out at the end)
                        const bool windowed = a.window_left >= 0 && (kpos != nullptr || sv.lo + x0 < low_max);
                        if (!all || windowed) {
#pragma unroll
                            for (int u = 0; u < KS; ++u)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const int x = (u0 + u) * 16 + kappa + 2 * h, j = sv.lo + x0 + x;
                                    const bool in = (okw(u0 + u) >> (x & 31)) & 1;
                                    const int32_t pos = in && kpos ? kpos[j] : j;
#pragma unroll
                                    for (int n = 0; n < NT; ++n)
#pragma unroll
                                        for (int e = 0; e < 2; ++e)
                                            if (!in || (windowed && pos < row_low[n][e])) sc[n][u][2 * h + e] = -INFINITY;
                                }
                        }
                        uint32_t hi[NT][KS][2], lo[NT][KS][2];
                        softmax(sc, hi, lo);
                        // O^T += V^T P^T
#pragma unroll
                        for (int u = 0; u < KS; ++u) {
                            const uint8_t* grp = step + C::kStage / 2 + (u0 + u) * Group4<HD>::kBytes;
                            const Words4<HD> vw = words4<HD>(grp, lane);
                            uint32_t x = v_scales4<HD>(grp, lane);
                            // what stands in the place of a key that does not count meets a P of 0: its scale has to be 0
                            if (!all) x &= (((okw(u0 + u) >> (((u0 + u) & 1) * 16 + 4 * t)) & 15) * 0x00204081u & 0x01010101u) * 255u;
                            const Scale4 v0 = scale4<0x1404>(x), v1 = scale4<0x3424>(x);
#pragma unroll
                            for (int w = 0; w < KW; ++w) {
                                uint32_t f0[4], f1[4];
                                values4(vw.w[0][w], v0, f0);
                                values4(vw.w[1][w], v1, f1);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int p = 0; p < 2; ++p) {
                                        mma_f16(o[n][w * 2 + p], f0[2 * p], f0[2 * p + 1], f1[2 * p], f1[2 * p + 1], hi[n][u][0],
                                                hi[n][u][1]);
                                        if constexpr (SPLIT)
                                            mma_f16(o[n][w * 2 + p], f0[2 * p], f0[2 * p + 1], f1[2 * p], f1[2 * p + 1], lo[n][u][0],
                                                lo[n][u][1]);
                                    }
                            }
                        }
                    }
                }
                // the stage is free when all four warps are done with it
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + st * 8);
            }

            // ---- the new tokens, 16 at a time, by the warp whose step they are (they begin with a warp's step, perhaps in a
            // CTA's step that has cached keys as well); of those that no row admits, which may hold anything, nothing is read
            const int32_t sn = (sv.new0 / GK - tile0 * kWarps4 - warp) / kWarps4;
            if (sv.new0 >= step_x(0) && sn < nt && step_x(sn) == sv.new0) {
                const uint16_t* kn = a.k + bi * a.k_stride[0] + gk * a.k_stride[2] + t * (HD / 4);
                const uint16_t* vn = a.v + bi * a.v_stride[0] + gk * a.v_stride[2] + g * (HD / 8);
#pragma unroll 1
                for (int w0 = 0; w0 < sv.nq; w0 += 16) {
                    float sc[NT][1][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n) sc[n][0][0] = sc[n][0][1] = sc[n][0][2] = sc[n][0][3] = 0.f;
                    auto there = [&](int w) -> bool { return w < sv.nq && (sh_used[w >> 5] >> (w & 31)) & 1; };
                    const bool in0 = there(w0 + kappa), in1 = there(w0 + kappa + 2);
#pragma unroll
                    for (int w = 0; w < KW; ++w) {
                        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                        const uint4 x = in0 ? ld_nc_v4(kn + (w0 + kappa) * a.k_stride[1] + w * 8) : z;
                        const uint4 y = in1 ? ld_nc_v4(kn + (w0 + kappa + 2) * a.k_stride[1] + w * 8) : z;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_f16(sc[n][0], to_f16x2<BF16>(x.x), to_f16x2<BF16>(y.x), to_f16x2<BF16>(x.y), to_f16x2<BF16>(y.y),
                                    q[n][w][0], q[n][w][1]);
                            mma_f16(sc[n][0], to_f16x2<BF16>(x.z), to_f16x2<BF16>(y.z), to_f16x2<BF16>(x.w), to_f16x2<BF16>(y.w),
                                    q[n][w][2], q[n][w][3]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint64_t rm = row_tok[n][e & 1] < 0 ? 0 : sh_mask[row_tok[n][e & 1]];
                            if (!((rm >> (w0 + kappa + 2 * (e >> 1))) & 1)) sc[n][0][e] = -INFINITY;
                        }
                    uint32_t hi[NT][1][2], lo[NT][1][2];
                    softmax(sc, hi, lo);
                    // V: 8 features at a time of the keys 4t .. 4t + 3
#pragma unroll
                    for (int c = 0; c < HD / 64; ++c) {
                        uint32_t v[4][4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int w = w0 + 4 * t + k;
                            const uint4 x = there(w) ? ld_nc_v4(vn + w * a.v_stride[1] + c * 8) : make_uint4(0u, 0u, 0u, 0u);
                            v[k][0] = to_f16x2<BF16>(x.x), v[k][1] = to_f16x2<BF16>(x.y);
                            v[k][2] = to_f16x2<BF16>(x.z), v[k][3] = to_f16x2<BF16>(x.w);
                        }
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const uint32_t a0 = __byte_perm(v[0][p], v[1][p], 0x5410), a1 = __byte_perm(v[0][p], v[1][p], 0x7632);
                            const uint32_t a2 = __byte_perm(v[2][p], v[3][p], 0x5410), a3 = __byte_perm(v[2][p], v[3][p], 0x7632);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                mma_f16(o[n][c * 4 + p], a0, a1, a2, a3, hi[n][0][0], hi[n][0][1]);
                                if constexpr (SPLIT) mma_f16(o[n][c * 4 + p], a0, a1, a2, a3, lo[n][0][0], lo[n][0][1]);
                            }
                        }
                    }
                }
            }

            // ---- the CTA's warps join their rows
            named_sync(1, 32 * kWarps4);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[n][e];
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
                    const int r = n * 8 + 2 * t + e;
                    const bool live = row_tok[n][e] >= 0;
                    if (g == 0) {
                        sh_m[warp][r] = live ? m[n][e] : -INFINITY;
                        sh_l[warp][r] = live ? x : 0.f;
                    }
                    float* dst = &sh_o[warp][r][g * (HD / 8)];
#pragma unroll
                    for (int p = 0; p < MT; ++p) {
                        dst[2 * p] = live ? o[n][p][e] : 0.f;
                        dst[2 * p + 1] = live ? o[n][p][2 + e] : 0.f;
                    }
                }
        }
        __syncthreads();
        const bool whole = nt == sv.tiles;
        const int64_t slot = blockIdx.x * 2 + (sh_done == 0 ? 0 : 1);
        for (int u = tid; u < ROWS * (HD / 8); u += kThreads4) {
            const int r = u / (HD / 8), c = (u % (HD / 8)) * 8;
            const float top = fmaxf(fmaxf(sh_m[0][r], sh_m[1][r]), fmaxf(sh_m[2][r], sh_m[3][r]));
            float f[4], sum = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                f[w] = sh_m[w][r] == -INFINITY ? 0.f : ex2_approx(sh_m[w][r] - top);
                sum += f[w] * sh_l[w][r];
            }
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = f[0] * sh_o[0][r][c + e] + f[1] * sh_o[1][r][c + e] + f[2] * sh_o[2][r][c + e] +
                       f[3] * sh_o[3][r][c + e];
            if (!whole) {
                float* po = a.part_o + (slot * ROWS + r) * HD + c;
                *reinterpret_cast<float4*>(po) = make_float4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<float4*>(po + 4) = make_float4(x[4], x[5], x[6], x[7]);
                if (c == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * ROWS + r) * 2) = make_float2(top, sum);
                continue;
            }
            const int rr = r0 + r;
            if (rr >= R) continue;
            const int tok = rr / a.group;
            const int64_t h = gk * a.group + (rr - tok * a.group);
            store_row<BF16, 8>(a, bi, tok, h, c, tok < sv.nq, top, sum, x);
        }
        __syncthreads();
        if (tid == 0) {
            sh_done += seg.line_n;
            sh_part.rem = rem + seg.line_n;
            if (rem + seg.line_n == (sv.tiles + a.unit_cost) * units) {
                ++sh_part.bi;
                sh_part.rem = 0;
            }
        }
        __syncthreads();
        if (sh_done == sh_count) break;
    }
    if (!a.whole) grid_dep_launch();
}

namespace {

template <int HD, bool BF16, int NT>
cudaError_t launch_rows4(const CacheTileArgs& qa, cudaStream_t s)
{
    auto kern = cache4_fwd_rows_kernel<HD, BF16, NT>;
    const uint32_t bytes = Rows4Cfg<HD, NT>::kBytes;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(kern, bytes, allowed);
    if (e != cudaSuccess) return e;
    kern<<<qa.f.parts, kThreads4, bytes, s>>>(qa);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_cache_fwd_join(qa.f, BF16 ? SDPA_BF16 : SDPA_F16, 8 * NT, s);
}

template <bool BF16>
cudaError_t launch_fwd4(const CacheTileArgs& qa, cudaStream_t s)
{
    switch (cache4_fwd_plan(qa.f.c.d, qa.f.s_q * qa.f.group).variant) {
        case kQ4Rows128x8: return launch_rows4<128, BF16, 1>(qa, s);
        case kQ4Rows128x16: return launch_rows4<128, BF16, 2>(qa, s);
        case kQ4Rows64x8: return launch_rows4<64, BF16, 1>(qa, s);
        case kQ4Rows64x16: return launch_rows4<64, BF16, 2>(qa, s);
        default: return launch_cache4_fwd_tiles(qa, BF16 ? SDPA_BF16 : SDPA_F16, s);
    }
}

}  // namespace

// Rows per kv-head above which the tile kernel is ahead, though the blocks of 16
// rows below read K and V again each (12 sequences of 16484 keys, 6 kv-heads):
// d = 128, 32 rows 109 us against 131, 48 rows 154 against 131; d = 64, 48 rows 83 us
// against 106, 64 rows 106 and 106, 80 rows 126 against 106. A unit's cost in tiles of 256 keys (64 ragged
// sequences of 5 to 16484 keys, 8 rows): 61, 49, 45, 48, 54 us at 1, 2, 3, 4, 6; in
// the tile kernel's of 64 (24 rows): 214, 178, 166 at 4, 8, 16.
CacheFwdPlan cache4_fwd_plan(int64_t d, int64_t rows)
{
    if (rows > (d == 128 ? 32 : 64)) return CacheFwdPlan{kQ4Tiles, 256, 64, 1, 16};
    if (d == 128) return rows <= 8 ? CacheFwdPlan{kQ4Rows128x8, 8, kTile4, 2, 3} : CacheFwdPlan{kQ4Rows128x16, 16, kTile4, 2, 3};
    return rows <= 8 ? CacheFwdPlan{kQ4Rows64x8, 8, kTile4, 2, 3} : CacheFwdPlan{kQ4Rows64x16, 16, kTile4, 2, 3};
}

cudaError_t launch_cache4_fwd(const CacheTileArgs& a, int dtype, cudaStream_t s)
{
    return dtype == SDPA_BF16 ? launch_fwd4<true>(a, s) : launch_fwd4<false>(a, s);
}

}  // namespace swa
