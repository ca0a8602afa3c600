// cache_fwd.cu -- attention of a few new tokens per sequence over the paged
// cache and over each other (sdpa_cache_fwd).
//
// Rows. A kv-head's query rows are the s_q tokens of its `group` q-heads:
// row r is token r / group, head r % group. The keys of a sequence are its
// cached ones in reach, then its new ones, in groups of 16 that hold one kind.
//
// Few rows (cache_fwd_rows_kernel): the call is bound by reading K and V once,
// so every row of a kv-head is computed by the warp that reads a key, and keys
// go from global memory into the registers that the matrix instruction reads,
// without a stage in shared memory:
//   S^T = K Q^T   m16n8k16, M = 16 keys, N = 8 rows. A dot product does not
//                 depend on the order of the features, so the instruction's k
//                 index is mapped to features such that a thread's operand
//                 registers are the 16-byte pieces that it loads (a quad of
//                 threads reads 64 consecutive bytes of a key).
//   O^T += V^T P^T   M = 16 features, N = 8 rows, K = 16 keys. A thread loads 8
//                 consecutive features of the 4 keys of its k indexes and pairs
//                 two keys' values by byte permutes; P^T comes from the S^T
//                 registers by an 8 x 8 transpose (movmatrix).
// Both keep a row in one column: its maximum and its scale are per-thread
// values. The reference of a row's exponentials moves only when a score exceeds
// it by more than 2^8 (one vote per step instead of shuffles); P up to 2^8 costs
// no precision in floating point. P is split into a 16-bit value and its 16-bit
// remainder, two products: O then has the error of its own rounding only, and
// the second product runs in the shadow of the loads.
//
// Work: the 64- or 128-key tiles of all (sequence, kv-head, row block) units
// form one line that the persistent CTAs cut into equal parts, whatever the
// sequences' lengths. A unit inside one part is finished there; a unit cut
// between parts leaves fp32 partials (row reference, sum, O) that
// cache_fwd_join_kernel adds in the order of the parts.
#include "cache_fwd.cuh"

namespace swa {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ uint32_t movm_trans(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes that this kernel reads once.
__device__ __forceinline__ uint4 ld_stream(const uint16_t* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

}  // namespace

// Features per thread and step: see the comment at the top of the file.
template <int HD, bool BF16, int NT, int OCC>
__global__ void __launch_bounds__(kThreads, OCC) cache_fwd_rows_kernel(const __grid_constant__ CacheFwdArgs a)
{
    constexpr int KG = 128 / HD;       // 16-key groups per warp and step: 8 KB of K and V in flight either way
    constexpr int GK = 16 * KG;
    constexpr int TK = 4 * GK;
    constexpr int CH = HD / 32;        // 16-byte pieces of a key's K per thread
    constexpr int VJ = HD / 64;        // 16-byte pieces of a key's V per thread
    constexpr int MT = HD / 16;        // feature tiles of O^T
    constexpr int ROWS = 8 * NT;
    constexpr int PAD = HD + 4;
    __shared__ float sh_o[4][ROWS][PAD];
    __shared__ float sh_m[4][ROWS], sh_l[4][ROWS];
    __shared__ uint64_t sh_mask[64];
    __shared__ int64_t sh_sum[4];
    __shared__ int64_t sh_at[2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int R = a.s_q * a.group;
    const int blocks = (R + ROWS - 1) / ROWS;
    const int64_t units = a.c.h_kv * blocks;      // per sequence

    // ---- this CTA's part of the line
    Part part{1, 0, 0, 0, 0, Line{0}};
    CacheFwdCut cut{-1, 0, 0, 0};
    if (a.whole) {
        // short units: a CTA takes one from end to end, nothing is cut
        part.bi = blockIdx.x / units;
        part.end = seq_view(a, part.bi, TK).tiles;
        part.rem = (blockIdx.x - part.bi * units) * part.end;
    } else {
        part = find_part<kThreads>(a.c.b, [&](int64_t i) { return seq_view(a, i, TK).tiles * units; }, sh_sum, sh_at);
        if (part.end == 0) {
            if (tid == 0) a.cuts[blockIdx.x] = cut;
            grid_dep_launch();
            return;
        }
    }
    const Line& line = part.line;
    const int64_t parts = part.parts, end = part.end, part0 = part.at;
    int64_t at = part.at, bi = part.bi, rem = part.rem;

    SeqView sv{};
    int64_t cur = -1;
    while (at < end) {
        if (cur != bi) {
            sv = seq_view(a, bi, TK);
            __syncthreads();
            if (tid < 64) {
                const uint64_t in = sv.nq == 64 ? ~0ull : (1ull << sv.nq) - 1;
                uint64_t m = 0;
                if (tid < sv.nq) m = in & (a.tree ? static_cast<uint64_t>(a.tree[bi * a.s_q + tid]) : (2ull << tid) - 1);
                sh_mask[tid] = (m >> tid) & 1 ? m : 0;   // without its own bit: an empty row
            }
            __syncthreads();
            cur = bi;
        }
        const int64_t un = rem / sv.tiles;
        const int32_t tile0 = static_cast<int32_t>(rem - un * sv.tiles);
        const int32_t nt = static_cast<int32_t>(imin64(sv.tiles - tile0, end - at));
        const int64_t gk = un / blocks;                     // kv-head
        const int r0 = static_cast<int>(un - gk * blocks) * ROWS;
        // the part that holds the first cut of a unit names the join's work
        if (at == part0 && tile0 > 0) {
            const int64_t u0 = at - tile0, p0 = line.part_of(u0, parts);
            if (p0 + 1 == blockIdx.x)
                cut = CacheFwdCut{bi, un, static_cast<int32_t>(line.part_of(u0 + sv.tiles - 1, parts)),
                                  line.start(p0, parts) == u0 ? 0 : 1};
        }
        const int64_t npos = a.c.next_pos ? a.c.next_pos[bi] : sv.len;
        const int32_t* kpos = a.c.positions ? a.c.positions + (bi * a.c.h_kv + gk) * a.c.cap : nullptr;

        // ---- rows: Q pieces (row g of each 8), masks and windows (rows 2t, 2t + 1)
        uint4 q[NT][CH];
        int row_tok[NT][2];           // the row's token, -1: admits nothing
        int32_t row_low[NT][2];       // lowest position in the row's window
        int32_t low_max = INT32_MIN;  // the highest of them (this CTA's rows)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = r0 + n * 8 + g;
            const int tok = r / a.group;
            const bool real = r < R && tok < sv.nq;
            const uint16_t* qp = a.q + bi * a.q_stride[0] + tok * a.q_stride[1] +
                                 (gk * a.group + (r - tok * a.group)) * a.q_stride[2] + t * 8;
#pragma unroll
            for (int i = 0; i < CH; ++i) q[n][i] = real ? ld_nc_v4(qp + i * 32) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = r0 + n * 8 + 2 * t + e;
                const int tk = rr < R ? rr / a.group : 0;
                const uint64_t m = rr < R ? sh_mask[tk] : 0;
                row_tok[n][e] = m ? tk : -1;
                row_low[n][e] = INT32_MIN;
                if (a.window_left >= 0)
                    row_low[n][e] = static_cast<int32_t>(
                        imax64(INT32_MIN, imin64(INT32_MAX, npos + __popcll(m) - 1 - a.window_left)));
                if (m) low_max = max(low_max, row_low[n][e]);
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) low_max = max(low_max, __shfl_xor_sync(0xffffffffu, low_max, o));

        // ---- the line of keys of this unit: groups of GK per warp
        auto step_x = [&](int32_t s) -> int32_t { return (tile0 + s) * TK + warp * GK; };
        // Lane l's key of step s: whether it is held, the cached key's page entry
        // (loaded a step ahead of its use) and position.
        struct Key {
            int32_t entry;    // page-table entry
            int32_t pos;      // cached key's position
        };
        auto fetch_key = [&](int32_t s) -> Key {
            Key k{0, 0};
            const int32_t x = step_x(s) + lane;
            if (lane < GK && x < sv.new0) {
                const int32_t j = sv.lo + x;
                if (j < sv.len) {
                    if (a.c.page_table)
                        k.entry = a.c.page_table[bi * a.c.max_pages +
                                                 (a.c.page_shift >= 0 ? static_cast<uint32_t>(j) >> a.c.page_shift
                                                                      : static_cast<uint32_t>(j) / a.c.page_size)];
                    k.pos = kpos && a.window_left >= 0 ? kpos[j] : j;
                }
            }
            return k;
        };
        // Offsets of lane l's key in K and V, and whether the key is there.
        auto place = [&](int32_t s, const Key& k, int64_t& ko, int64_t& vo, bool& ok) {
            const int32_t x = step_x(s) + lane;
            ok = false;
            ko = vo = 0;
            if (lane < GK) {
                if (x < sv.new0) {
                    const int32_t j = sv.lo + x;
                    if (j < sv.len) {
                        int64_t page = bi;
                        uint32_t row = j;
                        ok = true;
                        if (a.c.page_table) {
                            page = k.entry;
                            row = a.c.page_shift >= 0 ? static_cast<uint32_t>(j) & ((1u << a.c.page_shift) - 1)
                                                      : static_cast<uint32_t>(j) % a.c.page_size;
                            ok = page >= 0 && page < a.c.n_pages;
                            if (!ok) set_status(a.c.status, SDPA_ERR_BOUNDS);
                        }
                        ko = page * a.c.k_stride[0] + row * a.c.k_stride[1];
                        vo = page * a.c.v_stride[0] + row * a.c.v_stride[1];
                    }
                } else if (x - sv.new0 < sv.nq) {
                    ok = true;
                    ko = (x - sv.new0) * a.k_stride[1];
                    vo = (x - sv.new0) * a.v_stride[1];
                }
            }
        };
        const uint16_t* kc = a.c.k + gk * a.c.k_stride[2] + t * 8;
        const uint16_t* vc = a.c.v + gk * a.c.v_stride[2] + g * 8;
        const uint16_t* kn = a.k + bi * a.k_stride[0] + gk * a.k_stride[2] + t * 8;
        const uint16_t* vn = a.v + bi * a.v_stride[0] + gk * a.v_stride[2] + g * 8;

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

        uint4 kr[KG][2][CH];      // K of keys g, g + 8 of each group
        uint4 vr[KG][4][VJ];      // V of keys 2t, 2t + 1, 2t + 8, 2t + 9
        int64_t vo_next = 0;
        uint32_t ok_next = 0;
        auto load_k = [&](int32_t s, const Key& k) {
            int64_t ko;
            bool ok;
            place(s, k, ko, vo_next, ok);
            ok_next = __ballot_sync(0xffffffffu, ok);
#pragma unroll
            for (int u = 0; u < KG; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int x = u * 16 + h * 8 + g;
                    const int64_t off = __shfl_sync(0xffffffffu, ko, x);
                    const uint16_t* p = (step_x(s) + u * 16 < sv.new0 ? kc : kn) + off;
                    const bool have = (ok_next >> x) & 1;
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        kr[u][h][i] = have ? ld_stream(p + i * 32) : make_uint4(0u, 0u, 0u, 0u);
                }
        };
        auto load_v = [&](int32_t s) {
#pragma unroll
            for (int u = 0; u < KG; ++u)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int x = u * 16 + (h >> 1) * 8 + 2 * t + (h & 1);
                    const int64_t off = __shfl_sync(0xffffffffu, vo_next, x);
                    const uint16_t* p = (step_x(s) + u * 16 < sv.new0 ? vc : vn) + off;
                    const bool have = (ok_next >> x) & 1;
#pragma unroll
                    for (int j = 0; j < VJ; ++j)
                        vr[u][h][j] = have ? ld_stream(p + j * 64) : make_uint4(0u, 0u, 0u, 0u);
                }
        };

        Key key = fetch_key(0), key1 = fetch_key(1);
        load_k(0, key);
        load_v(0);
#pragma unroll 1
        for (int32_t s = 0; s < nt; ++s) {
            const uint32_t ok = ok_next;
            const int32_t x0 = step_x(s);
            const int32_t my_pos = key.pos;
            // S^T
            float sc[NT][KG][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < KG; ++u) {
                    sc[n][u][0] = sc[n][u][1] = sc[n][u][2] = sc[n][u][3] = 0.f;
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        mma_16816<BF16>(sc[n][u], kr[u][0][i].x, kr[u][1][i].x, kr[u][0][i].y, kr[u][1][i].y, q[n][i].x,
                                        q[n][i].y);
                        mma_16816<BF16>(sc[n][u], kr[u][0][i].z, kr[u][1][i].z, kr[u][0][i].w, kr[u][1][i].w, q[n][i].z,
                                        q[n][i].w);
                    }
                }
            // the next step's keys start their way
            key = key1;
            if (s + 1 < nt) {
                load_k(s + 1, key);
                key1 = fetch_key(s + 2);
            }
            // masks, the row's reference, P
            uint32_t hi[NT][KG][2], lo[NT][KG][2];
            float mx[NT][2];
            bool up = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mx[n][0] = mx[n][1] = -INFINITY;
#pragma unroll
                for (int u = 0; u < KG; ++u) {
                    const bool fresh = x0 + u * 16 >= sv.new0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int x = u * 16 + (e >> 1) * 8 + g;
                        bool in = (ok >> x) & 1;
                        if (fresh) {
                            const int w = x0 + x - sv.new0;      // the new token
                            const uint64_t rm = row_tok[n][e & 1] < 0 ? 0 : sh_mask[row_tok[n][e & 1]];
                            in = in && ((rm >> (w & 63)) & 1) &&
                                 (a.window_left < 0 || __popcll(rm) - __popcll(sh_mask[w & 63]) <= a.window_left);
                        } else {
                            in = in && row_tok[n][e & 1] >= 0;
                        }
                        const float v = in ? sc[n][u][e] * a.scale_log2 : -INFINITY;
                        sc[n][u][e] = v;
                    }
                }
            }
            // the window over cached keys, where any of the step's keys is below the highest row's
            if (a.window_left >= 0 && x0 < sv.new0 && (kpos != nullptr || sv.lo + x0 < low_max)) {
#pragma unroll
                for (int u = 0; u < KG; ++u) {
                    const int32_t p0 = __shfl_sync(0xffffffffu, my_pos, u * 16 + g);
                    const int32_t p1 = __shfl_sync(0xffffffffu, my_pos, u * 16 + 8 + g);
                    if (x0 + u * 16 < sv.new0) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if ((e < 2 ? p0 : p1) < row_low[n][e & 1]) sc[n][u][e] = -INFINITY;
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int u = 0; u < KG; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[n][e & 1] = fmaxf(mx[n][e & 1], sc[n][u][e]);
                up = up || mx[n][0] > m[n][0] + 8.f || mx[n][1] > m[n][1] + 8.f;
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
                        x = fmaxf(x, m[n][e]);
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
                for (int u = 0; u < KG; ++u) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = sc[n][u][e] == -INFINITY ? 0.f : ex2_approx(sc[n][u][e] - m[n][e & 1]);
                        l[n][e & 1] += p[e];
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        hi[n][u][h] = pack2<BF16>(p[2 * h], p[2 * h + 1]);
                        const float2 f = unpack2<BF16>(hi[n][u][h]);
                        lo[n][u][h] = movm_trans(pack2<BF16>(p[2 * h] - f.x, p[2 * h + 1] - f.y));
                        hi[n][u][h] = movm_trans(hi[n][u][h]);
                    }
                }
            // O^T += V^T P^T
#pragma unroll
            for (int u = 0; u < KG; ++u)
#pragma unroll
                for (int j = 0; j < VJ; ++j)
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        auto reg = [&](int h) -> uint32_t {
                            const uint4& v = vr[u][h][j];
                            return p == 0 ? v.x : p == 1 ? v.y : p == 2 ? v.z : v.w;
                        };
                        const uint32_t a0 = __byte_perm(reg(0), reg(1), 0x5410), a1 = __byte_perm(reg(0), reg(1), 0x7632);
                        const uint32_t a2 = __byte_perm(reg(2), reg(3), 0x5410), a3 = __byte_perm(reg(2), reg(3), 0x7632);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_16816<BF16>(o[n][j * 4 + p], a0, a1, a2, a3, hi[n][u][0], hi[n][u][1]);
                            mma_16816<BF16>(o[n][j * 4 + p], a0, a1, a2, a3, lo[n][u][0], lo[n][u][1]);
                        }
                    }
            if (s + 1 < nt) load_v(s + 1);
        }

        // ---- the CTA's warps join their rows
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[n][e];
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
                const int r = n * 8 + 2 * t + e;
                if (g == 0) {
                    sh_m[warp][r] = m[n][e];
                    sh_l[warp][r] = x;
                }
#pragma unroll
                for (int j = 0; j < VJ; ++j) {
                    float* dst = &sh_o[warp][r][(g + 8 * j) * 8];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        dst[2 * p] = o[n][j * 4 + p][e];
                        dst[2 * p + 1] = o[n][j * 4 + p][2 + e];
                    }
                }
            }
        __syncthreads();
        const bool whole = nt == sv.tiles;
        const int64_t slot = blockIdx.x * 2 + (at == part0 ? 0 : 1);
        for (int u = tid; u < ROWS * (HD / 8); u += kThreads) {
            const int r = u / (HD / 8), c = (u % (HD / 8)) * 8;
            float top = fmaxf(fmaxf(sh_m[0][r], sh_m[1][r]), fmaxf(sh_m[2][r], sh_m[3][r]));
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

        at += nt;
        rem += nt;
        if (rem == sv.tiles * units) {
            ++bi;
            rem = 0;
        }
    }
    if (a.whole) return;
    if (tid == 0) a.cuts[blockIdx.x] = cut;
    grid_dep_launch();
}

// Adds the partials of a unit that was cut between parts, in the order of the
// parts. CTA x looks after the unit whose first cut is at part x's start.
// SPREAD: CTA y takes row y, its warps every eighth part (few units, many
// parts each); else CTA y takes 8 rows, a warp each with all its parts.
template <int HD, bool BF16, int ROWS, bool SPREAD>
__global__ void __launch_bounds__(256) cache_fwd_join_kernel(const __grid_constant__ CacheFwdArgs a)
{
    constexpr int E = HD / 32;
    __shared__ float sh_x[8][HD], sh_s[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    const CacheFwdCut cut = a.cuts[blockIdx.x];
    if (cut.bi < 0) return;
    const int R = a.s_q * a.group, blocks = (R + ROWS - 1) / ROWS;
    const int64_t gk = cut.un / blocks;
    const int r0 = static_cast<int>(cut.un - gk * blocks) * ROWS;
    const int c0 = static_cast<int>(blockIdx.x) - 1, n = cut.last - c0 + 1;
    // parts behind the first begin with this unit
    auto slot = [&](int i) -> int64_t { return i == 0 ? c0 * int64_t(2) + cut.slot0 : (c0 + i) * int64_t(2); };
    int nq = a.s_q;
    if (a.seq_q_lens) nq = max(0, min(a.seq_q_lens[cut.bi], a.s_q));
    {
        const int r = SPREAD ? blockIdx.y : blockIdx.y * 8 + warp;
        const int rr = r0 + r;
        if (rr >= R) return;
        float top = -INFINITY;
        for (int i = lane; i < n; i += 32) top = fmaxf(top, a.part_ml[(slot(i) * ROWS + r) * 2]);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float sum = 0.f, x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.f;
#pragma unroll 8
        for (int i = SPREAD ? warp : 0; i < n; i += SPREAD ? 8 : 1) {
            const int64_t at = slot(i) * ROWS + r;
            const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
            const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
            sum += f * ml.y;
            const float* p = a.part_o + at * HD + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = *reinterpret_cast<const float2*>(p + e);
                x[e] += f * v.x;
                x[e + 1] += f * v.y;
            }
        }
        if (SPREAD) {
#pragma unroll
            for (int e = 0; e < E; ++e) sh_x[warp][lane * E + e] = x[e];
            if (lane == 0) sh_s[warp] = sum;
            __syncthreads();
            if (warp > 0) return;
            sum = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                sum += sh_s[w];
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] += sh_x[w][lane * E + e];
            }
        }
        const int tok = rr / a.group;
        store_row<BF16, E>(a, cut.bi, tok, gk * a.group + (rr - tok * a.group), lane * E, tok < nq, top, sum, x);
    }
}

namespace {

template <int HD, bool BF16, int ROWS>
cudaError_t launch_join(const CacheFwdArgs& a, cudaStream_t s)
{
    if (a.whole || a.parts == 1) return cudaSuccess;
    const int blocks = (a.s_q * a.group + ROWS - 1) / ROWS;
    // with an eighth as many units as parts a unit has few cuts
    const bool spread = a.c.b * a.c.h_kv * blocks * 8 < a.parts;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.parts), spread ? ROWS : ROWS / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return spread ? cudaLaunchKernelEx(&cfg, cache_fwd_join_kernel<HD, BF16, ROWS, true>, a)
                  : cudaLaunchKernelEx(&cfg, cache_fwd_join_kernel<HD, BF16, ROWS, false>, a);
}

template <int HD, bool BF16, int NT, int OCC>
cudaError_t launch_rows(const CacheFwdArgs& a, cudaStream_t s)
{
    cache_fwd_rows_kernel<HD, BF16, NT, OCC><<<a.parts, kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join<HD, BF16, 8 * NT>(a, s);
}

template <int HD, bool BF16>
cudaError_t launch_tiles(const CacheTileArgs& ta, cudaStream_t s)
{
    const cudaError_t e = launch_cache_fwd_tiles(ta, BF16 ? SDPA_BF16 : SDPA_F16, s);
    return e != cudaSuccess ? e : launch_join<HD, BF16, 256>(ta.f, s);
}

template <bool BF16>
cudaError_t launch_fwd_typed(const CacheTileArgs& ta, cudaStream_t s)
{
    const CacheFwdArgs& a = ta.f;
    switch (cache_fwd_plan(a.c.d, a.s_q * a.group).variant) {
        case kRows128x8: return launch_rows<128, BF16, 1, 3>(a, s);
        case kRows128x16: return launch_rows<128, BF16, 2, 2>(a, s);
        case kRows64x8: return launch_rows<64, BF16, 1, 4>(a, s);
        case kRows64x16: return launch_rows<64, BF16, 2, 3>(a, s);
        case kRows64x32: return launch_rows<64, BF16, 4, 2>(a, s);
        case kTiles128: return launch_tiles<128, BF16>(ta, s);
        default: return launch_tiles<64, BF16>(ta, s);
    }
}

}  // namespace

CacheFwdPlan cache_fwd_plan(int64_t d, int64_t rows)
{
    if (d == 128) {
        if (rows <= 8) return CacheFwdPlan{kRows128x8, 8, 64, 3};
        if (rows <= 16) return CacheFwdPlan{kRows128x16, 16, 64, 2};
        return CacheFwdPlan{kTiles128, 256, 64, 1};
    }
    if (rows <= 8) return CacheFwdPlan{kRows64x8, 8, 128, 4};
    if (rows <= 16) return CacheFwdPlan{kRows64x16, 16, 128, 3};
    if (rows <= 32) return CacheFwdPlan{kRows64x32, 32, 128, 2};
    return CacheFwdPlan{kTiles64, 256, 64, 1};
}

cudaError_t launch_cache_fwd(const CacheTileArgs& a, int dtype, cudaStream_t s)
{
    return dtype == SDPA_BF16 ? launch_fwd_typed<true>(a, s) : launch_fwd_typed<false>(a, s);
}

}  // namespace swa
