// cache_fwd.cu -- attention of a few new tokens per sequence over the paged
// cache and over each other (sdpa_cache_fwd).
//
// Rows. A kv-head's query rows are the s_q tokens of its `group` q-heads:
// row r is token r / group, head r % group. The keys of a sequence are its
// cached ones in reach, then its new ones, in groups of 16 that hold one kind.
//
// Few rows (cache_fwd_rows_kernel): the call is bound by reading K and V once,
// so every row of a kv-head is computed by the warp that reads a key. A warp
// fetches 16 keys of 128 features (32 of 64) a step into a ring of its own: by
// TMA boxes of 16 or 8 keys where a page's size is a multiple of it (or the keys
// are one run), else by one bulk copy per key and tensor. A copy of a single row of
// 128 bytes costs the engine what one of 256 does (4.3 TB/s in all, against
// 7.0). Through registers (LDG) or cp.async the same loads reached 6.0 and 4.3
// TB/s at d = 128: 16 instructions a step and warp instead of one. A warp waits
// for no other. 64 sequences of 5 to 16484 keys, 6 kv-heads of 8 rows, d = 128
// in f16: 79 us, 5.4 TB/s; at d = 64 49 us, 4.4 TB/s.
//   S^T = K Q^T   m16n8k16, M = 16 keys, N = 8 rows. A dot product does not
//                 depend on the order of the features, so the instruction's k
//                 index is mapped to features such that a thread's operand
//                 registers are 16-byte pieces of a key.
//   O^T += V^T P^T   M = 16 features, N = 8 rows, K = 16 keys. A thread reads 8
//                 consecutive features of the 4 keys of its k indexes and pairs
//                 two keys' values by byte permutes; P^T comes from the S^T
//                 registers by an 8 x 8 transpose (movmatrix).
// Both keep a row in one column: its maximum and its scale are per-thread
// values. The reference of a row's exponentials moves only when a score exceeds
// it by more than 2^8 (one vote per step instead of shuffles; f16: 2^15, from 2^7
// on, see kBelow); a P above 1 costs no precision in floating point. P is split
// into a 16-bit value and its 16-bit remainder, two products: O then has the
// error of its own rounding only (in f16 also half of 2^-24 a key next to a
// largest P of 2^7 at least), and the second product runs in the shadow of the
// loads.
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

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

constexpr int kStages = 3;              // steps of a warp that are on their way or worked on

// A step's K, then its V: rows of the keys, 16 bytes apart more than they are
// long, or (boxes of 64 features) 128 bytes of them in the 128-byte swizzle.
template <int HD>
struct RowsCfg {
    static constexpr int KG = 128 / HD;                   // 16-key groups of a step
    static constexpr int GK = 16 * KG;
    static constexpr uint32_t kPitch = HD * 2 + 16;
    static constexpr uint32_t kStage = 9216;              // both forms, and boxes begin on 1024 bytes
    static constexpr uint32_t kRings = 4 * kStages * kStage;
    static constexpr uint32_t kBytes = kRings + 1024;
    static_assert(2 * GK * kPitch <= kStage, "");
};

}  // namespace

template <int HD, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, 2) cache_fwd_rows_kernel(const __grid_constant__ CacheTileArgs ta)
{
    const CacheFwdArgs& a = ta.f;
    using C = RowsCfg<HD>;
    constexpr int KG = C::KG, GK = C::GK;
    constexpr int TK = 4 * GK;
    constexpr int CH = HD / 32;        // 16-byte pieces of a key's K per thread
    constexpr int VJ = HD / 64;        // 16-byte pieces of a key's V per thread
    constexpr int MT = HD / 16;        // feature tiles of O^T
    constexpr int ROWS = 8 * NT;
    constexpr int PAD = HD + 4;
    extern __shared__ __align__(1024) uint8_t raw[];
    // the warps' rings; at a unit's end their O. Boxes begin on 1024 bytes (kBytes has the slack)
    uint8_t* dyn = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t sh_bar[4][kStages];
    float (*sh_o)[ROWS][PAD] = reinterpret_cast<float (*)[ROWS][PAD]>(dyn);
    static_assert(4 * ROWS * PAD * 4 <= C::kRings, "the warps' O in the rings' place");
    __shared__ int32_t sh_pos[4][kStages][GK];         // per step of a ring: the keys' positions,
    __shared__ uint32_t sh_ok[4][kStages];             // and which are there
    __shared__ float sh_m[4][ROWS], sh_l[4][ROWS];
    __shared__ uint64_t sh_mask[64];       // new tokens that each one's rows admit
    __shared__ int32_t sh_bits[64];        // and its mask's number of bits
    __shared__ uint32_t sh_used[2];        // new tokens that some row admits
    __shared__ int64_t sh_sum[4];
    __shared__ int64_t sh_at[2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int R = a.s_q * a.group;
    const int blocks = (R + ROWS - 1) / ROWS;
    const int64_t units = a.c.h_kv * blocks;      // per sequence

    // ---- this CTA's part of the line; where it stands is kept in shared memory,
    // the registers are for the keys
    __shared__ Part sh_part;
    __shared__ int64_t sh_done, sh_count;      // places of the part in the line: done, all
    {
        Part part{1, 0, 0, 0, 0, Line{0}};
        if (a.whole) {
            // short units: a CTA takes one from end to end, nothing is cut
            part.bi = blockIdx.x / units;
            part.end = seq_view(a, part.bi, TK).tiles;
            part.rem = (blockIdx.x - part.bi * units) * (part.end + a.unit_cost) + a.unit_cost;
        } else {
            part = find_part<kThreads>(
                a.c.b, [&](int64_t i) { return (seq_view(a, i, TK).tiles + a.unit_cost) * units; }, sh_sum, sh_at);
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

    if (tid < 4 * kStages) mbar_init(smem_u32(&sh_bar[0][0]) + tid * 8, 1);
    fence_mbar_init();
    __syncthreads();
    uint32_t sent = 0;        // per stage: the parity of its next step
    bool good = true;         // no wait has run out
    int64_t cur = -1;
    for (;;) {
        const int64_t bi = sh_part.bi, rem = sh_part.rem;
        const SeqView sv = seq_view(a, bi, TK);
        if (cur != bi) {
            if (tid < 64) {
                int bits;
                sh_mask[tid] = admitted_tokens(a, bi, sv.nq, tid, bits);
                sh_bits[tid] = bits;
            }
            if (tid < 2) sh_used[tid] = 0;
            __syncthreads();
            if (warp < 2) {
                const uint64_t m = sh_mask[tid];
                const uint32_t lo32 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(m));
                const uint32_t hi32 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(m >> 32));
                if (lane == 0) {
                    atomicOr(&sh_used[0], lo32);
                    atomicOr(&sh_used[1], hi32);
                }
            }
            __syncthreads();
            cur = bi;
        }
        const Segment seg = segment_at(rem, sv.tiles, a.unit_cost, sh_count - sh_done);
        const int64_t un = seg.un;
        const int32_t tile0 = seg.tile0, nt = seg.n;
        if (nt == 0) break;                                 // the part ends before the unit's first tile
        const int64_t gk = un / blocks;                     // kv-head
        const int r0 = static_cast<int>(un - gk * blocks) * ROWS;
        if (tid == 0 && !a.whole)
            name_cut(a, sh_part, sh_done == 0, sh_part.at + sh_done + seg.line_n - tile0 - nt, a.unit_cost, bi, un, units, tile0,
                     nt, sv.tiles);
        const int64_t npos = a.c.next_pos ? a.c.next_pos[bi] : sv.len;
        const int32_t* kpos = a.c.positions ? a.c.positions + (bi * a.c.h_kv + gk) * a.c.cap : nullptr;

        // ---- rows: Q pieces (row g of each 8), masks and windows (rows 2t, 2t + 1)
        uint4 q[NT][CH];
        int row_tok[NT][2];           // the row's token, -1: admits nothing
        int32_t row_low[NT][2];       // lowest position in the row's window
        int32_t low_max = INT32_MIN, low_min = INT32_MAX;  // the highest and the lowest of them (this CTA's rows)
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
                        imax64(INT32_MIN, imin64(INT32_MAX, npos + sh_bits[tk] - 1 - a.window_left)));
                if (m) {
                    low_max = max(low_max, row_low[n][e]);
                    low_min = min(low_min, row_low[n][e]);
                }
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            low_max = max(low_max, __shfl_xor_sync(0xffffffffu, low_max, o));
            low_min = min(low_min, __shfl_xor_sync(0xffffffffu, low_min, o));
        }

        // ---- the line of keys of this unit: groups of GK per warp
        auto step_x = [&](int32_t s) -> int32_t { return (tile0 + s) * TK + warp * GK; };
        // Lane l's key (l % GK) of step s, if it is a cached one: its page entry,
        // loaded a step ahead of its use, and its position.
        struct Key {
            int32_t entry;    // page-table entry
            int32_t pos;      // cached key's position
        };
        const bool by_pos = kpos != nullptr && a.window_left >= 0;
        auto fetch_key = [&](int32_t s) -> Key {
            Key k{0, 0};
            const int32_t x = step_x(s) + lane % GK;
            if (x < sv.new0) {
                const int32_t j = sv.lo + x;
                if (j < sv.len) {
                    if (a.c.page_table) k.entry = cache_entry(a.c, bi, j);
                    k.pos = by_pos ? kpos[j] : j;
                }
            }
            return k;
        };
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

        const uint32_t ring = smem_u32(dyn) + warp * (kStages * C::kStage);
        const uint32_t bars = smem_u32(&sh_bar[warp][0]);
        // 16-byte piece c of a key of a step, relative to the step's K or V
        const bool boxed = ta.box_rows != 0;
        const uint32_t half = boxed ? 4096 : GK * C::kPitch;           // where V begins
        const uint32_t pitch = boxed ? 128 : C::kPitch, swz = boxed ? 7 : 0, blk = boxed ? GK * 128 - 128 : 0;
        auto piece = [&](uint32_t key_row, uint32_t c) -> uint32_t {
            return key_row * pitch + ((c ^ (key_row & swz)) << 4) + (c >> 3) * blk;
        };
        // Sends step s's copies on their way: lane l looks after key l % GK.
        auto issue = [&](int32_t s, const Key& k) {
            const uint32_t st = static_cast<uint32_t>(s) % kStages, at = ring + st * C::kStage, bar = bars + st * 8;
            const int32_t x = step_x(s) + lane % GK, j = sv.lo + x;
            const uint32_t key_row = lane % GK;
            bool ok = x < sv.new0 && j < sv.len;        // a cached key
            int64_t page = bi;
            uint32_t row = j;
            const bool reach = ok && k.pos >= low_min;
            if (ok && a.c.page_table) {
                page = k.entry;
                row = cache_row(a.c, j);
                ok = page >= 0 && page < a.c.n_pages;
                if (reach && !ok) set_status(a.c.status, SDPA_ERR_BOUNDS);
            }
            ok = ok && reach;
            const uint32_t oks = __ballot_sync(0xffffffffu, ok);
            if (lane < GK) sh_pos[warp][st][lane] = k.pos;
            if (boxed) {
                // boxes of 16 or 8 keys (2 or 1 KB each: features 0-63, 64-127 of K, of V); rows of the page in front
                // of the first key in reach and behind the last one come along
                const int bk = ta.box_rows, nu = GK / bk;                 // keys of a box, boxes over a step's keys
                const uint32_t of_box = (1u << bk) - 1;
                // one lane a box
                const int u = lane % nu, b = lane / nu, is_v = b / (HD / 64), cb = b % (HD / 64);
                const int row0 = __shfl_sync(0xffffffffu, static_cast<int>(row), u * bk);
                const int page0 = __shfl_sync(0xffffffffu, static_cast<int>(page), u * bk);
                const bool mine = b < 2 * (HD / 64) && ((oks >> (u * bk)) & of_box) != 0;
                const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
                if (lane == 0) {
                    sh_ok[warp][st] = oks;
                    mbar_arrive_expect_tx(bar, boxes * bk * 128);
                }
                __syncwarp();
                if (mine)
                    tma_box(at + (is_v ? half : 0u) + cb * (GK * 128) + u * bk * 128, is_v ? &ta.tm_v : &ta.tm_k, bar, cb * 64,
                            static_cast<int>(gk), row0, page0);
            } else {
                if (lane == 0) {
                    sh_ok[warp][st] = oks;
                    mbar_arrive_expect_tx(bar, __popc(GK == 32 ? oks : oks & 0xffffu) * 2 * HD * 2);
                }
                __syncwarp();
                if (ok) {
                    const uint16_t* kp = a.c.k + page * a.c.k_stride[0] + row * a.c.k_stride[1] + gk * a.c.k_stride[2];
                    const uint16_t* vp = a.c.v + page * a.c.v_stride[0] + row * a.c.v_stride[1] + gk * a.c.v_stride[2];
                    // 32 keys: both by each lane; 16: K by the lower lanes, V by the upper
                    if (GK == 32 || lane < 16) bulk_load(at + key_row * C::kPitch, kp, HD * 2, bar);
                    if (GK == 32 || lane >= 16) bulk_load(at + half + key_row * C::kPitch, vp, HD * 2, bar);
                }
            }
            // new tokens: 16 bytes at a time, zeros in the rows of their group that hold none or one that no row
            // admits (padding may be anything, and meets a P of 0)
#pragma unroll
            for (int u = 0; u < KG; ++u) {
                const int32_t w0 = step_x(s) + u * 16 - sv.new0;      // the group's first new token
                if (w0 < 0 || w0 >= sv.nq) continue;
                for (int i = lane; i < 16 * (HD / 8); i += 32) {
                    const int r = i / (HD / 8), c = i % (HD / 8);
                    const bool have = w0 + r < sv.nq && (sh_used[(w0 + r) >> 5] >> ((w0 + r) & 31)) & 1;
                    const int64_t tok = have ? w0 + r : 0;
                    cp16(at + piece(u * 16 + r, c), a.k + bi * a.k_stride[0] + tok * a.k_stride[1] + gk * a.k_stride[2] + c * 8,
                         have);
                    cp16(at + half + piece(u * 16 + r, c),
                         a.v + bi * a.v_stride[0] + tok * a.v_stride[1] + gk * a.v_stride[2] + c * 8, have);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };

        // (rings hold the last unit's O: its reads are done, and known to the copy engine)
        fence_proxy_async_smem();
        __syncwarp();
        Key key = fetch_key(0);
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            const Key next = fetch_key(s + 1);
            if (good && s < nt && !(a.c.stall && s == 1)) issue(s, key);      // (test hook: a step that never comes)
            key = next;
        }
#pragma unroll 1
        for (int32_t s = 0; s < nt; ++s) {
            {
                const Key next = fetch_key(s + kStages);
                if (good && s + kStages - 1 < nt) issue(s + kStages - 1, key);
                key = next;
            }
            const uint32_t st = static_cast<uint32_t>(s) % kStages, at = ring + st * C::kStage;
            if (good) {
                good = __all_sync(0xffffffffu, mbar_wait(bars + st * 8, (sent >> st) & 1, a.timeout_ns));
                if (!good) {
                    // nothing more is sent; what is on its way ends before the CTA does
                    set_status(a.c.status, SDPA_ERR_TIMEOUT);
                    for (int32_t q = s; q < nt && q < s + kStages; ++q)
                        mbar_wait(bars + (q % kStages) * 8, (sent >> (q % kStages)) & 1, a.timeout_ns);
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    __syncwarp();
                }
            }
            sent ^= 1u << st;
            const int32_t x0 = step_x(s);
            const bool some_new = x0 + GK > sv.new0;
            if (some_new) asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            if (!good) continue;
            // keys that are there: cached ones, new tokens
            uint32_t ok = sh_ok[warp][st];
            if (some_new)
#pragma unroll
                for (int u = 0; u < KG; ++u) {
                    const int32_t w0 = x0 + u * 16 - sv.new0;
                    if (w0 >= 0) ok |= (w0 < sv.nq ? (sv.nq - w0 >= 16 ? 0xffffu : (1u << (sv.nq - w0)) - 1) : 0u) << (16 * u);
                }
            const bool full = GK == 32 ? ok == 0xffffffffu : (ok & 0xffffu) == 0xffffu;
            // S^T
            float sc[NT][KG][4];
#pragma unroll
            for (int u = 0; u < KG; ++u) {
#pragma unroll
                for (int n = 0; n < NT; ++n) sc[n][u][0] = sc[n][u][1] = sc[n][u][2] = sc[n][u][3] = 0.f;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const uint4 k0 = lds16(at + piece(u * 16 + g, t + 4 * i)), k1 = lds16(at + piece(u * 16 + 8 + g, t + 4 * i));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_16816<BF16>(sc[n][u], k0.x, k1.x, k0.y, k1.y, q[n][i].x, q[n][i].y);
                        mma_16816<BF16>(sc[n][u], k0.z, k1.z, k0.w, k1.w, q[n][i].z, q[n][i].w);
                    }
                }
            }
            // masks (a step whose keys are all there and in every row's window needs none; rows that admit nothing
            // are left out at the end), the row's reference, P
            uint32_t hi[NT][KG][2], lo[NT][KG][2];
            float mx[NT][2];
            bool up = false;
            const bool windowed = a.window_left >= 0 && x0 < sv.new0 && (kpos != nullptr || sv.lo + x0 < low_max);
            if (!full || some_new || windowed) {
#pragma unroll
                for (int u = 0; u < KG; ++u) {
                    const bool fresh = x0 + u * 16 >= sv.new0;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int x = u * 16 + (e >> 1) * 8 + g;
                            bool in = (ok >> x) & 1;
                            if (fresh) {
                                const int w = (x0 + x - sv.new0) & 63;      // the new token
                                const uint64_t rm = row_tok[n][e & 1] < 0 ? 0 : sh_mask[row_tok[n][e & 1]];
                                in = in && ((rm >> w) & 1);
                            } else if (windowed) {
                                in = in && sh_pos[warp][st][x] >= row_low[n][e & 1];
                            }
                            if (!in) sc[n][u][e] = -INFINITY;
                        }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mx[n][0] = mx[n][1] = -INFINITY;
#pragma unroll
                for (int u = 0; u < KG; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[n][e & 1] = fmaxf(mx[n][e & 1], sc[n][u][e]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[n][e] *= a.scale_log2;
                    up = up || mx[n][e] > m[n][e] + kMoves<BF16>;
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
                        x = fmaxf(x - kBelow<BF16>, m[n][e]);
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
                        // a masked score is -inf, its P is 0 (a row's reference is finite here, or 0)
                        p[e] = ex2_approx(fmaf(sc[n][u][e], a.scale_log2, m[n][e & 1] == -INFINITY ? 0.f : -m[n][e & 1]));
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
                for (int j = 0; j < VJ; ++j) {
                    uint4 v[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int x = u * 16 + (h >> 1) * 8 + 2 * t + (h & 1);
                        v[h] = lds16(at + half + piece(x, g + 8 * j));
                        // what stands in the place of a key that is not there meets a P of 0: it has to be finite
                        if (!full && !((ok >> x) & 1)) v[h] = make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        auto reg = [&](int h) -> uint32_t {
                            return p == 0 ? v[h].x : p == 1 ? v[h].y : p == 2 ? v[h].z : v[h].w;
                        };
                        const uint32_t a0 = __byte_perm(reg(0), reg(1), 0x5410), a1 = __byte_perm(reg(0), reg(1), 0x7632);
                        const uint32_t a2 = __byte_perm(reg(2), reg(3), 0x5410), a3 = __byte_perm(reg(2), reg(3), 0x7632);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_16816<BF16>(o[n][j * 4 + p], a0, a1, a2, a3, hi[n][u][0], hi[n][u][1]);
                            mma_16816<BF16>(o[n][j * 4 + p], a0, a1, a2, a3, lo[n][u][0], lo[n][u][1]);
                        }
                    }
                }
        }

        // ---- the CTA's warps join their rows
        __syncthreads();
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
#pragma unroll
                for (int j = 0; j < VJ; ++j) {
                    float* dst = &sh_o[warp][r][(g + 8 * j) * 8];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        dst[2 * p] = live ? o[n][j * 4 + p][e] : 0.f;
                        dst[2 * p + 1] = live ? o[n][j * 4 + p][2 + e] : 0.f;
                    }
                }
            }
        __syncthreads();
        const bool whole = nt == sv.tiles;
        const int64_t slot = blockIdx.x * 2 + (sh_done == 0 ? 0 : 1);
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

// Adds the partials of a unit that was cut between parts, in the order of the
// parts. CTA x looks after cuts[x].
// SPREAD: CTA y takes row y, its warps every eighth part (few units, many
// parts each); else a warp takes RW rows, all their parts, with the rows' loads
// on their way together.
template <int HD, bool BF16, int ROWS, bool SPREAD, int RW>
__global__ void __launch_bounds__(256) cache_fwd_join_kernel(const __grid_constant__ CacheFwdArgs a)
{
    static_assert(RW == 1 || !SPREAD, "");
    constexpr int E = HD / 32;
    __shared__ float sh_x[8][HD], sh_s[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    const CacheFwdCut cut = a.cuts[blockIdx.x];
    if (cut.bi < 0) return;
    const int R = a.s_q * a.group, blocks = (R + ROWS - 1) / ROWS;
    const int64_t gk = cut.un / blocks;
    const int r0 = static_cast<int>(cut.un - gk * blocks) * ROWS;
    const int c0 = cut.first, n = cut.last - c0 + 1;
    // parts behind the first begin with this unit
    auto slot = [&](int i) -> int64_t { return i == 0 ? c0 * int64_t(2) + cut.slot0 : (c0 + i) * int64_t(2); };
    int nq = a.s_q;
    if (a.seq_q_lens) nq = max(0, min(a.seq_q_lens[cut.bi], a.s_q));
    // this warp's rows; their partials are there up to the next multiple of RW behind the last real one (loads without
    // a bound on them are on their way together: 296 rows 11 us, 15 to 16 with one)
    static_assert(kPartialRows % RW == 0, "");
    const int r = SPREAD ? blockIdx.y : (blockIdx.y * 8 + warp) * RW;
    if (r0 + r >= R) return;
    float top[RW], sum[RW], x[RW][E];
#pragma unroll
    for (int j = 0; j < RW; ++j) {
        top[j] = -INFINITY;
        sum[j] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x[j][e] = 0.f;
    }
    for (int i = lane; i < n; i += 32) {
#pragma unroll
        for (int j = 0; j < RW; ++j) top[j] = fmaxf(top[j], a.part_ml[(slot(i) * ROWS + r + j) * 2]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int j = 0; j < RW; ++j) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
#pragma unroll(RW == 1 ? 8 : 2)
    for (int i = SPREAD ? warp : 0; i < n; i += SPREAD ? 8 : 1) {
        const int64_t at = slot(i) * ROWS + r;
#pragma unroll
        for (int j = 0; j < RW; ++j) {
            const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (at + j) * 2);
            const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top[j]);
            sum[j] += f * ml.y;
            const float* p = a.part_o + (at + j) * HD + lane * E;
            float v[E];
            if constexpr (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p);
            else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(p);
#pragma unroll
            for (int e = 0; e < E; ++e) x[j][e] += f * v[e];
        }
    }
    if (SPREAD) {
#pragma unroll
        for (int e = 0; e < E; ++e) sh_x[warp][lane * E + e] = x[0][e];
        if (lane == 0) sh_s[warp] = sum[0];
        __syncthreads();
        if (warp > 0) return;
        sum[0] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x[0][e] = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            sum[0] += sh_s[w];
#pragma unroll
            for (int e = 0; e < E; ++e) x[0][e] += sh_x[w][lane * E + e];
        }
    }
#pragma unroll
    for (int j = 0; j < RW; ++j) {
        const int rr = r0 + r + j;
        if (rr >= R) break;
        const int tok = rr / a.group;
        store_row<BF16, E>(a, cut.bi, tok, gk * a.group + (rr - tok * a.group), lane * E, tok < nq, top[j], sum[j], x[j]);
    }
}

namespace {

template <int HD, bool BF16, int ROWS>
cudaError_t launch_join(const CacheFwdArgs& a, cudaStream_t s)
{
    if (a.whole || a.parts == 1) return cudaSuccess;
    const int rows = a.s_q * a.group, blocks = (rows + ROWS - 1) / ROWS, most = rows < ROWS ? rows : ROWS;
    const int64_t units = a.c.b * a.c.h_kv * blocks;
    // with fewer units than an eighth of the parts a unit has many parts
    const bool spread = units * 8 < a.parts;
    cudaLaunchConfig_t cfg{};
    constexpr int RW = ROWS == 8 ? 1 : 4, CR = 8 * RW;      // rows of a warp, of a CTA
    cfg.gridDim = dim3(static_cast<unsigned>(a.cut_by_unit ? units : a.parts), spread ? most : (most + CR - 1) / CR);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return spread ? cudaLaunchKernelEx(&cfg, cache_fwd_join_kernel<HD, BF16, ROWS, true, 1>, a)
                  : cudaLaunchKernelEx(&cfg, cache_fwd_join_kernel<HD, BF16, ROWS, false, RW>, a);
}

template <int HD, bool BF16, int NT>
cudaError_t launch_rows(const CacheTileArgs& ta, cudaStream_t s)
{
    auto kern = cache_fwd_rows_kernel<HD, BF16, NT>;
    const uint32_t bytes = RowsCfg<HD>::kBytes;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(kern, bytes, allowed);
    if (e != cudaSuccess) return e;
    kern<<<ta.f.parts, kThreads, bytes, s>>>(ta);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join<HD, BF16, 8 * NT>(ta.f, s);
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
    switch (cache_fwd_plan(ta.f.c.d, ta.f.s_q * ta.f.group).variant) {
        case kRows128x8: return launch_rows<128, BF16, 1>(ta, s);
        case kRows64x8: return launch_rows<64, BF16, 1>(ta, s);
        case kRows64x16: return launch_rows<64, BF16, 2>(ta, s);
        case kTiles128: return launch_tiles<128, BF16>(ta, s);
        default: return launch_tiles<64, BF16>(ta, s);
    }
}

}  // namespace

// Rows per kv-head above which the tile kernel is ahead (12 sequences of 16484
// keys, 6 kv-heads): d = 128, 16 rows 116 us against 131 for a rows kernel of 16
// (8 rows: 107 against the tile kernel's 113); d = 64, 32 rows 98 us against 138
// (16 rows: 75 against 98), as measured together (the tile kernel's 16 and 32
// rows are 105 and 81 us now). A unit's cost (64 ragged sequences of 5 to 16484
// keys): rows kernel 123, 89, 79, 79, 84 us at 0, 2, 4, 8, 16; tile kernel with
// 24 rows 228, 127, 104, 126 us at 0, 4, 8, 16.
CacheFwdPlan cache_fwd_plan(int64_t d, int64_t rows)
{
    if (d == 128) return rows <= 8 ? CacheFwdPlan{kRows128x8, 8, 64, 2, 4} : CacheFwdPlan{kTiles128, 256, 64, 1, 8};
    if (rows <= 8) return CacheFwdPlan{kRows64x8, 8, 128, 2, 4};
    if (rows <= 16) return CacheFwdPlan{kRows64x16, 16, 128, 2, 4};
    return CacheFwdPlan{kTiles64, 256, 64, 1, 8};
}

cudaError_t launch_cache_fwd(const CacheTileArgs& a, int dtype, cudaStream_t s)
{
    return dtype == SDPA_BF16 ? launch_fwd_typed<true>(a, s) : launch_fwd_typed<false>(a, s);
}

}  // namespace swa
