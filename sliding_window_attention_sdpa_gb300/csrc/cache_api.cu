// cache_api.cu -- the C ABI declared in include/sdpa_cache.h: host-side
// argument checks and the launches on the caller's stream. Nothing here
// allocates or synchronises (except sdpa_cache_check_status).
#include <cstring>

#include <cuda_runtime.h>

#include "../../include/sdpa_cache.h"
#include "api_util.h"
#include "cache_internal.h"

namespace {

using swa::api::check_device_ptr;
using swa::api::clear_error;
using swa::api::cuda_status;
using swa::api::fail;
using swa::api::make_rows_map;

// sdpa_cache_test_hook's settings for this thread's next calls.
constexpr int64_t kWaitLimitNs = 2000000000LL;
thread_local int64_t g_test_wait_ns = 0;
thread_local int32_t g_test_stall = 0;

int64_t imin(int64_t x, int64_t y) { return x < y ? x : y; }

int64_t wait_limit() { return g_test_wait_ns > 0 ? g_test_wait_ns : kWaitLimitNs; }

constexpr int64_t kMax31 = int64_t(1) << 31;
// a sequence's keys, rounded up to tiles, are numbered in 32 bits
constexpr int64_t kMaxCap = kMax31 - (int64_t(1) << 16);
// rows of a call, in 32 bits up to the next multiple of a block of rows
constexpr int64_t kMaxRows = kMax31 - 1024;
// 16-byte pieces of an append's CTA (32769 rows at most), in 32 bits
constexpr int64_t kMaxHeads = 4096;

void copy3(int64_t* dst, const int64_t* src) { memcpy(dst, src, 3 * sizeof(int64_t)); }

template <typename T>
T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

sdpa_status_t check_strides(const char* name, const int64_t* st, int first = 0)
{
    for (int i = first; i < 3; ++i)
        if (st[i] < 0 || st[i] % 8 != 0)
            return fail(SDPA_ERR_INVALID_ARG,
                        "%s_stride[%d]=%lld: strides must be non-negative multiples of 8 elements", name, i,
                        (long long)st[i]);
    return SDPA_OK;
}

// Whether any sequence has room for a key; without, the arrays may be empty (NULL).
bool holds_keys(const sdpa_cache* c) { return c->b > 0 && c->max_pages > 0; }

// A cache in 4 bits: pages of whole groups of 16 keys, one behind the other; strides in bytes.
sdpa_status_t check_groups(const sdpa_cache* c)
{
    if (c->page_size % 16 != 0)
        return fail(SDPA_ERR_UNSUPPORTED, "cache page_size=%lld: a multiple of 16 in a cache of 4 bits", (long long)c->page_size);
    const struct { const char* n; const int64_t* s; } strides[] = {{"cache k", c->k_stride}, {"cache v", c->v_stride}};
    for (const auto& x : strides) {
        if (x.s[1] != 9 * c->d)
            return fail(SDPA_ERR_INVALID_ARG, "%s_stride[1]=%lld: groups of 16 keys follow one another, 9 d = %lld bytes each",
                        x.n, (long long)x.s[1], (long long)(9 * c->d));
        for (int i = 0; i < 3; i += 2)
            if (x.s[i] < 0 || x.s[i] % 16 != 0)
                return fail(SDPA_ERR_INVALID_ARG, "%s_stride[%d]=%lld: strides must be non-negative multiples of 16 bytes", x.n, i,
                            (long long)x.s[i]);
    }
    return SDPA_OK;
}

// What a cache in 4 bits does not do.
sdpa_status_t refuse_groups(const sdpa_cache* c, const char* what)
{
    if (c->bits != 4) return SDPA_OK;
    return fail(SDPA_ERR_UNSUPPORTED, "%s: not of a cache in 4 bits (bits=4); one in its dtype is weighed and evicted", what);
}

// The cache's fields, without device access.
sdpa_status_t check_cache(const sdpa_cache* c)
{
    if (c == nullptr) return fail(SDPA_ERR_INVALID_ARG, "cache is NULL");
    if (c->dtype != SDPA_BF16 && c->dtype != SDPA_F16)
        return fail(SDPA_ERR_INVALID_ARG, "cache dtype: expected SDPA_BF16 or SDPA_F16, got %d", c->dtype);
    if (c->b < 0 || c->h_kv <= 0 || c->n_pages < 0 || c->page_size <= 0 || c->max_pages < 0)
        return fail(SDPA_ERR_INVALID_ARG,
                    "cache: b=%lld h_kv=%lld n_pages=%lld page_size=%lld max_pages=%lld (need h_kv, page_size > 0, "
                    "others >= 0)",
                    (long long)c->b, (long long)c->h_kv, (long long)c->n_pages, (long long)c->page_size,
                    (long long)c->max_pages);
    if (c->d != 64 && c->d != 128)
        return fail(SDPA_ERR_UNSUPPORTED, "cache d=%lld: only head dimensions 64 and 128 are implemented",
                    (long long)c->d);
    if (c->page_size >= kMax31 || c->max_pages >= kMax31 || c->page_size * c->max_pages > kMaxCap)
        return fail(SDPA_ERR_UNSUPPORTED, "cache capacity max_pages * page_size = %lld * %lld: at most 2^31 - 2^16 keys",
                    (long long)c->max_pages, (long long)c->page_size);
    if (c->h_kv > kMaxHeads || c->b >= kMax31 || c->b * c->h_kv >= kMax31)
        return fail(SDPA_ERR_UNSUPPORTED, "cache b * h_kv = %lld * %lld: at most 2^31 - 1, h_kv at most 4096",
                    (long long)c->b, (long long)c->h_kv);
    if (holds_keys(c) && c->page_table == nullptr && (c->max_pages != 1 || c->n_pages < c->b))
        return fail(SDPA_ERR_INVALID_ARG,
                    "cache without a page_table: max_pages=%lld n_pages=%lld (need one page per sequence)",
                    (long long)c->max_pages, (long long)c->n_pages);
    if (holds_keys(c) && (c->positions == nullptr) != (c->next_pos == nullptr))
        return fail(SDPA_ERR_INVALID_ARG, "cache positions and next_pos must both be set or both be NULL");
    if (c->bits != 0 && c->bits != 4 && c->bits != 16)
        return fail(SDPA_ERR_INVALID_ARG, "cache bits=%d: expected 0 or 16 (K and V in dtype) or 4", c->bits);
    if (c->bits == 4) return check_groups(c);
    sdpa_status_t st;
    if ((st = check_strides("cache k", c->k_stride)) != SDPA_OK) return st;
    return check_strides("cache v", c->v_stride);
}

struct Ptr {
    const char* name;
    const void* p;
    bool required;
    unsigned align;
};

template <size_t N>
sdpa_status_t check_ptrs(const Ptr (&ptrs)[N], int dev)
{
    for (const Ptr& p : ptrs) {
        const sdpa_status_t st = check_device_ptr(p.name, p.p, p.required, dev, p.align);
        if (st != SDPA_OK) return st;
    }
    return SDPA_OK;
}

sdpa_status_t current_device(int* dev)
{
    if (cudaGetDevice(dev) == cudaSuccess) return SDPA_OK;
    cudaGetLastError();
    return fail(SDPA_ERR_CUDA, "no CUDA device available");
}

sdpa_status_t check_cache_ptrs(const sdpa_cache* c, int dev)
{
    const bool held = holds_keys(c) && c->n_pages > 0;
    const Ptr ptrs[] = {{"cache k", c->k, held, 16},
                        {"cache v", c->v, held, 16},
                        {"cache page_table", c->page_table, false, 4},
                        {"cache lengths", c->lengths, c->b > 0, 4},
                        {"cache next_pos", c->next_pos, false, 4},
                        {"cache positions", c->positions, false, 4},
                        {"cache weights", c->weights, false, 4},
                        {"cache status", c->status, true, 4}};
    return check_ptrs(ptrs, dev);
}

swa::CacheView view_of(const sdpa_cache* c)
{
    swa::CacheView v{};
    v.b = c->b;
    v.h_kv = c->h_kv;
    v.d = c->d;
    v.n_pages = c->n_pages;
    v.page_size = static_cast<uint32_t>(c->page_size);
    v.max_pages = static_cast<uint32_t>(c->max_pages);
    v.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (c->page_size == int64_t(1) << i) v.page_shift = i;
    v.bits = c->bits == 4 ? 4 : 16;
    v.cap = c->page_size * c->max_pages;
    v.k = static_cast<uint16_t*>(c->k);
    v.v = static_cast<uint16_t*>(c->v);
    copy3(v.k_stride, c->k_stride);
    copy3(v.v_stride, c->v_stride);
    v.page_table = c->page_table;
    v.lengths = c->lengths;
    v.next_pos = c->next_pos;
    v.positions = c->positions;
    v.weights = c->weights;
    v.status = c->status;
    v.stall = g_test_stall;
    return v;
}

sdpa_status_t check_rows(const sdpa_cache* c, int64_t s_q, int64_t h_q, int64_t window_left, float scale)
{
    if (h_q <= 0 || h_q % c->h_kv != 0)
        return fail(SDPA_ERR_INVALID_ARG, "h_q=%lld is not a positive multiple of h_kv=%lld", (long long)h_q,
                    (long long)c->h_kv);
    if (h_q > kMaxRows || s_q > kMaxRows || s_q * h_q > kMaxRows || c->b * s_q * h_q > kMaxRows)
        return fail(SDPA_ERR_UNSUPPORTED, "b * s_q * h_q = %lld * %lld * %lld rows: at most 2^31 - 1024", (long long)c->b,
                    (long long)s_q, (long long)h_q);
    if (window_left < -1)
        return fail(SDPA_ERR_INVALID_ARG, "window_left=%lld: must be >= -1", (long long)window_left);
    if (!(scale > 0.f) || scale - scale != 0.f)
        return fail(SDPA_ERR_INVALID_ARG, "scale must be a positive finite number");
    return SDPA_OK;
}

// Sizes of a forward's work: its units (a kv-head's block of rows), the most
// key tiles that one has (as many as the room and the window allow, and the new
// tokens'), their product in floating point (it cannot overflow).
struct FwdSize {
    int64_t blocks, tiles;
    double units, total;
};

FwdSize fwd_size(const sdpa_cache* c, const sdpa_cache_fwd_params* p, const swa::CacheFwdPlan& plan)
{
    FwdSize z{};
    int64_t keys = c->page_size * c->max_pages;
    const int64_t room = keys;
    if (p->window_left >= 0 && c->positions == nullptr && p->window_left < keys) keys = p->window_left;
    const int64_t rows = p->s_q * (p->h_q / c->h_kv);
    z.blocks = (rows + plan.rows - 1) / plan.rows;
    // the reach begins up to 15 keys before (63 in the tile kernel), the new tokens end up to 15 off a group of 16
    z.tiles = (keys + (plan.variant >= swa::kTiles128 ? 78 : 30) + ((p->s_q + 15) & ~int64_t(15)) + plan.tile - 1) / plan.tile;
    if (c->bits == 4) {
        // the reach begins up to a step - 1 before (a warp's, or a tile), ends as far behind, and the new tokens are a step
        const int64_t gk = plan.variant == swa::kQ4Tiles ? plan.tile : plan.tile / 4;
        z.tiles = (imin((keys + 2 * (gk - 1)), (room + gk - 1) / gk * gk) + gk + plan.tile - 1) / plan.tile;
    }
    z.units = double(c->b) * double(c->h_kv) * double(z.blocks);
    z.total = z.units * double(z.tiles);
    return z;
}

swa::CacheFwdPlan fwd_plan(const sdpa_cache* c, const sdpa_cache_fwd_params* p)
{
    const int64_t rows = p->s_q * (p->h_q / c->h_kv);
    return c->bits == 4 ? swa::cache4_fwd_plan(c->d, rows) : swa::cache_fwd_plan(c->d, rows);
}

struct FwdLayout {
    int32_t parts, whole;
    size_t part_o, part_ml, cuts, total;
};

// Units of up to kWholeKeys keys go to one CTA each: no second launch, no
// partials. Else the work is cut into as many parts as CTAs are resident on a
// GB300 (152 SMs), fewer if there are fewer tiles; each has two partials. One
// sequence of 16 kv-heads, d = 64, one row each: 301 keys 7.8 us whole, 8.8 and
// a join of 1.5 cut; 900 keys 13.4 whole, 7.6 and 4.1 cut; 1800 keys 20.5 whole,
// 8.0 and 3.4 cut. A cache in 4 bits, calls as timed from the host: that shape
// with 301, 900, 1800 keys 12.4, 14.3, 17.4 us whole and 15.4, 16.6, 17.4 cut; its
// tile kernel (6 kv-heads of 296 rows, d = 128) 28.7, 38.6, 51.8 whole and 33.8,
// 37.1, 37.9 cut, 12 such sequences 32.9, 43.0, 59.7 whole and 57.3, 70.3, 87.0 cut.
// More units than the 304 (tiles: 152) places, 4 bits, d = 128, as timed on the device:
// 512 units of 600, 1400, 1800 keys 28.7, 41.4, 49.2 whole and 32, 46.1, 52.2 cut, of 5 to
// 1800 keys 29 and 32; with a last wave that is nearly empty, 320 units, 1000, 1400, 1800
// keys 30.7, 36.8, 45.1 whole and 31.7, 35.1, 38.8 cut, of 5 to 1800 keys 22.6 and 25.6;
// tiles, 512 units of 900 keys 272 whole and 313 cut, 160 units 103 and 109.
constexpr int64_t kWholeKeys = 512, kWholeKeys4 = 2048, kWholeKeys4Tiles = 1024;

FwdLayout fwd_layout(const sdpa_cache* c, const sdpa_cache_fwd_params* p, const swa::CacheFwdPlan& plan)
{
    FwdLayout l{};
    const FwdSize z = fwd_size(c, p, plan);
    const int64_t whole = c->bits != 4 ? kWholeKeys : plan.variant == swa::kQ4Tiles ? kWholeKeys4Tiles : kWholeKeys4;
    if (z.tiles * plan.tile <= whole && z.units < double(kMax31)) {
        l.parts = static_cast<int32_t>(z.units);
        l.whole = 1;
        return l;
    }
    l.parts = 152 * plan.occ;
    if (z.total < l.parts) l.parts = z.total < 1 ? 1 : static_cast<int32_t>(z.total);
    const size_t rows = static_cast<size_t>(l.parts) * 2 * plan.rows;
    l.part_o = 0;
    l.part_ml = align256(rows * c->d * 4);
    l.cuts = align256(l.part_ml + rows * 8);
    l.total = align256(l.cuts + l.parts * sizeof(swa::CacheFwdCut));
    return l;
}

sdpa_status_t check_fwd(const sdpa_cache* c, const sdpa_cache_fwd_params* p)
{
    sdpa_status_t st = check_cache(c);
    if (st != SDPA_OK) return st;
    if (p == nullptr) return fail(SDPA_ERR_INVALID_ARG, "params is NULL");
    if (p->s_q < 1 || p->s_q > 64)
        return fail(SDPA_ERR_UNSUPPORTED,
                    "s_q=%lld: 1 to 64 new tokens per sequence (more: up to 64 a call, appended in between)",
                    (long long)p->s_q);
    if ((st = check_rows(c, p->s_q, p->h_q, p->window_left, p->scale)) != SDPA_OK) return st;
    const struct { const char* n; const int64_t* s; } strides[] = {
        {"q", p->q_stride}, {"k", p->k_stride}, {"v", p->v_stride}, {"o", p->o_stride}};
    for (const auto& x : strides)
        if ((st = check_strides(x.n, x.s)) != SDPA_OK) return st;
    const swa::CacheFwdPlan plan = fwd_plan(c, p);
    if (fwd_size(c, p, plan).total >= double(int64_t(1) << 50))
        return fail(SDPA_ERR_UNSUPPORTED, "the forward's tiles (b * h_kv * row blocks * keys) pass 2^50");
    return SDPA_OK;
}

sdpa_status_t check_append(const sdpa_cache* c, const sdpa_cache_append_params* p)
{
    sdpa_status_t st = check_cache(c);
    if (st != SDPA_OK) return st;
    if (p == nullptr) return fail(SDPA_ERR_INVALID_ARG, "params is NULL");
    if (p->layout != SDPA_BSHD && p->layout != SDPA_THD)
        return fail(SDPA_ERR_INVALID_ARG, "layout: expected SDPA_BSHD or SDPA_THD, got %d", p->layout);
    const bool thd = p->layout == SDPA_THD;
    if (p->s < 0 || p->s >= kMax31) return fail(SDPA_ERR_INVALID_ARG, "s=%lld: must be 0 to 2^31 - 1", (long long)p->s);
    if (p->index != nullptr && (p->n < 0 || p->n >= kMax31))
        return fail(SDPA_ERR_INVALID_ARG, "n=%lld: must be 0 to 2^31 - 1", (long long)p->n);
    if (thd && p->index != nullptr) return fail(SDPA_ERR_INVALID_ARG, "index: only with SDPA_BSHD");
    if (thd && p->offsets == nullptr) return fail(SDPA_ERR_INVALID_ARG, "THD layout needs offsets");
    if (thd && p->total < 0) return fail(SDPA_ERR_INVALID_ARG, "total=%lld: must be >= 0", (long long)p->total);
    if ((st = check_strides("k", p->k_stride, thd ? 1 : 0)) != SDPA_OK) return st;
    return check_strides("v", p->v_stride, thd ? 1 : 0);
}

sdpa_status_t check_evict(const sdpa_cache* c, const sdpa_cache_evict_params* p)
{
    sdpa_status_t st = check_cache(c);
    if (st != SDPA_OK) return st;
    if (p == nullptr) return fail(SDPA_ERR_INVALID_ARG, "params is NULL");
    if ((st = refuse_groups(c, "evict")) != SDPA_OK) return st;
    if (holds_keys(c) && (c->positions == nullptr || c->weights == nullptr))
        return fail(SDPA_ERR_INVALID_ARG, "evict needs a cache with positions and weights");
    if (p->keep < 0 || p->first < 0 || p->recent < 0 || p->keep >= kMax31 || p->first > p->keep ||
        p->recent > p->keep - p->first)
        return fail(SDPA_ERR_INVALID_ARG,
                    "keep=%lld first=%lld recent=%lld: need keep >= first + recent, all >= 0, keep < 2^31",
                    (long long)p->keep, (long long)p->first, (long long)p->recent);
    if (double(c->b) * double(c->h_kv) * double(c->page_size * c->max_pages) >= double(int64_t(1) << 50))
        return fail(SDPA_ERR_UNSUPPORTED, "evict: b * h_kv * capacity passes 2^50");
    return SDPA_OK;
}

sdpa_status_t check_ws(const void* ws, size_t have, size_t need)
{
    if (need == 0) return SDPA_OK;
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return fail(SDPA_ERR_WORKSPACE, "workspace=%p must be non-NULL and 256-byte aligned", ws);
    if (have < need) return fail(SDPA_ERR_WORKSPACE, "workspace_bytes=%zu, need %zu", have, need);
    return SDPA_OK;
}

struct EvictLayout {
    int64_t m;
    size_t holes, tails, counts, total;
};

EvictLayout evict_layout(const sdpa_cache* c, const sdpa_cache_evict_params* p)
{
    EvictLayout l{};
    const int64_t cap = c->page_size * c->max_pages;
    const int64_t over = cap > p->keep ? cap - p->keep : 0;
    l.m = p->keep < over ? p->keep : over;
    const size_t units = static_cast<size_t>(c->b) * c->h_kv;
    l.holes = 0;
    l.tails = align256(units * l.m * 4);
    l.counts = align256(l.tails + units * l.m * 4);
    l.total = align256(l.counts + units * 4 + 4);
    return l;
}

}  // namespace

extern "C" {

size_t sdpa_cache_bytes(void) { return sizeof(sdpa_cache); }
size_t sdpa_cache_fwd_params_bytes(void) { return sizeof(sdpa_cache_fwd_params); }
size_t sdpa_cache_append_params_bytes(void) { return sizeof(sdpa_cache_append_params); }
size_t sdpa_cache_read_params_bytes(void) { return sizeof(sdpa_cache_read_params); }
size_t sdpa_cache_weigh_params_bytes(void) { return sizeof(sdpa_cache_weigh_params); }
size_t sdpa_cache_evict_params_bytes(void) { return sizeof(sdpa_cache_evict_params); }

size_t sdpa_cache_fwd_workspace_bytes(const sdpa_cache* c, const sdpa_cache_fwd_params* p)
{
    if (check_fwd(c, p) != SDPA_OK) return 0;
    clear_error();
    return fwd_layout(c, p, fwd_plan(c, p)).total;
}

sdpa_status_t sdpa_cache_fwd(const sdpa_cache* c, const sdpa_cache_fwd_params* p, void* ws, size_t ws_bytes,
                             void* stream)
{
    sdpa_status_t st = check_fwd(c, p);
    if (st != SDPA_OK) return st;
    const swa::CacheFwdPlan plan = fwd_plan(c, p);
    const FwdLayout l = fwd_layout(c, p, plan);
    if ((st = check_ws(ws, ws_bytes, l.total)) != SDPA_OK) return st;
    int dev = 0;
    if ((st = current_device(&dev)) != SDPA_OK) return st;
    const bool rows = c->b > 0;
    const Ptr ptrs[] = {{"q", p->q, rows, 16},     {"k", p->k, rows, 16},           {"v", p->v, rows, 16},
                        {"o", p->o, rows, 16},     {"lse", p->lse, rows, 4},        {"tree", p->tree, false, 8},
                        {"sink", p->sink, false, 4}, {"seq_q_lens", p->seq_q_lens, false, 4}, {"workspace", ws, l.total > 0, 256}};
    if ((st = check_cache_ptrs(c, dev)) != SDPA_OK || (st = check_ptrs(ptrs, dev)) != SDPA_OK) return st;
    if (!rows) return SDPA_OK;
    swa::CacheTileArgs ta{};
    swa::CacheFwdArgs& a = ta.f;
    a.c = view_of(c);
    a.s_q = static_cast<int32_t>(p->s_q);
    a.h_q = static_cast<int32_t>(p->h_q);
    a.group = static_cast<int32_t>(p->h_q / c->h_kv);
    // positions stay below 2^31 and rows within 64 of it: a wider window is none
    a.window_left = p->window_left < (int64_t(1) << 32) ? p->window_left : -1;
    a.scale_log2 = p->scale * 1.4426950408889634f;
    a.q = static_cast<const uint16_t*>(p->q);
    a.k = static_cast<const uint16_t*>(p->k);
    a.v = static_cast<const uint16_t*>(p->v);
    copy3(a.q_stride, p->q_stride);
    copy3(a.k_stride, p->k_stride);
    copy3(a.v_stride, p->v_stride);
    copy3(a.o_stride, p->o_stride);
    a.tree = p->tree;
    a.seq_q_lens = p->seq_q_lens;
    a.sink = p->sink;
    a.o = static_cast<uint16_t*>(p->o);
    a.lse = p->lse;
    a.parts = l.parts;
    a.whole = l.whole;
    a.cut_by_unit = fwd_size(c, p, plan).units <= l.parts;
    a.unit_cost = plan.unit_cost;
    a.timeout_ns = wait_limit();
    a.part_o = at<float>(ws, l.part_o);
    a.part_ml = at<float>(ws, l.part_ml);
    a.cuts = at<swa::CacheFwdCut>(ws, l.cuts);
    if (c->bits == 4) {
        ta.box_rows = plan.variant == swa::kQ4Tiles ? plan.tile : plan.tile / 4;
        while (c->page_size % ta.box_rows != 0) ta.box_rows >>= 1;
        return cuda_status(swa::launch_cache4_fwd(ta, c->dtype, static_cast<cudaStream_t>(stream)), "cache forward launch");
    }
    if (c->n_pages > 0) {
        // boxes that divide a page, of 8 rows at least: up to 64 (a key tile) for the tile kernel, 16 for the other; an unpaged
        // sequence's keys follow one another
        const bool tiles = plan.variant >= swa::kTiles128;
        int32_t rows = tiles ? 64 : 16;
        while (c->page_table != nullptr && c->page_size % rows != 0) rows >>= 1;
        if (rows >= 8 &&
            make_rows_map(&ta.tm_k, c->k, c->dtype, c->d, c->h_kv, c->page_size, c->n_pages, c->k_stride, rows) &&
            make_rows_map(&ta.tm_v, c->v, c->dtype, c->d, c->h_kv, c->page_size, c->n_pages, c->v_stride, rows))
            ta.box_rows = rows;
    }
    return cuda_status(swa::launch_cache_fwd(ta, c->dtype, static_cast<cudaStream_t>(stream)), "cache forward launch");
}

sdpa_status_t sdpa_cache_append(const sdpa_cache* c, const sdpa_cache_append_params* p, void* stream)
{
    sdpa_status_t st = check_append(c, p);
    if (st != SDPA_OK) return st;
    int dev = 0;
    if ((st = current_device(&dev)) != SDPA_OK) return st;
    const bool thd = p->layout == SDPA_THD;
    // (without rows to take, counts and offsets are still looked at)
    const bool rows = c->b > 0 && p->s > 0 && (thd ? p->total > 0 : true) && (p->index == nullptr || p->n > 0);
    const Ptr ptrs[] = {{"k", p->k, rows, 16},
                        {"v", p->v, rows, 16},
                        {"index", p->index, false, 4},
                        {"counts", p->counts, false, 4},
                        {"offsets", p->offsets, thd, 4}};
    if ((st = check_cache_ptrs(c, dev)) != SDPA_OK || (st = check_ptrs(ptrs, dev)) != SDPA_OK) return st;
    if (c->b == 0 || (!rows && !thd && p->counts == nullptr && (p->index == nullptr || p->n == 0))) return SDPA_OK;
    swa::CacheAppendArgs a{};
    a.c = view_of(c);
    a.thd = thd ? 1 : 0;
    a.s = p->s;
    a.n = p->n;
    a.total = p->total;
    a.k = static_cast<const uint16_t*>(p->k);
    a.v = static_cast<const uint16_t*>(p->v);
    copy3(a.k_stride, p->k_stride);
    copy3(a.v_stride, p->v_stride);
    a.index = p->index;
    a.counts = p->counts;
    a.offsets = thd ? p->offsets : nullptr;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return cuda_status(c->bits == 4 ? swa::launch_cache4_append(a, c->dtype, cs) : swa::launch_cache_append(a, cs),
                       "cache append launch");
}

sdpa_status_t sdpa_cache_read(const sdpa_cache* c, const sdpa_cache_read_params* p, void* stream)
{
    sdpa_status_t st = check_cache(c);
    if (st != SDPA_OK) return st;
    if (p == nullptr) return fail(SDPA_ERR_INVALID_ARG, "params is NULL");
    if (p->layout != SDPA_BSHD && p->layout != SDPA_THD)
        return fail(SDPA_ERR_INVALID_ARG, "layout: expected SDPA_BSHD or SDPA_THD, got %d", p->layout);
    const bool thd = p->layout == SDPA_THD;
    if (!thd && (p->s < 0 || p->s >= kMax31)) return fail(SDPA_ERR_INVALID_ARG, "s=%lld: must be 0 to 2^31 - 1", (long long)p->s);
    if (thd && (p->total < 0 || p->total >= kMax31))
        return fail(SDPA_ERR_INVALID_ARG, "total=%lld: must be 0 to 2^31 - 1", (long long)p->total);
    if (thd && p->offsets == nullptr) return fail(SDPA_ERR_INVALID_ARG, "THD layout needs offsets");
    if (thd && c->b == 0 && p->total > 0)
        return fail(SDPA_ERR_INVALID_ARG, "total=%lld: there are no sequences", (long long)p->total);
    const int64_t rows = c->b == 0 ? 0 : thd ? p->total : c->b * p->s;
    if (rows >= int64_t(1) << 36) return fail(SDPA_ERR_UNSUPPORTED, "b * s = %lld: at most 2^36 - 1 rows", (long long)rows);
    if ((st = check_strides("k", p->k_stride, thd ? 1 : 0)) != SDPA_OK) return st;
    if ((st = check_strides("v", p->v_stride, thd ? 1 : 0)) != SDPA_OK) return st;
    int dev = 0;
    if ((st = current_device(&dev)) != SDPA_OK) return st;
    const Ptr ptrs[] = {{"k", p->k, rows > 0, 16},
                        {"v", p->v, rows > 0, 16},
                        {"start", p->start, false, 4},
                        {"counts", p->counts, false, 4},
                        {"offsets", p->offsets, thd, 4}};
    if ((st = check_cache_ptrs(c, dev)) != SDPA_OK || (st = check_ptrs(ptrs, dev)) != SDPA_OK) return st;
    if (rows == 0) return SDPA_OK;
    swa::CacheReadArgs a{};
    a.c = view_of(c);
    a.s = p->s;
    a.rows = rows;
    a.start = p->start;
    a.counts = p->counts;
    a.offsets = thd ? p->offsets : nullptr;
    a.k = static_cast<uint16_t*>(p->k);
    a.v = static_cast<uint16_t*>(p->v);
    copy3(a.k_stride, p->k_stride);
    copy3(a.v_stride, p->v_stride);
    return cuda_status(swa::launch_cache_read(a, c->dtype, static_cast<cudaStream_t>(stream)), "cache read launch");
}

sdpa_status_t sdpa_cache_weigh(const sdpa_cache* c, const sdpa_cache_weigh_params* p, void* stream)
{
    sdpa_status_t st = check_cache(c);
    if (st != SDPA_OK) return st;
    if (p == nullptr) return fail(SDPA_ERR_INVALID_ARG, "params is NULL");
    if ((st = refuse_groups(c, "weigh")) != SDPA_OK) return st;
    if (holds_keys(c) && c->weights == nullptr) return fail(SDPA_ERR_INVALID_ARG, "weigh needs a cache with weights");
    if (p->s_q < 1) return fail(SDPA_ERR_INVALID_ARG, "s_q=%lld: must be >= 1", (long long)p->s_q);
    if ((st = check_rows(c, p->s_q, p->h_q, p->window_left, p->scale)) != SDPA_OK) return st;
    if ((st = check_strides("q", p->q_stride)) != SDPA_OK) return st;
    int dev = 0;
    if ((st = current_device(&dev)) != SDPA_OK) return st;
    const bool rows = holds_keys(c);
    const Ptr ptrs[] = {{"q", p->q, c->b > 0, 16}, {"lse", p->lse, c->b > 0, 4}, {"q_pos", p->q_pos, false, 4}};
    if ((st = check_cache_ptrs(c, dev)) != SDPA_OK || (st = check_ptrs(ptrs, dev)) != SDPA_OK) return st;
    if (!rows) return SDPA_OK;
    swa::CacheWeighArgs a{};
    a.c = view_of(c);
    a.s_q = static_cast<int32_t>(p->s_q);
    a.h_q = static_cast<int32_t>(p->h_q);
    a.group = static_cast<int32_t>(p->h_q / c->h_kv);
    a.window_left = p->window_left < (int64_t(1) << 32) ? p->window_left : -1;
    a.scale_log2 = p->scale * 1.4426950408889634f;
    a.q = static_cast<const uint16_t*>(p->q);
    copy3(a.q_stride, p->q_stride);
    a.lse = p->lse;
    a.q_pos = p->q_pos;
    a.timeout_ns = wait_limit();
    // a CTA per SM, fewer if there are fewer tiles of 128 keys
    const double tiles = double(c->b) * double(c->h_kv) * double((c->page_size * c->max_pages + 127) / 128);
    a.parts = tiles < 152 ? static_cast<int32_t>(tiles) : 152;
    if (c->n_pages > 0) {
        int32_t box = 128;
        while (c->page_table != nullptr && c->page_size % box != 0) box >>= 1;
        if (box >= 8 && make_rows_map(&a.tm_k, c->k, c->dtype, c->d, c->h_kv, c->page_size, c->n_pages, c->k_stride, box))
            a.box_rows = box;
    }
    return cuda_status(swa::launch_cache_weigh(a, c->dtype, static_cast<cudaStream_t>(stream)), "cache weigh launch");
}

size_t sdpa_cache_evict_workspace_bytes(const sdpa_cache* c, const sdpa_cache_evict_params* p)
{
    if (check_evict(c, p) != SDPA_OK) return 0;
    clear_error();
    return evict_layout(c, p).total;
}

sdpa_status_t sdpa_cache_evict(const sdpa_cache* c, const sdpa_cache_evict_params* p, void* ws, size_t ws_bytes,
                               void* stream)
{
    sdpa_status_t st = check_evict(c, p);
    if (st != SDPA_OK) return st;
    const EvictLayout l = evict_layout(c, p);
    if ((st = check_ws(ws, ws_bytes, l.total)) != SDPA_OK) return st;
    int dev = 0;
    if ((st = current_device(&dev)) != SDPA_OK) return st;
    const Ptr ptrs[] = {{"workspace", ws, true, 256}};
    if ((st = check_cache_ptrs(c, dev)) != SDPA_OK || (st = check_ptrs(ptrs, dev)) != SDPA_OK) return st;
    swa::CacheEvictArgs a{};
    a.c = view_of(c);
    a.keep = p->keep;
    a.first = p->first;
    a.recent = p->recent;
    a.m = l.m;
    a.holes = at<int32_t>(ws, l.holes);
    a.tails = at<int32_t>(ws, l.tails);
    a.counts = at<int32_t>(ws, l.counts);
    a.timeout_ns = wait_limit();
    return cuda_status(swa::launch_cache_evict(a, static_cast<cudaStream_t>(stream)), "cache evict launch");
}

sdpa_status_t sdpa_cache_test_hook(int64_t wait_limit_ns, int32_t flags)
{
    if (flags & ~1) return fail(SDPA_ERR_INVALID_ARG, "test hook flags=%d: only bit 0 is defined", flags);
    g_test_wait_ns = wait_limit_ns > 0 ? wait_limit_ns : 0;
    g_test_stall = flags;
    clear_error();
    return SDPA_OK;
}

sdpa_status_t sdpa_cache_check_status(const sdpa_cache* c, void* stream)
{
    if (c == nullptr) return fail(SDPA_ERR_INVALID_ARG, "cache is NULL");
    if (c->status == nullptr) return fail(SDPA_ERR_INVALID_ARG, "cache status is NULL");
    sdpa_status_t st = cuda_status(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)), "stream synchronize");
    if (st != SDPA_OK) return st;
    int32_t host = 0;
    if ((st = cuda_status(cudaMemcpy(&host, c->status, sizeof(host), cudaMemcpyDeviceToHost), "status read")) != SDPA_OK)
        return st;
    if (host == 0) return SDPA_OK;
    // (on the stream: ordered before the calls that follow)
    if ((st = cuda_status(cudaMemsetAsync(c->status, 0, sizeof(int32_t), static_cast<cudaStream_t>(stream)),
                          "status reset")) != SDPA_OK)
        return st;
    if (host == SDPA_ERR_BAD_LENGTHS)
        return fail(SDPA_ERR_BAD_LENGTHS, "a length, count or row index of the cache is out of its range");
    if (host == SDPA_ERR_BOUNDS) return fail(SDPA_ERR_BOUNDS, "a page-table entry is outside [0, n_pages)");
    if (host == SDPA_ERR_TIMEOUT) return fail(SDPA_ERR_TIMEOUT, "a wait of a cache call ran out on the device");
    return fail(SDPA_ERR_CUDA, "unknown cache status %d", host);
}

}  // extern "C"
