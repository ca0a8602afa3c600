// rope_api.cu -- the C ABI declared in include/sdpa_rope.h: host-side argument
// checks and the launches on the caller's stream. Nothing here allocates or
// synchronises.
#include <cstring>

#include <cuda_runtime.h>

#include "../../include/sdpa_rope.h"
#include "api_util.h"
#include "rope_internal.h"

namespace {

using swa::api::check_device_ptr;
using swa::api::clear_error;
using swa::api::cuda_status;
using swa::api::fail;

constexpr int64_t kMax31 = int64_t(1) << 31;

bool finite(float x) { return x - x == 0.f; }

bool normed(const sdpa_rope_params* p) { return p->q_weight != nullptr; }

sdpa_status_t check(const sdpa_rope_params* p, bool backward)
{
    if (p == nullptr) return fail(SDPA_ERR_INVALID_ARG, "params is NULL");
    if (p->dtype != SDPA_BF16 && p->dtype != SDPA_F16)
        return fail(SDPA_ERR_INVALID_ARG, "dtype: expected SDPA_BF16 or SDPA_F16, got %d", p->dtype);
    if (p->layout != SDPA_BSHD && p->layout != SDPA_THD)
        return fail(SDPA_ERR_INVALID_ARG, "layout: expected SDPA_BSHD or SDPA_THD, got %d", p->layout);
    const bool thd = p->layout == SDPA_THD;
    if (thd ? p->total < 0 : p->b < 0 || p->s < 0)
        return fail(SDPA_ERR_INVALID_ARG, "b=%lld s=%lld total=%lld: must be >= 0", (long long)p->b, (long long)p->s,
                    (long long)p->total);
    if (thd ? p->total >= kMax31 : p->b >= kMax31 || p->s >= kMax31 || p->b * p->s >= kMax31)
        return fail(SDPA_ERR_UNSUPPORTED, "rows: at most 2^31 - 1");
    if (p->d != 64 && p->d != 128)
        return fail(SDPA_ERR_UNSUPPORTED, "d=%lld: only head dimensions 64 and 128 are implemented", (long long)p->d);
    if (p->h_q <= 0 || p->h_kv < 0 || p->h_q > (1 << 20) || p->h_kv > (1 << 20))
        return fail(SDPA_ERR_INVALID_ARG, "h_q=%lld h_kv=%lld: need 1 to 2^20 and 0 to 2^20 heads", (long long)p->h_q,
                    (long long)p->h_kv);
    if (p->rot < 0 || p->rot > p->d || p->rot % 2 != 0)
        return fail(SDPA_ERR_INVALID_ARG, "rot=%lld: an even number of features from 0 to d=%lld", (long long)p->rot,
                    (long long)p->d);
    if (p->n_axes < 1 || p->n_axes > 8) return fail(SDPA_ERR_INVALID_ARG, "n_axes=%lld: 1 to 8", (long long)p->n_axes);
    if ((p->interleaved & ~1) || (p->weight_f32 & ~1))
        return fail(SDPA_ERR_INVALID_ARG, "interleaved=%d weight_f32=%d: 0 or 1", p->interleaved, p->weight_f32);
    if (!finite(p->rot_scale) || !finite(p->weight_offset))
        return fail(SDPA_ERR_INVALID_ARG, "rot_scale and weight_offset must be finite");
    if (normed(p) && (!(p->eps > 0.f) || !finite(p->eps)))
        return fail(SDPA_ERR_INVALID_ARG, "eps must be a positive finite number");
    if (p->h_kv > 0 && normed(p) != (p->k_weight != nullptr))
        return fail(SDPA_ERR_INVALID_ARG, "q_weight and k_weight must both be set or both be NULL");
    if (thd && p->seq_lens != nullptr) return fail(SDPA_ERR_INVALID_ARG, "seq_lens: only with SDPA_BSHD");
    const struct { const char* n; const int64_t* s; bool used; } strides[] = {
        {"q", p->q_stride, !backward || normed(p)},
        {"k", p->k_stride, (!backward || normed(p)) && p->h_kv > 0},
        {"gq", p->gq_stride, backward},
        {"gk", p->gk_stride, backward && p->h_kv > 0},
        {"oq", p->oq_stride, true},
        {"ok", p->ok_stride, p->h_kv > 0}};
    for (const auto& x : strides)
        for (int i = thd ? 1 : 0; x.used && i < 3; ++i)
            if (x.s[i] < 0 || x.s[i] % 8 != 0)
                return fail(SDPA_ERR_INVALID_ARG, "%s_stride[%d]=%lld: strides must be non-negative multiples of 8 elements", x.n,
                            i, (long long)x.s[i]);
    return SDPA_OK;
}

swa::RopeArgs args_of(const sdpa_rope_params* p, bool backward)
{
    swa::RopeArgs a{};
    const bool thd = p->layout == SDPA_THD;
    const void* x[2] = {p->q, p->k};
    const void* g[2] = {p->gq, p->gk};
    void* o[2] = {p->oq, p->ok};
    const void* w[2] = {p->q_weight, p->k_weight};
    float* dw[2] = {p->dq_weight, p->dk_weight};
    const int64_t* st[2][3] = {{p->q_stride, p->gq_stride, p->oq_stride}, {p->k_stride, p->gk_stride, p->ok_stride}};
    const int64_t heads[2] = {p->h_q, p->h_kv};
    for (int n = 0; n < 2; ++n) {
        swa::RopeTensor& t = a.t[n];
        t.x = static_cast<const uint16_t*>(x[n]);
        t.g = static_cast<const uint16_t*>(g[n]);
        t.o = static_cast<uint16_t*>(o[n]);
        memcpy(t.x_stride, st[n][0], sizeof(t.x_stride));
        memcpy(t.g_stride, st[n][1], sizeof(t.g_stride));
        memcpy(t.o_stride, st[n][2], sizeof(t.o_stride));
        if (thd) t.x_stride[0] = t.g_stride[0] = t.o_stride[0] = 0;
        t.weight = w[n];
        t.dw = dw[n];
        t.heads = static_cast<int32_t>(heads[n]);
    }
    a.rows = thd ? p->total : p->b * p->s;
    a.s = thd ? (p->total > 0 ? p->total : 1) : p->s;
    a.d = static_cast<int32_t>(p->d);
    // (without rows there is nothing to turn: positions, axes and frequencies may be missing, and are not read)
    a.rot = a.rows > 0 ? static_cast<int32_t>(p->rot) : 0;
    a.n_axes = static_cast<int32_t>(p->n_axes);
    a.interleaved = p->interleaved;
    a.weight_f32 = p->weight_f32;
    a.eps = p->eps;
    a.weight_offset = p->weight_offset;
    a.rot_scale = p->rot_scale;
    a.positions = p->positions;
    a.axis = p->axis;
    a.seq_lens = p->seq_lens;
    a.freq = p->freq;
    swa::rope_plan(a, backward);
    return a;
}

size_t workspace_bytes(const sdpa_rope_params* p)
{
    if (!normed(p)) return 0;
    return (static_cast<size_t>(args_of(p, true).ctas) * 2 * p->d * sizeof(float) + 255) & ~static_cast<size_t>(255);
}

sdpa_status_t run(const sdpa_rope_params* p, bool backward, void* ws, cudaStream_t stream)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return fail(SDPA_ERR_CUDA, "no CUDA device available");
    }
    swa::RopeArgs a = args_of(p, backward);
    const bool rows = a.rows > 0, turns = rows && p->rot > 0, k = rows && p->h_kv > 0, norm = normed(p);
    const unsigned wa = p->weight_f32 ? 4 : 2;
    const struct { const char* n; const void* p; bool need; unsigned align; } ptrs[] = {
        {"positions", p->positions, turns, 4},
        {"axis", p->axis, false, 4},
        {"freq", p->freq, turns, 4},
        {"seq_lens", p->seq_lens, false, 4},
        {"q_weight", p->q_weight, false, wa},
        {"k_weight", p->k_weight, false, wa},
        {"q", p->q, rows && (!backward || norm), 16},
        {"k", p->k, k && (!backward || norm), 16},
        {"gq", p->gq, rows && backward, 16},
        {"gk", p->gk, k && backward, 16},
        {"oq", p->oq, rows, 16},
        {"ok", p->ok, k, 16},
        {"dq_weight", p->dq_weight, backward && norm, 4},
        {"dk_weight", p->dk_weight, backward && norm && p->h_kv > 0, 4},
        {"workspace", ws, backward && norm, 256}};
    for (const auto& x : ptrs) {
        const sdpa_status_t st = check_device_ptr(x.n, x.p, x.need, dev, x.align);
        if (st != SDPA_OK) return st;
    }
    if (!rows && !(backward && norm)) return SDPA_OK;
    a.partial = static_cast<float*>(ws);
    return cuda_status(swa::launch_rope(a, p->dtype, backward, stream), "rotation launch");
}

}  // namespace

extern "C" {

size_t sdpa_rope_params_bytes(void) { return sizeof(sdpa_rope_params); }

sdpa_status_t sdpa_rope_fwd(const sdpa_rope_params* p, void* stream)
{
    const sdpa_status_t st = check(p, false);
    return st != SDPA_OK ? st : run(p, false, nullptr, static_cast<cudaStream_t>(stream));
}

size_t sdpa_rope_bwd_workspace_bytes(const sdpa_rope_params* p)
{
    if (check(p, true) != SDPA_OK) return 0;
    clear_error();
    return workspace_bytes(p);
}

sdpa_status_t sdpa_rope_bwd(const sdpa_rope_params* p, void* ws, size_t ws_bytes, void* stream)
{
    const sdpa_status_t st = check(p, true);
    if (st != SDPA_OK) return st;
    const size_t need = workspace_bytes(p);
    if (need > 0) {
        if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
            return fail(SDPA_ERR_WORKSPACE, "workspace=%p must be non-NULL and 256-byte aligned", ws);
        if (ws_bytes < need) return fail(SDPA_ERR_WORKSPACE, "workspace_bytes=%zu, need %zu", ws_bytes, need);
    }
    return run(p, true, need > 0 ? ws : nullptr, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
