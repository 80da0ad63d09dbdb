// api_heads.cu -- the C ABI of the query / key functions declared in
// include/crmsnorm.h: argument checks and the choice of the kernel's form.
// Nothing here allocates, synchronises or throws; every check happens before
// the first launch.
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "api_tensors.h"

using namespace crmsn;

namespace {

struct Common {
    const void *wq, *wk;
    int w_dtype;
    float bias, eps;
    const float *cs;
    int64_t ldcs, cs_rows, R;
    int64_t T, D, Hq, Hk;
};

Common common(const crmsn_qk_layer &l)
{
    return {l.wq, l.wk, l.w_dtype, l.weight_bias, l.eps, l.cos_sin, l.ldcs, l.cs_rows, l.R, l.T, l.D, l.Hq, l.Hk};
}

// What the three functions share; on CRMSN_OK with T == 0 there is nothing to
// launch.
crmsn_status check_common(const Common &c)
{
    if (c.T < 0 || c.T > kMaxTokens || c.Hq < 0 || c.Hk < 0 || c.Hq + c.Hk < 1 || c.Hq > kMaxHeads || c.Hk > kMaxHeads)
        return CRMSN_ERR_SHAPE;
    if (c.D < 1) return CRMSN_ERR_SHAPE;
    if (c.D > CRMSN_MAX_HEAD_DIM || (c.D & 1)) return CRMSN_ERR_UNSUPPORTED_H;
    if (c.R < 0 || c.R > c.D || (c.R & 1)) return CRMSN_ERR_SHAPE;
    if (c.w_dtype != CRMSN_BF16 && c.w_dtype != CRMSN_F32) return CRMSN_ERR_DTYPE;
    const bool norm = c.wq || c.wk;
    if (norm && (!std::isfinite(c.eps) || c.eps < 0.f || !std::isfinite(c.bias))) return CRMSN_ERR_ARG;
    if (norm && ((c.Hq && !c.wq) || (c.Hk && !c.wk))) return CRMSN_ERR_NULL;
    if (norm && (!al(c.wq, c.w_dtype == CRMSN_F32 ? 4 : 2) || !al(c.wk, c.w_dtype == CRMSN_F32 ? 4 : 2)))
        return CRMSN_ERR_ALIGNMENT;
    if (c.T == 0) return CRMSN_OK;
    if (c.R > 0) {
        if (!c.cs) return CRMSN_ERR_NULL;
        if (c.cs_rows < 1 || c.T % c.cs_rows) return CRMSN_ERR_SHAPE;
        if (c.cs_rows > 1 && (c.ldcs < c.R || c.ldcs > kMaxStride || c.ldcs > ((int64_t)1 << 60) / c.cs_rows))
            return CRMSN_ERR_SHAPE;
        if (!al(c.cs, 4)) return CRMSN_ERR_ALIGNMENT;
    }
    return CRMSN_OK;
}

// The pieces that the kernels move (heads.cuh) hold whole pairs and whole
// accesses of v elements; the 16-byte form also reads weights, cosines and
// sines by 16 bytes.
bool common_vec(const Common &c, int v)
{
    if (c.D % v || (c.R / 2) % v || (c.R / 2 + 7) / 8 + (c.D - c.R + 15) / 16 > 32) return false;
    if (v < 8) return true;
    if (c.R > 0 && (!al(c.cs, 16) || (c.cs_rows > 1 && c.ldcs % 4))) return false;
    return al(c.wq, 16) && al(c.wk, 16);
}

// The widest access that every tensor of a call allows (fits(v)), or 0.
template <typename Fits>
int widest(const Common &c, Fits fits)
{
    for (int v = 8; v >= 2; v /= 2)
        if (common_vec(c, v) && fits(v)) return v;
    return 0;
}

Region weight_region(const Common &c, const void *w)
{
    return vec_region(w, c.D, c.w_dtype == CRMSN_F32 ? 4 : 2);
}

Region cs_region(const Common &c)
{
    const bool rot = c.R > 0;
    return {rot ? c.cs : nullptr, 4, c.R, {rot ? c.cs_rows : 1, 1, 1}, {rot && c.cs_rows > 1 ? c.ldcs : 0, 0, 0}, false, -1};
}

template <typename P>
void set_common(P &p, const Common &c, int interleaved)
{
    p.w[0] = c.wq;
    p.w[1] = c.wk;
    p.w32 = c.w_dtype == CRMSN_F32;
    p.bias = c.bias;
    p.eps = c.eps;
    p.inv_d = 1.f / (float)c.D;
    p.cs = c.cs;
    p.ldcs = c.ldcs;
    p.cs_rows = c.R > 0 ? (int)c.cs_rows : 1;
    p.R = (int)c.R;
    p.pairs = interleaved != 0;
    p.T = (int)c.T;
    p.D = (int)c.D;
}

}  // namespace

// ======================================================================
extern "C" {

crmsn_status rope_cos_sin(const crmsn_rope_call *call, cudaStream_t stream)
{
    if (!call) return CRMSN_ERR_NULL;
    const int64_t T = call->T, R = call->R, ldp = call->ldp, ldcs = call->ldcs;
    const int n_axes = call->n_axes, pos_dtype = call->pos_dtype;
    const void *const positions = call->positions;
    const float *const inv_freq = call->inv_freq;
    float *const cos_sin = call->cos_sin;
    if (T < 0 || T > kMaxTokens || R < 2 || (R & 1) || R > CRMSN_MAX_HEAD_DIM || n_axes < 1 || n_axes > 4)
        return CRMSN_ERR_SHAPE;
    if (pos_dtype != CRMSN_I32 && pos_dtype != CRMSN_I64) return CRMSN_ERR_DTYPE;
    if (!std::isfinite(call->scaling)) return CRMSN_ERR_ARG;
    const int half = (int)(R / 2);
    RopeParams p{};
    int64_t sum = 0;
    for (int a = 0; a < n_axes; ++a) {
        p.sections[a] = n_axes == 1 && call->sections[0] == 0 ? half : call->sections[a];
        if (p.sections[a] < 0 || p.sections[a] > half) return CRMSN_ERR_SHAPE;
        sum += p.sections[a];
    }
    if (sum != half) return CRMSN_ERR_SHAPE;
    // Interleaved: the last column of every later axis must exist.
    for (int a = 1; call->interleaved_axes && a < n_axes; ++a)
        if (p.sections[a] > 0 && (int64_t)n_axes * (p.sections[a] - 1) + a >= half) return CRMSN_ERR_SHAPE;
    if (T == 0) return CRMSN_OK;
    if (!positions || !inv_freq || !cos_sin) return CRMSN_ERR_NULL;
    const int es = pos_dtype == CRMSN_I64 ? 8 : 4;
    // Axis stride 0: the same positions on every axis.
    if ((n_axes > 1 && ldp != 0 && (ldp < T || ldp > kMaxStride)) ||
        (T > 1 && (ldcs < R || ldcs > kMaxStride || ldcs > ((int64_t)1 << 60) / T)))
        return CRMSN_ERR_SHAPE;
    if (!al(positions, es) || !al(inv_freq, 4) || !al(cos_sin, 4)) return CRMSN_ERR_ALIGNMENT;
    const Region ts[] = {
        {positions, es, T, {n_axes, 1, 1}, {n_axes > 1 ? ldp : 0, 0, 0}, false, -1},
        vec_region(inv_freq, half, 4),
        {cos_sin, 4, R, {T, 1, 1}, {T > 1 ? ldcs : 0, 0, 0}, true, -1},
    };
    if (crmsn_status s = check_alias(ts, 3)) return s;
    int dev, sms;
    if (crmsn_status s = device_sms(dev, sms)) return s;
    CRMSN_SET_DEBUG(p, ts);
    p.pos = positions;
    p.pos64 = pos_dtype == CRMSN_I64;
    p.ldp = ldp;
    p.axes = n_axes;
    p.mixed = call->interleaved_axes != 0;
    p.freq = inv_freq;
    p.scaling = call->scaling;
    p.T = T;
    p.half = half;
    p.out = cos_sin;
    p.ldo = T > 1 ? ldcs : R;
    const bool vec = half % 4 == 0 && al(cos_sin, 16) && (T <= 1 || ldcs % 4 == 0);
    return launched(launch_rope(p, vec, sms, stream));
}

crmsn_status qk_rmsnorm_rope_fwd(const crmsn_qk_fwd_call *call, cudaStream_t stream)
{
    if (!call) return CRMSN_ERR_NULL;
    const Common c = common(call->layer);
    const int64_t T = c.T, D = c.D, Hq = c.Hq, Hk = c.Hk;
    if (crmsn_status s = check_common(c)) return s;
    if (Hq < 1) return CRMSN_ERR_SHAPE;
    if (T == 0) return CRMSN_OK;
    const Heads in[2] = {heads(call->q, Hq), heads(call->k, Hk)};
    const Heads out[2] = {heads(call->q_out, Hq), heads(call->k_out, Hk)};
    for (int i = 0; i < 2; ++i) {
        if (crmsn_status s = check_heads(in[i], T, D)) return s;
        if (crmsn_status s = check_heads(out[i], T, D)) return s;
    }
    const int vec = widest(c, [&](int v) {
        return heads_vec(in[0], T, v) && heads_vec(in[1], T, v) && heads_vec(out[0], T, v) && heads_vec(out[1], T, v);
    });
    const Region ts[] = {
        heads_region(in[0], T, D), heads_region(in[1], T, D), weight_region(c, c.wq), weight_region(c, c.wk), cs_region(c),
        heads_region(out[0], T, D, true, 0), heads_region(out[1], T, D, true, 1),
    };
    if (crmsn_status s = check_alias(ts, 7)) return s;
    int dev, sms;
    if (crmsn_status s = device_sms(dev, sms)) return s;
    QkParams p{};
    CRMSN_SET_DEBUG(p, ts);
    set_common(p, c, call->layer.interleaved);
    for (int i = 0; i < 2; ++i) {
        p.in[i] = view(in[i]);
        p.out[i] = view(out[i]);
    }
    p.heads = (int)(Hq + Hk);
    return launched(launch_qk_fwd(p, c.wq || c.wk, false, vec, sms, stream));
}

size_t qk_rmsnorm_rope_bwd_workspace_bytes(int64_t D, int device)
{
    if (D < 2 || D > CRMSN_MAX_HEAD_DIM || (D & 1)) return 0;
    const int sms = sm_count(device);
    if (sms <= 0) return 0;
    return ((size_t)sms * kQkBwdCtasPerSm * (size_t)D * sizeof(float) + 255) / 256 * 256;
}

crmsn_status qk_rmsnorm_rope_bwd(const crmsn_qk_bwd_call *call, cudaStream_t stream)
{
    if (!call) return CRMSN_ERR_NULL;
    const Common c = common(call->layer);
    const int64_t T = c.T, D = c.D, Hq = c.Hq, Hk = c.Hk;
    void *const workspace = call->workspace;
    const uint64_t workspace_bytes = call->workspace_bytes;
    if (crmsn_status s = check_common(c)) return s;
    if (Hq < 1) return CRMSN_ERR_SHAPE;
    const bool norm = c.wq || c.wk;
    float *const dw[2] = {norm ? call->dwq : nullptr, norm ? call->dwk : nullptr};
    if (norm && (!dw[0] || (Hk && !dw[1]))) return CRMSN_ERR_NULL;
    if (!al(dw[0], 4) || !al(dw[1], 4)) return CRMSN_ERR_ALIGNMENT;
    // Sums over no rows are zero.
    auto zero = [&](float *w) {
        return w ? launched(cudaMemsetAsync(w, 0, (size_t)D * sizeof(float), stream)) : CRMSN_OK;
    };
    if (T == 0) {
        if (crmsn_status s = zero(dw[0])) return s;
        return zero(dw[1]);
    }
    const Heads g[2] = {heads(call->gq, Hq), heads(call->gk, Hk)}, dx[2] = {heads(call->dq, Hq), heads(call->dk, Hk)};
    const Heads x[2] = {heads(call->q, norm ? Hq : 0), heads(call->k, norm ? Hk : 0)};
    for (int i = 0; i < 2; ++i)
        for (const Heads *h : {&g[i], &x[i], &dx[i]})
            if (crmsn_status s = check_heads(*h, T, D)) return s;
    const int vec = widest(c, [&](int v) {
        return heads_vec(g[0], T, v) && heads_vec(g[1], T, v) && heads_vec(x[0], T, v) && heads_vec(x[1], T, v) &&
               heads_vec(dx[0], T, v) && heads_vec(dx[1], T, v);
    });
    if (norm && !workspace) return CRMSN_ERR_NULL;
    if (norm && (workspace_bytes == 0 || workspace_bytes > (uint64_t)1 << 40)) return CRMSN_ERR_WORKSPACE;
    const Region ts[] = {
        heads_region(g[0], T, D), heads_region(g[1], T, D), heads_region(x[0], T, D), heads_region(x[1], T, D),
        weight_region(c, c.wq), weight_region(c, c.wk), cs_region(c),
        heads_region(dx[0], T, D, true, 0), heads_region(dx[1], T, D, true, 1),
        vec_region(dw[0], D, 4, true), vec_region(dw[1], D, 4, true),
        vec_region(norm ? workspace : nullptr, (int64_t)workspace_bytes, 1, true),
    };
    if (crmsn_status s = check_alias(ts, 12)) return s;
    int dev, sms;
    if (crmsn_status s = device_sms(dev, sms)) return s;
    if (norm && (!al(workspace, 256) || workspace_bytes < qk_rmsnorm_rope_bwd_workspace_bytes(D, dev)))
        return CRMSN_ERR_WORKSPACE;
    QkBwdParams p{};
    CRMSN_SET_DEBUG(p, ts);
    set_common(p, c, call->layer.interleaved);
    for (int i = 0; i < 2; ++i) {
        p.g[i] = view(g[i]);
        p.x[i] = view(x[i]);
        p.x[i].H = p.g[i].H;
        p.dx[i] = view(dx[i]);
        p.dw[i] = dw[i];
    }
    p.part = static_cast<float *>(workspace);
    if (Hk == 0)
        if (crmsn_status s = zero(dw[1])) return s;
    return launched(launch_qk_bwd(p, norm, vec, sms, stream));
}

crmsn_status qk_rmsnorm_rope_append(const crmsn_qk_append_call *call, cudaStream_t stream)
{
    if (!call) return CRMSN_ERR_NULL;
    const crmsn_qk_append_call &a = *call;
    const Common c = common(a.layer);
    const int64_t T = c.T, D = c.D, Hq = c.Hq, Hk = c.Hk, num_pages = a.num_pages, page_size = a.page_size;
    if (crmsn_status s = check_common(c)) return s;
    if (a.cache_kind != CRMSN_CACHE_BF16 && a.cache_kind != CRMSN_CACHE_E4M3 && a.cache_kind != CRMSN_CACHE_E5M2)
        return CRMSN_ERR_DTYPE;
    if (a.slot_dtype != CRMSN_I32 && a.slot_dtype != CRMSN_I64) return CRMSN_ERR_DTYPE;
    if (Hk < 1 || num_pages < 0 || page_size < 1 || page_size > 0x7fffffff || num_pages > 0x7fffffff / page_size)
        return CRMSN_ERR_SHAPE;
    if (T == 0) return CRMSN_OK;
    const bool fp8 = a.cache_kind != CRMSN_CACHE_BF16;
    const int es = fp8 ? 1 : 2;
    const Heads in[3] = {heads(a.q, Hq), heads(a.k, Hk), heads(a.v, Hk)}, out = heads(a.q_out, Hq);
    for (const Heads &h : in)
        if (crmsn_status s = check_heads(h, T, D)) return s;
    if (crmsn_status s = check_heads(out, T, D)) return s;
    if (!a.slots || (fp8 && (!a.k_scale || !a.v_scale))) return CRMSN_ERR_NULL;
    if (!al(a.slots, a.slot_dtype == CRMSN_I64 ? 8 : 4) || (fp8 && (!al(a.k_scale, 4) || !al(a.v_scale, 4))))
        return CRMSN_ERR_ALIGNMENT;
    if (num_pages > 0) {
        if (crmsn_status s = check_cache(a.k_cache, a.kps, a.kss, a.khs, es, num_pages, page_size, Hk, D)) return s;
        if (crmsn_status s = check_cache(a.v_cache, a.vps, a.vss, a.vhs, es, num_pages, page_size, Hk, D)) return s;
    }
    const int vec = widest(c, [&](int v) {
        return heads_vec(in[0], T, v) && heads_vec(in[1], T, v) && heads_vec(in[2], T, v) && heads_vec(out, T, v) &&
               (num_pages == 0 || (cache_vec(a.k_cache, a.kps, a.kss, a.khs, es, num_pages, page_size, Hk, v) &&
                                   cache_vec(a.v_cache, a.vps, a.vss, a.vhs, es, num_pages, page_size, Hk, v)));
    });
    const int64_t pages = num_pages > 0 ? num_pages : 1;
    const Region ts[] = {
        heads_region(in[0], T, D), heads_region(in[1], T, D), heads_region(in[2], T, D),
        weight_region(c, c.wq), weight_region(c, c.wk), cs_region(c),
        vec_region(a.slots, T, a.slot_dtype == CRMSN_I64 ? 8 : 4),
        vec_region(fp8 ? a.k_scale : nullptr, 1, 4), vec_region(fp8 ? a.v_scale : nullptr, 1, 4),
        heads_region(out, T, D, true, 0),
        cache_region(num_pages > 0 ? a.k_cache : nullptr, a.kps, a.kss, a.khs, es, pages, page_size, Hk, D, true),
        cache_region(num_pages > 0 ? a.v_cache : nullptr, a.vps, a.vss, a.vhs, es, pages, page_size, Hk, D, true),
    };
    if (crmsn_status s = check_alias(ts, 12)) return s;
    int dev, sms;
    if (crmsn_status s = device_sms(dev, sms)) return s;
    QkParams p{};
    CRMSN_SET_DEBUG(p, ts);
    set_common(p, c, call->layer.interleaved);
    for (int i = 0; i < 3; ++i) p.in[i] = view(in[i]);
    p.out[0] = view(out);
    p.cache[0] = {a.k_cache, a.kps, a.kss, a.khs};
    p.cache[1] = {a.v_cache, a.vps, a.vss, a.vhs};
    p.kind = a.cache_kind;
    p.scale[0] = a.k_scale;
    p.scale[1] = a.v_scale;
    p.slots = a.slots;
    p.slot64 = a.slot_dtype == CRMSN_I64;
    p.num_slots = num_pages * page_size;
    p.page_size = (int)page_size;
    p.heads = (int)(Hq + 2 * Hk);
    return launched(launch_qk_fwd(p, c.wq || c.wk, true, vec, sms, stream));
}

}  // extern "C"
