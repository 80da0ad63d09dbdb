// api_heads.cu -- the C ABI of the query / key functions declared in
// include/crmsnorm.h: argument checks and the choice of the kernel's form.
// Nothing here allocates, synchronises or throws; every check happens before
// the first launch.
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "crmsnorm.h"
#include "heads.h"

using namespace crmsn;

namespace {

// Tokens: the kernels count them, and a step beyond, in 32 bits.
constexpr int64_t kMaxTokens = 0x7ff00000, kMaxHeads = 4096, kMaxStride = (int64_t)1 << 40;

bool al(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

crmsn_status launched(cudaError_t e)
{
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return CRMSN_ERR_CUDA;
    }
    return CRMSN_OK;
}

// Up to three strided dimensions over `cols` contiguous elements.
struct Region {
    const void *p;
    int es;
    int64_t cols, n[3], s[3];
    bool out;
    int may_replace;    // index of the input it may equal, or -1
};

int64_t span_bytes(const Region &r)
{
    int64_t e = r.cols;
    for (int i = 0; i < 3; ++i) e += (r.n[i] - 1) * r.s[i];
    return e * r.es;
}

bool same_tensor(const Region &a, const Region &b)
{
    if (a.p != b.p || a.es != b.es || a.cols != b.cols) return false;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.s[i] != b.s[i])) return false;
    return true;
}

// Bytes that a region covers modulo `period`: dimensions whose stride is a
// multiple of it fall on themselves.
int64_t width_modulo(const Region &r, int64_t period)
{
    int64_t e = r.cols;
    for (int i = 0; i < 3; ++i)
        if (r.n[i] > 1 && r.s[i] * r.es % period) e += (r.n[i] - 1) * r.s[i];
    return e * r.es;
}

// True when two regions may share a byte.  Slices of one buffer that
// interleave (a common stride inside whose period they do not meet) are
// disjoint.
bool overlaps(const Region &a, const Region &b)
{
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    if (a0 + (uintptr_t)span_bytes(a) <= b0 || b0 + (uintptr_t)span_bytes(b) <= a0) return false;
    for (int i = 0; i < 3; ++i) {
        const int64_t period = a.s[i] * a.es;
        if (a.n[i] <= 1 || period <= 0) continue;
        bool shared = false;
        for (int j = 0; j < 3; ++j) shared = shared || (b.n[j] > 1 && b.s[j] * b.es == period);
        if (!shared) continue;
        const int64_t wa = width_modulo(a, period), wb = width_modulo(b, period);
        int64_t off = (int64_t)(b0 - a0) % period;
        if (off < 0) off += period;
        if (off >= wa && off + wb <= period) return false;
    }
    return true;
}

crmsn_status check_alias(const Region *ts, int n)
{
    for (int i = 0; i < n; ++i) {
        if (!ts[i].out || !ts[i].p) continue;
        for (int j = 0; j < n; ++j) {
            if (j == i || !ts[j].p) continue;
            if (ts[i].may_replace == j && same_tensor(ts[i], ts[j])) continue;
            if (ts[j].out && ts[j].may_replace == i && same_tensor(ts[i], ts[j])) continue;
            if (overlaps(ts[i], ts[j])) return CRMSN_ERR_ALIAS;
        }
    }
    return CRMSN_OK;
}

Region vec_region(const void *p, int64_t n, int es, bool out = false)
{
    return {p, es, n, {1, 1, 1}, {0, 0, 0}, out, -1};
}

#ifdef CRMSN_DEBUG
template <int N>
DebugRanges debug_ranges(const Region (&ts)[N])
{
    static_assert(N <= kDebugMaxRanges, "more tensors than debug ranges");
    DebugRanges d{};
    d.word = debug_word();
    for (int i = 0; i < N; ++i) {
        if (!ts[i].p) continue;
        d.lo[d.n] = (uintptr_t)ts[i].p;
        d.hi[d.n] = (uintptr_t)ts[i].p + (uintptr_t)span_bytes(ts[i]);
        if (ts[i].out) d.writable |= 1u << d.n;
        ++d.n;
    }
    return d;
}
#define CRMSN_SET_DEBUG(p, ts) ((p).dbg = debug_ranges(ts))
#else
#define CRMSN_SET_DEBUG(p, ts) ((void)0)
#endif

// ------------------------------------------------------------ heads ------

struct Heads {
    const void *p;
    int64_t ld, hs, H;
};

// A tensor of no heads is absent.
bool given(const Heads &h) { return h.H > 0; }

crmsn_status check_heads(const Heads &h, int64_t T, int64_t D)
{
    if (!given(h)) return CRMSN_OK;
    if (!h.p) return CRMSN_ERR_NULL;
    if ((T > 1 && (h.ld < D || h.ld > kMaxStride)) || (h.H > 1 && (h.hs < D || h.hs > kMaxStride)))
        return CRMSN_ERR_SHAPE;
    // Strides within 2^40 and at most 2^12 heads: only the span of the
    // tokens can pass 64 bits, so it is tested by division.
    if (T > 1 && h.ld > ((int64_t)1 << 60) / T) return CRMSN_ERR_SHAPE;
    if (T > 1 && h.H > 1 && h.ld < (h.H - 1) * h.hs + D && h.hs < (T - 1) * h.ld + D) return CRMSN_ERR_SHAPE;
    return al(h.p, 2) ? CRMSN_OK : CRMSN_ERR_ALIGNMENT;
}

bool heads_vec(const Heads &h, int64_t T, int v)
{
    return !given(h) || (al(h.p, 2 * v) && (T <= 1 || h.ld % v == 0) && (h.H <= 1 || h.hs % v == 0));
}

Region heads_region(const Heads &h, int64_t T, int64_t D, bool out = false, int may_replace = -1)
{
    return {given(h) ? h.p : nullptr, 2, D, {T, h.H, 1}, {T > 1 ? h.ld : 0, h.H > 1 ? h.hs : 0, 0}, out, may_replace};
}

HeadView view(const Heads &h)
{
    return {static_cast<const uint16_t *>(h.p), h.ld, h.hs, (int)h.H};
}

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

Heads heads(const crmsn_heads &h, int64_t H) { return {h.p, h.ld, h.hs, H}; }

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

// The current device and its SM count.
crmsn_status device_sms(int &dev, int &sms)
{
    dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return launched(cudaErrorNoDevice);
    sms = sm_count(dev);
    return sms > 0 ? CRMSN_OK : CRMSN_ERR_CUDA;
}

// ------------------------------------------------------------ cache ------

crmsn_status check_cache(const void *p, int64_t ps, int64_t ss, int64_t hs, int es, int64_t pages, int64_t page_size,
                         int64_t Hk, int64_t D)
{
    if (!p) return CRMSN_ERR_NULL;
    const int64_t n[3] = {pages, page_size, Hk}, s[3] = {ps, ss, hs};
    // Slots and heads must not overlap: sorted by stride, each dimension
    // steps over everything inside it.
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i) {
        if (n[i] > 1 && (s[i] < D || s[i] > kMaxStride || s[i] > ((int64_t)1 << 60) / n[i])) return CRMSN_ERR_SHAPE;
        for (int j = i; j > 0 && (n[order[j]] > 1 ? s[order[j]] : 0) < (n[order[j - 1]] > 1 ? s[order[j - 1]] : 0); --j) {
            const int x = order[j];
            order[j] = order[j - 1];
            order[j - 1] = x;
        }
    }
    int64_t extent = D;
    for (int i = 0; i < 3; ++i) {
        const int k = order[i];
        if (n[k] <= 1) continue;
        if (s[k] < extent) return CRMSN_ERR_SHAPE;
        extent += (n[k] - 1) * s[k];
    }
    return al(p, es) ? CRMSN_OK : CRMSN_ERR_ALIGNMENT;
}

bool cache_vec(const void *p, int64_t ps, int64_t ss, int64_t hs, int es, int64_t pages, int64_t page_size, int64_t Hk,
               int v)
{
    return al(p, v * es) && (pages <= 1 || ps % v == 0) && (page_size <= 1 || ss % v == 0) && (Hk <= 1 || hs % v == 0);
}

Region cache_region(const void *p, int64_t ps, int64_t ss, int64_t hs, int es, int64_t pages, int64_t page_size,
                    int64_t Hk, int64_t D)
{
    return {p, es, D, {pages, page_size, Hk},
            {pages > 1 ? ps : 0, page_size > 1 ? ss : 0, Hk > 1 ? hs : 0}, true, -1};
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
        cache_region(num_pages > 0 ? a.k_cache : nullptr, a.kps, a.kss, a.khs, es, pages, page_size, Hk, D),
        cache_region(num_pages > 0 ? a.v_cache : nullptr, a.vps, a.vss, a.vhs, es, pages, page_size, Hk, D),
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
