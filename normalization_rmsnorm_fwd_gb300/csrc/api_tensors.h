// api_tensors.h -- what the C ABI's argument checks (api_heads.cu, api_attn.cu)
// know of tensors: strided regions and their overlaps, heads, paged caches.
#pragma once

#include <cstdint>

#include "crmsnorm.h"
#include "heads.h"

namespace {

using namespace crmsn;

// Tokens: the kernels count them, and a step beyond, in 32 bits.
constexpr int64_t kMaxTokens = 0x7ff00000, kMaxHeads = 4096, kMaxStride = (int64_t)1 << 40;

inline bool al(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

inline crmsn_status launched(cudaError_t e)
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

inline int64_t span_bytes(const Region &r)
{
    int64_t e = r.cols;
    for (int i = 0; i < 3; ++i) e += (r.n[i] - 1) * r.s[i];
    return e * r.es;
}

inline bool same_tensor(const Region &a, const Region &b)
{
    if (a.p != b.p || a.es != b.es || a.cols != b.cols) return false;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.s[i] != b.s[i])) return false;
    return true;
}

// Bytes that a region covers modulo `period`: dimensions whose stride is a
// multiple of it fall on themselves.
inline int64_t width_modulo(const Region &r, int64_t period)
{
    int64_t e = r.cols;
    for (int i = 0; i < 3; ++i)
        if (r.n[i] > 1 && r.s[i] * r.es % period) e += (r.n[i] - 1) * r.s[i];
    return e * r.es;
}

// True when two regions may share a byte.  Slices of one buffer that
// interleave (a common stride inside whose period they do not meet) are
// disjoint.
inline bool overlaps(const Region &a, const Region &b)
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

inline crmsn_status check_alias(const Region *ts, int n)
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

inline Region vec_region(const void *p, int64_t n, int es, bool out = false)
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
inline bool given(const Heads &h) { return h.H > 0; }

inline crmsn_status check_heads(const Heads &h, int64_t T, int64_t D)
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

inline bool heads_vec(const Heads &h, int64_t T, int v)
{
    return !given(h) || (al(h.p, 2 * v) && (T <= 1 || h.ld % v == 0) && (h.H <= 1 || h.hs % v == 0));
}

inline Region heads_region(const Heads &h, int64_t T, int64_t D, bool out = false, int may_replace = -1)
{
    return {given(h) ? h.p : nullptr, 2, D, {T, h.H, 1}, {T > 1 ? h.ld : 0, h.H > 1 ? h.hs : 0, 0}, out, may_replace};
}

inline HeadView view(const Heads &h)
{
    return {static_cast<const uint16_t *>(h.p), h.ld, h.hs, (int)h.H};
}

inline Heads heads(const crmsn_heads &h, int64_t H) { return {h.p, h.ld, h.hs, H}; }

// The current device and its SM count.
inline crmsn_status device_sms(int &dev, int &sms)
{
    dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return launched(cudaErrorNoDevice);
    sms = sm_count(dev);
    return sms > 0 ? CRMSN_OK : CRMSN_ERR_CUDA;
}

// ------------------------------------------------------------ cache ------

inline crmsn_status check_cache(const void *p, int64_t ps, int64_t ss, int64_t hs, int es, int64_t pages, int64_t page_size,
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

inline bool cache_vec(const void *p, int64_t ps, int64_t ss, int64_t hs, int es, int64_t pages, int64_t page_size, int64_t Hk,
               int v)
{
    return al(p, v * es) && (pages <= 1 || ps % v == 0) && (page_size <= 1 || ss % v == 0) && (Hk <= 1 || hs % v == 0);
}

inline Region cache_region(const void *p, int64_t ps, int64_t ss, int64_t hs, int es, int64_t pages, int64_t page_size,
                    int64_t Hk, int64_t D, bool out)
{
    return {p, es, D, {pages, page_size, Hk},
            {pages > 1 ? ps : 0, page_size > 1 ? ss : 0, Hk > 1 ? hs : 0}, out, -1};
}

}  // namespace
