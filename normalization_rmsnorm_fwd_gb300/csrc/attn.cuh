// attn.cuh -- what the attention kernels share: sequences, the keys a row
// sees, where a key lies, and one row computed key by key.
//
// Scores are kept times log2(e), so that every exponential is a power of two.
#pragma once

#include "attn.h"

namespace crmsn {

// Element kinds of keys and values.
enum { KV_BF16 = CRMSN_CACHE_BF16, KV_E4M3 = CRMSN_CACHE_E4M3, KV_E5M2 = CRMSN_CACHE_E5M2 };

__device__ __forceinline__ int ld_index(const int *p)
{
    if (!dbg_global(p, 4, false)) return 0;
    return __ldg(p);
}

// Sequence b: its tokens [first, first + n) and its m keys.  Values that no
// caller may pass (sequences out of order, lengths beyond the table) are
// brought into range, so that no access leaves the tensors.
struct Seq {
    int first, n, m;
};
__device__ __forceinline__ Seq sequence(const AttnParams &p, int b)
{
    Seq s;
    if (p.starts) {
        s.first = min(max(ld_index(p.starts + b), 0), p.T);
        s.n = min(max(ld_index(p.starts + b + 1), s.first), p.T) - s.first;
    } else {
        s.first = b * p.n;
        s.n = p.n;
    }
    s.m = p.table ? min(max(ld_index(p.lens + b), 0), p.max_keys) : s.n;
    return s;
}

// The keys [lo, hi) that token i of a sequence sees.
__device__ __forceinline__ int key_hi(const AttnParams &p, const Seq &s, int i)
{
    return p.causal ? min(max(s.m - s.n + i + 1, 0), s.m) : s.m;
}
__device__ __forceinline__ int key_lo(const AttnParams &p, const Seq &s, int i)
{
    return p.window ? max(s.m - s.n + i + 1 - p.window, 0) : 0;
}

// Page and row of key j of sequence b (page < 0: a page number out of range,
// whose keys and values are zeros).
__device__ __forceinline__ void locate(const AttnParams &p, int b, const Seq &s, int j, int &page, int &row)
{
    if (p.table) {
        const int at = p.page.div(j);
        row = j - at * p.page.d;
        page = ld_index(p.table + (int64_t)b * p.ldt + at);
        if ((unsigned)page >= (unsigned)p.num_pages) page = -1;
    } else {
        page = 0;
        row = s.first + j;
    }
}
__device__ __forceinline__ int64_t kv_offset(const KvView &v, int page, int row, int h)
{
    return page * v.ps + row * v.ss + h * v.hs;
}

// One element of the keys or values in FP32 (exact).
template <int KIND>
__device__ __forceinline__ float ld_kv(const KvView &v, int64_t at)
{
    if constexpr (KIND == KV_BF16) {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(v.p) + at;
        if (!dbg_global(p, 2, false)) return 0.f;
        return __uint_as_float((uint32_t)__ldg(p) << 16);
    } else {
        const uint8_t *p = v.p + at;
        if (!dbg_global(p, 1, false)) return 0.f;
        const uint16_t b = __ldg(p);
        float f;
        if constexpr (KIND == KV_E4M3)
            asm("{\n\t.reg .b32 h;\n\t.reg .b16 a, b;\n\tcvt.rn.f16x2.e4m3x2 h, %1;\n\tmov.b32 {a, b}, h;\n\t"
                "cvt.f32.f16 %0, a;\n}" : "=f"(f) : "h"(b));
        else
            asm("{\n\t.reg .b32 h;\n\t.reg .b16 a, b;\n\tcvt.rn.f16x2.e5m2x2 h, %1;\n\tmov.b32 {a, b}, h;\n\t"
                "cvt.f32.f16 %0, a;\n}" : "=f"(f) : "h"(b));
        return f;
    }
}

__device__ __forceinline__ void st_out(uint16_t *p, float v)
{
    if (!dbg_global(p, 2, true)) return;
    *p = (uint16_t)pack_bf16(v, 0.f);
}

// Row (token i of sequence s = sequence(b), query head hq) by the whole warp,
// key by key: lane l holds the elements l, l + 32, ...; masked keys and values
// are never read.  Running maximum M and sum L in FP32:
//   M' = max(M, s_j),  L = L 2^(M-M') + 2^(s_j-M'),  o = o 2^(M-M') + 2^(s_j-M') v_j
template <int KIND, int NE>
__device__ __forceinline__ void attend_row(const AttnParams &p, int b, const Seq &s, int i, int hq, bool with_lse)
{
    const int lane = threadIdx.x & 31, h = p.group.div(hq);
    const int64_t t = s.first + i;
    float q[NE], o[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        const int d = lane + 32 * e;
        const uint16_t *a = p.q.p + t * p.q.ld + hq * p.q.hs + d;
        q[e] = 0.f;
        o[e] = 0.f;
        if (d < p.D && dbg_global(a, 2, false)) q[e] = __uint_as_float((uint32_t)*a << 16);
    }
    float c = p.qk_scale, vs = 1.f;
    if (KIND != KV_BF16) {
        c *= ld_f32_ro(p.scale[0]);
        vs = ld_f32_ro(p.scale[1]);
    }
    const int hi = key_hi(p, s, i);
    float M = -INFINITY, L = 0.f;
    for (int j = key_lo(p, s, i); j < hi; ++j) {
        int page, row;
        locate(p, b, s, j, page, row);
        const int64_t ko = kv_offset(p.kv[0], page, row, h), vo = kv_offset(p.kv[1], page, row, h);
        float k[NE], v[NE];
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int d = lane + 32 * e;
            const bool in = d < p.D && page >= 0;
            k[e] = in ? ld_kv<KIND>(p.kv[0], ko + d) : 0.f;
            v[e] = in ? ld_kv<KIND>(p.kv[1], vo + d) : 0.f;
        }
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < NE; ++e) x = fmaf(q[e], k[e], x);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        x *= c;
        const float M1 = fmaxf(M, x), base = M1 == -INFINITY ? 0.f : M1;
        const float keep = exp2f(M - base), w = exp2f(x - base);
        L = fmaf(L, keep, w);
#pragma unroll
        for (int e = 0; e < NE; ++e) o[e] = fmaf(o[e], keep, w * v[e]);
        M = M1;
    }
    const float r = L == 0.f ? 0.f : vs / L;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        const int d = lane + 32 * e;
        if (d < p.D) st_out(const_cast<uint16_t *>(p.out.p) + t * p.out.ld + hq * p.out.hs + d, o[e] * r);
    }
    if (with_lse && p.lse && lane == 0)
        st_f32(p.lse + t * p.out.H + hq, L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718f);
}

}  // namespace crmsn
