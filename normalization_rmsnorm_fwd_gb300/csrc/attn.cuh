// attn.cuh -- what the attention kernels share: sequences, the keys a row
// sees, where a key lies, and one row computed key by key.
//
// Scores are kept times log2(e), so that every exponential is a power of two.
#pragma once

#include <cfloat>

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
    return p.window ? (int)max((int64_t)s.m - s.n + i + 1 - p.window, (int64_t)0) : 0;
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
// U keys' loads are under way together (1 where this is a rare call inside
// another kernel, whose registers it would take).
template <int KIND, int NE, int U>
__device__ __noinline__ void attend_row(const AttnParams &p, int b, const Seq &s, int i, int hq, bool with_lse)
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
    for (int j = key_lo(p, s, i); j < hi; j += U) {
        float k[U][NE], v[U][NE], x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int page = -1, row = 0;
            if (j + u < hi) locate(p, b, s, j + u, page, row);
            const int64_t ko = kv_offset(p.kv[0], page, row, h), vo = kv_offset(p.kv[1], page, row, h);
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                const int d = lane + 32 * e;
                const bool in = d < p.D && page >= 0;
                k[u][e] = in ? ld_kv<KIND>(p.kv[0], ko + d) : 0.f;
                v[u][e] = in ? ld_kv<KIND>(p.kv[1], vo + d) : 0.f;
            }
        }
        float M1 = M;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = 0.f;
#pragma unroll
            for (int e = 0; e < NE; ++e) x[u] = fmaf(q[e], k[u][e], x[u]);
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) x[u] += __shfl_xor_sync(0xffffffffu, x[u], w);
            x[u] = j + u < hi ? x[u] * c : -INFINITY;
            M1 = fmaxf(M1, x[u]);
        }
        const float base = M1 == -INFINITY ? 0.f : M1, keep = exp2f(M - base);
        L *= keep;
#pragma unroll
        for (int e = 0; e < NE; ++e) o[e] *= keep;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float w = exp2f(x[u] - base);
            L += w;
#pragma unroll
            for (int e = 0; e < NE; ++e) o[e] = fmaf(w, v[u][e], o[e]);
        }
        M = M1;
    }
    const float r = L == 0.f ? 0.f : vs / L;
    __syncwarp();                                 // behind what other lanes have stored of the row before
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        const int d = lane + 32 * e;
        if (d < p.D) st_out(const_cast<uint16_t *>(p.out.p) + t * p.out.ld + hq * p.out.hs + d, o[e] * r);
    }
    if (with_lse && p.lse && lane == 0)
        st_f32(p.lse + t * p.out.H + hq, L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718f);
}

// A row's result that is not finite although its sum is: a value that the row
// does not see may have met its weight 0 in a matrix product (0 inf = NaN).
__device__ __forceinline__ bool suspect(float o, float L)
{
    return !(fabsf(o) < INFINITY) && L > 0.f && L < INFINITY;
}

// Elements of a word that are not finite, infinite, or NaN: ones in their place.
enum { V_BAD, V_INFINITE, V_NAN };
template <int KIND, int WHAT>
__device__ __forceinline__ uint32_t flags_of(uint32_t x)
{
    if constexpr (KIND == KV_BF16) {
        x &= 0x7fff7fffu;
        return WHAT == V_BAD ? __vcmpgeu2(x, 0x7f807f80u) : WHAT == V_NAN ? __vcmpgtu2(x, 0x7f807f80u) : __vcmpeq2(x, 0x7f807f80u);
    } else if constexpr (KIND == KV_E4M3) {
        return WHAT == V_INFINITE ? 0u : __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu);
    } else {
        x &= 0x7f7f7f7fu;
        return WHAT == V_BAD ? __vcmpgeu4(x, 0x7c7c7c7cu) : WHAT == V_NAN ? __vcmpgtu4(x, 0x7c7c7c7cu) : __vcmpeq4(x, 0x7c7c7c7cu);
    }
}
template <int KIND, int WHAT>
__device__ __forceinline__ uint4 flags_of(uint4 v)
{
    return make_uint4(flags_of<KIND, WHAT>(v.x), flags_of<KIND, WHAT>(v.y), flags_of<KIND, WHAT>(v.z), flags_of<KIND, WHAT>(v.w));
}
// 16 bytes of the values of key j, from byte `at` on (the forms whose rows are
// whole 16-byte pieces); zeros if its page is out of range.
template <int KIND>
__device__ __forceinline__ uint4 values_of(const AttnParams &p, int b, const Seq &s, int h, int j, int at)
{
    int page, row;
    locate(p, b, s, j, page, row);
    if (page < 0) return make_uint4(0, 0, 0, 0);
    const uint8_t *v = p.kv[1].p + kv_offset(p.kv[1], page, row, h) * (KIND == KV_BF16 ? 2 : 1) + at;
    return dbg_global(v, 16, false) ? __ldg(reinterpret_cast<const uint4 *>(v)) : make_uint4(0, 0, 0, 0);
}

// The first and the last of the keys [from, to) of sequence b whose values for
// key head h are not all finite, or (V_INFINITE) some infinite; first > last:
// none.  columns: their columns, in lane l those of piece l modulo the pieces of
// a row.  V_INFINITE: none, too, once a key of [all_from, all_to) has nothing
// but NaN.  By a whole warp.
struct BadValues {
    int first, last;
    uint4 columns;
};
template <int KIND, int WHAT>
__device__ __noinline__ BadValues bad_values(const AttnParams &p, int b, const Seq &s, int h, int from, int to, int all_from, int all_to)
{
    constexpr int U = WHAT == V_INFINITE ? 1 : 2; // loads under way together
    const int lane = threadIdx.x & 31, pieces = p.D * (KIND == KV_BF16 ? 2 : 1) / 16;
    const int rows = 32 / pieces, sub = lane / pieces, piece = lane - sub * pieces;
    const uint32_t row_lanes = pieces == 32 ? ~0u : ((1u << pieces) - 1u) << (sub * pieces & 31);
    BadValues r{0x7fffffff, -1, {0, 0, 0, 0}};
#pragma unroll 1
    for (int64_t j0 = from; j0 < to; j0 += U * rows) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t j = j0 + u * rows + sub;
            v[u] = sub < rows && j < to ? values_of<KIND>(p, b, s, h, (int)j, piece * 16) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = (int)(j0 + u * rows + sub);
            const uint4 f = flags_of<KIND, WHAT>(v[u]);
            if (f.x | f.y | f.z | f.w) {
                r.first = min(r.first, j);
                r.last = max(r.last, j);
                r.columns = make_uint4(r.columns.x | f.x, r.columns.y | f.y, r.columns.z | f.z, r.columns.w | f.w);
            }
            if constexpr (WHAT == V_INFINITE) {
                const uint4 n = flags_of<KIND, V_NAN>(v[u]);
                const uint32_t full = __ballot_sync(0xffffffffu, (n.x & n.y & n.z & n.w) == ~0u && j >= all_from && j < all_to);
                if (__any_sync(0xffffffffu, sub < rows && (full & row_lanes) == row_lanes)) return {0x7fffffff, -1, {0, 0, 0, 0}};
            }
        }
    }
    r.first = __reduce_min_sync(0xffffffffu, r.first);
    r.last = __reduce_max_sync(0xffffffffu, r.last);
    const uint4 mine = r.columns;
    for (int i = 0; i < rows; ++i) {
        const int l = i * pieces + piece;
        r.columns.x |= __shfl_sync(0xffffffffu, mine.x, l);
        r.columns.y |= __shfl_sync(0xffffffffu, mine.y, l);
        r.columns.z |= __shfl_sync(0xffffffffu, mine.z, l);
        r.columns.w |= __shfl_sync(0xffffffffu, mine.w, l);
    }
    return r;
}

// Whether a row of results, written by this CTA before a barrier, holds a value
// that is not finite.
__device__ __forceinline__ bool not_finite(const uint16_t *out, int D)
{
    uint32_t bad = 0;
    for (int d = 0; d < D; d += 8) {
        if (!dbg_global(out + d, 16, false)) continue;
        const uint4 f = flags_of<KV_BF16, V_BAD>(*reinterpret_cast<const uint4 *>(out + d));
        bad |= f.x | f.y | f.z | f.w;
    }
    return bad != 0;
}

// Each lane's row (token t of sequence b, query head hq of key head h), where it
// is suspect, is worked out again key by key if it has to be.  The tile of the
// tokens [tok, tok + ntok) loaded the keys that any of them sees: a result stands
// if no value among those that the row does not see, at most ntok - 1 on either
// side, is bad, or if the last key that it does see has NaN in all columns of
// such values.  (So a bad value that all rows see, and values that are NaN
// throughout, cost this look and no more; worked out again, a prompt of 16384
// tokens takes 1.2 s.)  Over E5M2 a weight that FP16 rounds to 0 turns an
// infinite value that the row does see into NaN as well; there the seen values
// are looked through too, up to one of nothing but NaN.  (No other kind needs
// that: E4M3 has no infinity, and BF16 weights reach down to 2^-126.)
// Kernels call this last: nothing waits for its warps, and no register is live
// across it.
template <int KIND, int NE>
__device__ __noinline__ void work_out_again(const AttnParams &p, int b, int h, int tok, int ntok, int t, int hq, bool suspect)
{
    constexpr int kNone = 0x7fffffff;
    const Seq s = sequence(p, b);
    const int i = t - s.first;
    const int lo = key_lo(p, s, i), hi = key_hi(p, s, i);
    suspect = suspect && lo < hi;                 // (without keys: the scales are to blame)
    const int first_hi = __reduce_min_sync(0xffffffffu, suspect ? hi : kNone), last_lo = __reduce_max_sync(0xffffffffu, suspect ? lo : 0);
    const BadValues above = bad_values<KIND, V_BAD>(p, b, s, h, first_hi, key_hi(p, s, tok - s.first + ntok - 1), 0, 0);
    const BadValues below = bad_values<KIND, V_BAD>(p, b, s, h, key_lo(p, s, tok - s.first), last_lo, 0, 0);
    bool seen = false;
    if (KIND == KV_E5M2) {
        const int first_lo = __reduce_min_sync(0xffffffffu, suspect ? lo : kNone), last_hi = __reduce_max_sync(0xffffffffu, suspect ? hi : 0);
        const BadValues at = bad_values<KIND, V_INFINITE>(p, b, s, h, first_lo, last_hi, last_lo, first_hi);
        seen = at.first < hi && at.last >= lo;
    }
    const bool unseen = above.last >= hi || below.first < lo;
    const int lane = threadIdx.x & 31;
    const bool piece = lane < p.D * (KIND == KV_BF16 ? 2 : 1) / 16;
    int looked = -1;
    bool covered = false;
    for (uint32_t rows = __ballot_sync(0xffffffffu, (seen || unseen) && suspect); rows; rows &= rows - 1) {
        const int l = __ffs(rows) - 1, last = __shfl_sync(0xffffffffu, hi, l) - 1;
        if (last != looked) {
            uint4 n = make_uint4(0, 0, 0, 0);
            if (piece) n = flags_of<KIND, V_NAN>(values_of<KIND>(p, b, s, h, last, lane * 16));
            covered = __all_sync(0xffffffffu, !piece || (((above.columns.x | below.columns.x) & ~n.x) | ((above.columns.y | below.columns.y) & ~n.y) |
                                                         ((above.columns.z | below.columns.z) & ~n.z) | ((above.columns.w | below.columns.w) & ~n.w)) == 0);
            looked = last;
        }
        if (covered && !__shfl_sync(0xffffffffu, seen, l)) continue;
        attend_row<KIND, NE, 1>(p, b, s, __shfl_sync(0xffffffffu, i, l), __shfl_sync(0xffffffffu, hq, l), false);
    }
}

// ------------------------------------------------------------- work split --
// All tiles (rows that share keys) of one key head, each as many units as it
// has blocks of keys, in one line; group g of C takes the units from U g / C to
// U (g + 1) / C.  So every group has the same work whatever the lengths are, and
// only the tiles at its two ends are shared with others.  A group is Hk CTAs
// (CTA g Hk + h: head h), which walk through the same keys at the same time: a
// cache that holds the heads of a slot side by side is read by whole slots.
// (One head after another reads 128 bytes of each kilobyte: 16 sequences of up
// to 16384 keys in E4M3 took 75 us.)
struct Work {
    int64_t units;               // U
    int groups;                  // C
    int64_t u0, u1;              // this group's
    int b;                       // the sequence of u0,
    int64_t rest;                // and u0 less the units of those before it
};
// Quotient of x >= 0 and d > 0 by the 32-bit division (a fifth of the cost) where that does.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t d)
{
    if (((x | d) >> 32) == 0) return (int64_t)((uint32_t)x / (uint32_t)d);
    return x / d;
}
__device__ __forceinline__ int64_t first_unit(int64_t U, int C, int g) { return quotient(U * g, C); }
// The group that takes unit u: the largest g with floor(U g / C) <= u.
__device__ __forceinline__ int unit_owner(int64_t U, int C, int64_t u) { return (int)quotient((u + 1) * C - 1, U); }

struct WorkScratch {
    int64_t sum[2][32], total[2];
    int64_t rest;
    int b;
};

// count(b, units, tiles): what sequence b has for a key head.  groups(units,
// tiles): how many share them; g: this CTA's.  All THREADS threads call this;
// sequences are counted THREADS at a time, and found again by a scan.
template <int THREADS, typename Count, typename Groups>
__device__ __forceinline__ Work share_work(int B, int g, WorkScratch &sm, Count count, Groups groups)
{
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t mine = 0, first = 0, tiles = 0;
    for (int b = tid; b < B; b += THREADS) {
        int64_t u, t;
        count(b, u, t);
        if (b == tid) first = u;
        mine += u;
        tiles += t;
    }
    for (int o = 16; o > 0; o >>= 1) {
        mine += __shfl_xor_sync(0xffffffffu, mine, o);
        tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
    }
    if (lane == 0) {
        sm.sum[0][warp] = mine;
        sm.sum[1][warp] = tiles;
    }
    __syncthreads();
    Work w;
    w.units = lane < W ? sm.sum[0][lane] : 0;
    tiles = lane < W ? sm.sum[1][lane] : 0;
    for (int o = W / 2; o > 0; o >>= 1) {
        w.units += __shfl_xor_sync(0xffffffffu, w.units, o);
        tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
    }
    w.units = __shfl_sync(0xffffffffu, w.units, 0);
    tiles = __shfl_sync(0xffffffffu, tiles, 0);
    w.groups = groups(w.units, tiles);
    w.u0 = w.u1 = w.rest = 0;
    w.b = 0;
    if (g >= w.groups) return w; // the same for all threads (no units: no groups)
    w.u0 = first_unit(w.units, w.groups, g);
    w.u1 = first_unit(w.units, w.groups, g + 1);
    // The sequence of u0: the one in which the running sum passes it.
    const int64_t want = w.u0;
    int64_t before = 0;
    for (int base = 0; base < B; base += THREADS) {
        const int b = base + tid;
        int64_t u = 0, t;
        if (base == 0) u = first;
        else if (b < B) count(b, u, t);
        int64_t incl = u;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        __syncthreads();
        if (lane == 31) sm.sum[0][warp] = incl;
        __syncthreads();
        int64_t chunk = 0;
        for (int i = 0; i < W; ++i) {
            if (i < warp) incl += sm.sum[0][i];
            chunk += sm.sum[0][i];
        }
        const int64_t lo = before + incl - u;
        if (b < B && want >= lo && want < lo + u) {
            sm.b = b;
            sm.rest = w.u0 - lo;
        }
        before += chunk;
        if (want < before) break;
    }
    __syncthreads();
    w.b = sm.b;
    w.rest = sm.rest;
    return w;
}

// Where the parts of CTA c lie.
__device__ __forceinline__ float *part_of(uint8_t *ws, int c, int which, int rows, int DP)
{
    return reinterpret_cast<float *>(ws + kAttnParts) + (int64_t)(2 * c + which) * rows * (2 + DP);
}
__device__ __forceinline__ void st_header(uint8_t *ws, int c, const AttnHeader &h)
{
    AttnHeader *at = reinterpret_cast<AttnHeader *>(ws) + c;
    if (dbg_global(at, (int)sizeof(AttnHeader), true)) *at = h;
}
__device__ __forceinline__ void st_f32x4(float *p, float a, float b, float c, float d)
{
    if (dbg_global(p, 16, true)) *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void st_u32x2(uint16_t *p, uint32_t a, uint32_t b)
{
    if (dbg_global(p, 8, true)) *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
}
__device__ __forceinline__ void st_u32x4(uint16_t *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    if (dbg_global(p, 16, true)) *reinterpret_cast<uint4 *>(p) = make_uint4(a, b, c, d);
}

// ------------------------------------------------------------ shared memory --

__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes to shared memory, zeros where `ok` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok)
{
    const int n = ok && dbg_global(src, 16, false, 3) ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two FP8 codes in the low half -> packed FP16 pair (exact).
template <int KIND>
__device__ __forceinline__ uint32_t f16_fp8(uint32_t codes)
{
    uint32_t r;
    const uint16_t c = (uint16_t)codes;
    if constexpr (KIND == KV_E4M3) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}
// Four FP8 codes -> two packed FP16 pairs.  An E5M2 code is the upper half of its
// FP16 value.
template <int KIND>
__device__ __forceinline__ void f16_codes(uint32_t codes, uint32_t &lo, uint32_t &hi)
{
    if constexpr (KIND == KV_E5M2) {
        lo = __byte_perm(codes, 0, 0x1404);
        hi = __byte_perm(codes, 0, 0x3424);
    } else {
        lo = f16_fp8<KIND>(codes);
        hi = f16_fp8<KIND>(codes >> 16);
    }
}
// Two floats -> packed FP16 pair (lo in bits 0..15), round to nearest even.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// FP8 caches: weights in FP16, whose smallest number is 2^-24.  They are held
// times a power of two, so that they reach 2^12: a small one is off by at most
// 2^-37 of the largest (2^-29 where the reference may lag by 2^8), and what
// many small ones add up to is kept.  (Up to 2^15 would fit; the rest is room
// for the exponent's rounding, 4 at scores of 2^26.)  The factor is part of the
// reference, and so of the sums.
constexpr int kWeightTop = 12;

// FP8 caches: queries in FP16.  A row is scaled by 2^e so that its largest
// element lies in [2^11, 2^12): the elements down to 2^-28 of it keep all
// their bits, and smaller ones are off by at most 2^-25, 2^-36 of the largest.
// A score is below 256 * 2^12 * 2^16 and cannot overflow.
__device__ __forceinline__ int row_exponent(float amax)
{
    if (!(amax > 0.f) || !(amax < INFINITY)) return 0;
    return 11 - (int)floorf(log2f(amax));
}
// x 2^e for |e| up to 160.
__device__ __forceinline__ float scaled(float x, int e)
{
    const int a = e / 2, b = e - a;
    return x * __int_as_float((127 + a) << 23) * __int_as_float((127 + b) << 23);
}
// Such a row's factor from products of queries and codes to scores: |c| 2^-e,
// c = scale * k_scale; c's sign goes into the queries (score_sign), so that
// masked places stay -infinity.  At least FLT_MIN, for the same reason: 0 times
// -infinity is NaN.  (Products are below 2^36: with a factor at or below FLT_MIN
// all scores are nothing beside 1.)
__device__ __forceinline__ float score_factor(float c, int e)
{
    const float f = fabsf(scaled(c, -e));
    return f < FLT_MIN ? FLT_MIN : f;
}
// What turns the signs of a packed FP16 pair.
__device__ __forceinline__ uint32_t score_sign(float c) { return c < 0.f ? 0x80008000u : 0u; }

}  // namespace crmsn
