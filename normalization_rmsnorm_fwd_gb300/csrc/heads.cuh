// heads.cuh -- device helpers of the query / key kernels.
//
// A head is a row of D elements.  A row belongs to n lanes (about D / 16), each
// holding two pieces of at most 8 elements: a lane of the rotated part (the
// first ceil(R/16) lanes) holds [8l, 8l+8) and [R/2 + 8l, R/2 + 8l + 8), so
// that both members of every pair are in one lane whichever pairing is used;
// the lanes behind them hold a piece each of the two halves of the rest.  The
// rotation then needs no exchange between lanes, and the pieces that
// neighbouring lanes load are neighbours in memory (with 16 elements in a row
// in one lane instead, each load takes half of every 32-byte sector: D = 256,
// R = 64 backward beside a gate 54 instead of 44 us).  A warp works on 32 / n
// rows at a time.
//
// A piece is moved V elements at a time: 8 (16-byte accesses), or 4 or 2 where
// sizes, strides or addresses allow no more.
//
// Rows of one tensor are numbered t H + h.  A warp walks through its rows by
// running offsets (no division or product per row), and its rows stream
// through a ring of shared-memory slots filled with cp.async: every thread
// copies exactly the pieces that it will itself use, the next two steps while
// it works on two, and waits only on its own copies, so that the loads in
// flight cost no registers and no barrier.
#pragma once

#include "common.cuh"
#include "heads.h"

namespace crmsn {

#ifdef CRMSN_DEBUG
constexpr unsigned DBG_ASYNC_COPY_KIND = DBG_ASYNC_COPY;
#else
constexpr unsigned DBG_ASYNC_COPY_KIND = 0;
#endif

struct Pieces {
    int a, b;        // first element of the two pieces
    int ca, cb;      // their elements inside the row: 8, or in the row's last pieces 0 .. 8
    bool rot;        // rotated pieces
};

// WHOLE: every lane is rotated (D = R = 16 N).
template <int N, bool WHOLE>
__device__ __forceinline__ Pieces lane_pieces(int l, int R, int D)
{
    if constexpr (WHOLE) return {8 * l, 8 * l + 8 * N, 8, 8, true};
    Pieces s;
    const int turned = (R / 2 + 7) / 8;              // rotated lanes
    s.rot = l < turned;
    if (s.rot) {
        s.a = 8 * l;
        s.b = R / 2 + 8 * l;
        s.ca = s.cb = min(8, R / 2 - s.a);
    } else {
        s.a = R + 8 * (l - turned);
        s.b = s.a + (D - R + 15) / 16 * 8;
        s.ca = max(0, min(8, D - s.a));
        s.cb = max(0, min(8, D - s.b));
    }
    if (N > 0) s.ca = s.cb = 8;
    return s;
}
// The lanes of a row.
__host__ __device__ inline int row_lanes(int R, int D) { return (R / 2 + 7) / 8 + (D - R + 15) / 16; }

// The cosines and sines of a lane's 8 pairs: columns 8l.. (halves), or
// 4l.. and R/4 + 4l.. (adjacent pairs: 4 pairs in each piece).
struct Turn {
    F2 c[4], s[4];
};

__device__ __forceinline__ void ld_f32x4(const float *p, F2 &x, F2 &y)
{
    if (!dbg_global(p, 16, false)) {
        x = y = f2(0.f);
        return;
    }
    float a, b, c, d;
    asm volatile("ld.global.nc.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(a), "=f"(b), "=f"(c), "=f"(d) : "l"(p));
    x = f2(a, b);
    y = f2(c, d);
}

template <bool PAIRS, int V>
__device__ __forceinline__ void ld_turn(Turn &t, const float *row, int l, int R, const Pieces &pc)
{
    const int c0 = PAIRS ? 4 * l : 8 * l, c1 = PAIRS ? R / 4 + 4 * l : 8 * l + 4;
    if constexpr (V == 8) {
        ld_f32x4(row + c0, t.c[0], t.c[1]);
        ld_f32x4(row + c1, t.c[2], t.c[3]);
        ld_f32x4(row + R / 2 + c0, t.s[0], t.s[1]);
        ld_f32x4(row + R / 2 + c1, t.s[2], t.s[3]);
    } else {
        // As many pairs as the pieces hold; zeros behind them.
        const int pairs = PAIRS ? pc.ca / 2 : pc.ca;
        float c[8], s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool on = PAIRS ? (i & 3) < pairs : i < pairs;
            const int k = i < 4 ? c0 + i : c1 + i - 4;
            c[i] = on ? ld_f32_ro(row + k) : 0.f;
            s[i] = on ? ld_f32_ro(row + R / 2 + k) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t.c[i] = f2(c[2 * i], c[2 * i + 1]);
            t.s[i] = f2(s[2 * i], s[2 * i + 1]);
        }
    }
}

// The rotation of a lane's 8 pairs, in place: (a, b) -> (a c - b s, b c + a s)
// (INV: the transpose, by the sines' sign).
template <bool PAIRS, bool INV>
__device__ __forceinline__ void rotate(F2 (&a)[4], F2 (&b)[4], const Turn &t)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (PAIRS) {
            // a[i] and b[i] are one pair each: pair i of the piece has the
            // i-th angle of the piece (c[0..1] for a, c[2..3] for b).
            const float ca = i & 1 ? f2_hi(t.c[i / 2]) : f2_lo(t.c[i / 2]);
            const float sa = i & 1 ? f2_hi(t.s[i / 2]) : f2_lo(t.s[i / 2]);
            const float cb = i & 1 ? f2_hi(t.c[2 + i / 2]) : f2_lo(t.c[2 + i / 2]);
            const float sb = i & 1 ? f2_hi(t.s[2 + i / 2]) : f2_lo(t.s[2 + i / 2]);
            const F2 pa = f2_mul(f2(f2_hi(a[i]), f2_lo(a[i])), INV ? f2(sa, -sa) : f2(-sa, sa));
            const F2 pb = f2_mul(f2(f2_hi(b[i]), f2_lo(b[i])), INV ? f2(sb, -sb) : f2(-sb, sb));
            a[i] = f2_fma(a[i], f2(ca), pa);
            b[i] = f2_fma(b[i], f2(cb), pb);
        } else {
            // The product that is taken off is negated in a scalar FMA
            // (a packed one has no negated operand).
            const F2 s = t.s[i], c = t.c[i], as = f2_mul(a[i], s), bs = f2_mul(b[i], s);
            const F2 x = a[i], y = b[i];
            if constexpr (INV) {
                a[i] = f2_fma(x, c, bs);
                b[i] = f2(__fmaf_rn(f2_lo(y), f2_lo(c), -f2_lo(as)), __fmaf_rn(f2_hi(y), f2_hi(c), -f2_hi(as)));
            } else {
                a[i] = f2(__fmaf_rn(f2_lo(x), f2_lo(c), -f2_lo(bs)), __fmaf_rn(f2_hi(x), f2_hi(c), -f2_hi(bs)));
                b[i] = f2_fma(y, c, as);
            }
        }
    }
}

// 8 effective weights f32(w + bias) from element i on.
__device__ __forceinline__ void ld_weight8(F2 (&f)[4], const void *w, int w32, float bias, int i)
{
    if (w32) {
        const float *q = static_cast<const float *>(w) + i;
        ld_f32x4(q, f[0], f[1]);
        ld_f32x4(q + 4, f[2], f[3]);
    } else {
        const BVec<8> v = ld_keep<8>(static_cast<const uint16_t *>(w) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = f2_bf16(v.w[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = f2_add(f[j], f2(bias));
}

// The end of the kernels before: from here on their results may be read and
// their inputs overwritten.  What needs the arguments alone (a warp's first
// row, its count of rows: divisions) comes before it and overlaps with them:
// one token's append 2.06 -> 1.70 us, its angles 1.94 -> 1.41, 1001 tokens of
// 15 + 5 heads of 80 3.92 -> 3.28.
__device__ __forceinline__ void grid_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The lanes of a warp: n to a row; lanes past the last whole row are idle
// (their group is >= rows).  N > 0: n is known, and D = 16 N.
template <int N>
struct Lanes {
    int n, l, grp;   // lanes of a row; lane in its row, row in the step
    __device__ __forceinline__ explicit Lanes(int n_) : n(N > 0 ? N : n_)
    {
        const int lane = threadIdx.x & 31;
        grp = lane / n;
        l = lane - grp * n;
    }
    __device__ __forceinline__ int rows() const { return 32 / n; }
    // Sums over the lanes of a row, the same bits in all of them.
    template <int K>
    __device__ __forceinline__ void sum(float (&v)[K]) const
    {
        if constexpr (N > 0 && (N & (N - 1)) == 0) {
#pragma unroll
            for (int o = N / 2; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        } else if ((n & (n - 1)) == 0) {
            for (int o = n >> 1; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (o >= n) continue;
                    const float w = __shfl_down_sync(0xffffffffu, v[k], o);
                    if (l + o < n) v[k] += w;
                }
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], grp * n);
        }
    }
};
__device__ __forceinline__ float warp_sum(float v)
{
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A running position in [T, H, D].
template <typename E>
struct Walk {
    E *p;
    int h;
    // True when the step passes the end of a token's heads.
    __device__ __forceinline__ bool step(const Stride &s, int dh, int H)
    {
        p += s.step;
        h += dh;
        const bool over = h >= H;
        if (over) {
            h -= H;
            p += s.wrap;
        }
        return over;
    }
};

// A lane's first row in a share, and how many it has.
struct LaneRows {
    int64_t t;       // token
    int h, mine;     // head; rows of this lane
    int most;        // of any lane of the warp
    __device__ __forceinline__ LaneRows(const Share &s, int H, int warp, int grp, int rows_per_step)
    {
        const int64_t r0 = (int64_t)warp * s.run * rows_per_step + grp, rest = s.rows - r0;
        mine = 0;
        t = h = 0;
        if (grp < rows_per_step && rest > 0) {
            const int64_t runs = (rest - 1) / s.inc, last = rest - runs * s.inc;
            const int64_t in_last = (last + rows_per_step - 1) / rows_per_step;
            mine = (int)runs * s.run + (int)(in_last < s.run ? in_last : s.run);
            t = r0 / H;
            h = (int)(r0 - t * H);
        }
        most = __reduce_max_sync(0xffffffffu, mine);
    }
};

// A piece of `count` elements into a slot of the ring.  Where a row's two
// copies (its lanes' first and second pieces) meet inside a 32-byte sector the
// copies go through L1, in which the second finds what the first fetched:
// always in the general form (D = 80, R = 32 forward 47.5 -> 37.8 us, D = 32
// 58.9 -> 54.5; D = 96, whose pieces are whole sectors, loses 1 %), never in
// the wholly rotated forms, and as `l1` says in the partly rotated ones with
// known lanes (D = 64, R = 16 65.0 -> 52.8 us; D = 128 and 256, R = 64 lose
// 1 %).
template <int N, bool WHOLE, int V>
__device__ __forceinline__ void copy_piece(uint4 *slot, const uint16_t *g, int count, bool l1)
{
#pragma unroll
    for (int e = 0; e < 8; e += V) {
        if (e >= count) continue;
        uint16_t *to = reinterpret_cast<uint16_t *>(slot) + e;
        if (!dbg_shared(to, 2 * V)) continue;
        if (!dbg_global(g + e, 2 * V, false, DBG_ASYNC_COPY_KIND)) {
            for (int i = 0; i < V; ++i) to[i] = 0;
            continue;
        }
        const unsigned a = (unsigned)__cvta_generic_to_shared(to);
        if (N == 0 || (!WHOLE && l1))
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(a), "l"(g + e), "n"(2 * V) : "memory");
        else if constexpr (V == 8)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(a), "l"(g + e) : "memory");
    }
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait()
{
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}
// The CTA's dynamic shared memory.
extern __shared__ __align__(16) unsigned char heads_smem[];
__device__ __forceinline__ BVec<8> ld_slot(const uint4 *s)
{
    const uint4 q = dbg_shared(s, 16) ? *s : make_uint4(0, 0, 0, 0);
    BVec<8> v;
    v.w[0] = q.x;
    v.w[1] = q.y;
    v.w[2] = q.z;
    v.w[3] = q.w;
    return v;
}
// A piece of `count` values to BF16 memory.
template <int V>
__device__ __forceinline__ void st_piece(uint16_t *y, const F2 (&a)[4], int count)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_f2(a[i]);
#pragma unroll
    for (int e = 0; e < 8; e += V) {
        if (e >= count || !dbg_global(y + e, 2 * V, true)) continue;
        if constexpr (V == 8) *reinterpret_cast<uint4 *>(y) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (V == 4) *reinterpret_cast<uint2 *>(y + e) = make_uint2(w[e / 2], w[e / 2 + 1]);
        else *reinterpret_cast<uint32_t *>(y + e) = w[e / 2];
    }
}

// One element at a time (any alignment a BF16 or FP8 tensor can have).
__device__ __forceinline__ float ld_bf16_1(const uint16_t *p)
{
    if (!dbg_global(p, 2, false)) return 0.f;
    return __uint_as_float((uint32_t)*p << 16);
}
__device__ __forceinline__ void st_bf16_1(uint16_t *p, float v)
{
    if (!dbg_global(p, 2, true)) return;
    *p = (uint16_t)pack_bf16(v, 0.f);
}
__device__ __forceinline__ void st_u8_1(uint8_t *p, uint32_t v)
{
    if (!dbg_global(p, 1, true)) return;
    *p = (uint8_t)v;
}
__device__ __forceinline__ float weight_1(const void *w, int w32, float bias, int i)
{
    if (w32) return __fadd_rn(ld_f32_ro(static_cast<const float *>(w) + i), bias);
    return __fadd_rn(ld_bf16_1(static_cast<const uint16_t *>(w) + i), bias);
}
// The effective weights of a piece, zeros behind it.
template <int V>
__device__ __forceinline__ void ld_weights(F2 (&f)[4], const void *w, int w32, float bias, int i, int count)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = f2(0.f);
    if constexpr (V == 8) {
        if (count > 0) ld_weight8(f, w, w32, bias, i);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (2 * j < count) f[j] = f2(weight_1(w, w32, bias, i + 2 * j), weight_1(w, w32, bias, i + 2 * j + 1));
    }
}
__device__ __forceinline__ int64_t ld_index(const void *p, int is64, int64_t i)
{
    if (is64) {
        const int64_t *q = static_cast<const int64_t *>(p) + i;
        return dbg_global(q, 8, false) ? __ldg(reinterpret_cast<const long long *>(q)) : 0;
    }
    const int32_t *q = static_cast<const int32_t *>(p) + i;
    return dbg_global(q, 4, false) ? __ldg(q) : 0;
}

// The elements of pair unit u in the element-wise form: unit u < R/2 is a
// rotated pair, the units behind them are two neighbours of the rest.
__device__ __forceinline__ void unit_elems(int u, int R, int pairs, int &i, int &j)
{
    if (u < R / 2 && !pairs) {
        i = u;
        j = u + R / 2;
    } else {
        i = 2 * u;
        j = i + 1;
    }
}

}  // namespace crmsn
