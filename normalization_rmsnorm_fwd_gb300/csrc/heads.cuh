// heads.cuh -- device helpers of the query / key kernels.
//
// A head is a row of D elements.  In the 16-byte form a row belongs to
// 2^lg lanes, each holding two pieces of 8 elements: a lane of the rotated
// part (the first R/16 lanes) holds [8l, 8l+8) and [R/2 + 8l, R/2 + 8l + 8),
// so that both members of every pair are in one lane whichever pairing is
// used; a lane behind them holds 16 consecutive elements of the rest.  The
// rotation then needs no exchange between lanes, and a warp's loads of one
// piece cover whole 32-byte sectors.
#pragma once

#include "common.cuh"
#include "heads.h"

namespace crmsn {

struct Pieces {
    int a, b;        // first element of the two pieces
    bool va, vb;     // piece inside the row
    bool rot;        // rotated pieces
};

__device__ __forceinline__ Pieces lane_pieces(int l, int R, int D)
{
    Pieces s;
    s.rot = l < R / 16;
    if (s.rot) {
        s.a = 8 * l;
        s.b = R / 2 + 8 * l;
        s.va = s.vb = true;
    } else {
        s.a = R + 16 * (l - R / 16);
        s.b = s.a + 8;
        s.va = s.a < D;
        s.vb = s.b < D;
    }
    return s;
}

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

template <bool PAIRS>
__device__ __forceinline__ void ld_turn(Turn &t, const float *row, int l, int R)
{
    const int c0 = PAIRS ? 4 * l : 8 * l, c1 = PAIRS ? R / 4 + 4 * l : 8 * l + 4;
    ld_f32x4(row + c0, t.c[0], t.c[1]);
    ld_f32x4(row + c1, t.c[2], t.c[3]);
    ld_f32x4(row + R / 2 + c0, t.s[0], t.s[1]);
    ld_f32x4(row + R / 2 + c1, t.s[2], t.s[3]);
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
            const F2 s = t.s[i], n = f2(-f2_lo(s), -f2_hi(s)), c = t.c[i];
            const F2 x = f2_fma(a[i], c, f2_mul(b[i], INV ? s : n));
            b[i] = f2_fma(b[i], c, f2_mul(a[i], INV ? n : s));
            a[i] = x;
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

// Sum over the 2^lg lanes of a row.
__device__ __forceinline__ float row_lanes_sum(float v, int lg)
{
    for (int o = 1 << lg >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
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
