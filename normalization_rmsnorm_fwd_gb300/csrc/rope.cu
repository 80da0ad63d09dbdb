// rope.cu -- the cosines and sines of rotary positions on one or several axes.
//
//   out[t][j] = m cos(p f_j), out[t][R/2 + j] = m sin(p f_j),  p = pos[axis(j)][t]
//
// The angle is kept exact modulo a turn: f_j / 2 pi is turned once into a
// 64-bit fraction F of a turn, and p F modulo 2^64 (one wrapping integer
// product) is the fraction of p f_j / 2 pi, off by at most 2^-65 |p| turns:
// 2^-33 for any 32-bit position, where an FP32 product has lost every digit
// of the angle at p f = 2^24.
#include "heads.cuh"

namespace crmsn {

namespace {

// CTAs per SM.  Five (3, 6) instead: 131072 tokens of 128 13.5 (16.0, 14.4)
// instead of 13.0 us, 16384 tokens 3.00 instead of 2.83; 1 to 2 % better only
// where columns of several axes meet in a thread.
constexpr int kThreads = 256, kPerSm = 4;

// f / 2 pi modulo 1 as a 64-bit fraction, rounded (two's complement: -f gives
// -F); |f| < 2^40.  f = m 2^e with a whole m < 2^24; m times the first 160
// bits of 1 / 2 pi, moved to 64 bits behind the point.  Integers alone: FP64
// runs at a small fraction of the other rates here (as FP64 products, done by
// every thread, this took three quarters of the kernel's time).
__device__ __forceinline__ uint64_t turn_fraction(float f)
{
    // floor(2^160 / 2 pi), low word first.
    constexpr uint32_t K[5] = {0x36d8a566u, 0x7d4d3770u, 0x7f09d5f4u, 0x9391054au, 0x28be60dbu};
    const uint32_t bits = __float_as_uint(f) & 0x7fffffffu, ex = bits >> 23;
    const uint32_t m = ex ? (bits & 0x7fffffu) | 0x800000u : bits;
    uint32_t P[8];
    uint64_t carry = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        carry += (uint64_t)m * K[i];
        P[i] = (uint32_t)carry;
        carry >>= 32;
    }
    P[5] = (uint32_t)carry;
    P[6] = P[7] = 0;
    // P 2^(e - 96), modulo 2^64; one bit more for the rounding.
    const int shift = 95 + 150 - (int)(ex ? ex : 1), word = shift >> 5, bit = shift & 31;   // shift >= 79
    uint32_t a = 0, b = 0, c = 0;
#pragma unroll
    for (int i = 2; i < 6; ++i)
        if (word == i) {
            a = P[i];
            b = P[i + 1];
            c = P[i + 2];
        }
    const uint64_t twice = (uint64_t)__funnelshift_r(a, b, bit) | (uint64_t)__funnelshift_r(b, c, bit) << 32;
    const uint32_t top = (c >> bit) & 1u;                    // the bit above those 64
    const uint64_t F = (twice >> 1) + (twice & 1) + ((uint64_t)top << 63);
    return f < 0.f ? 0 - F : F;
}

// The nearest quarter turn q of a fraction u of a turn, and the signed rest in
// half turns, |x| <= 1/4, as an FP32 value.  u is taken as hi 2^32 + lo with
// the nearest hi and a signed lo; each part and their sum round once: within
// 2^-22 of the rest however small it is, and opposite for -u.  (An unsigned lo
// lost the digits of a small negative rest; the carry costs 1 %: 131072 tokens
// on three axes 12.8 -> 13.0 us.  Adding it in the product instead: 13.3.)
__device__ __forceinline__ float quarter(uint64_t u, uint32_t &q)
{
    const uint32_t hi = (uint32_t)((u + 0x80000000u) >> 32);
    q = (hi + 0x20000000u) >> 30;
    return __fmaf_rn(__int2float_rn((int)(hi - (q << 30))), 0x1p-31f, __fmul_rn(__int2float_rn((int)(uint32_t)u), 0x1p-63f));
}

// sin(pi x) and cos(pi x) for two |x| <= 1/4: x pi + x z Q(z) and
// 1 + z P(z), z = x^2, with Q and P fitted to the functions by Remez exchange
// (relative error 3.3e-9 of the sine, absolute 5.4e-11 of the cosine, both
// below the FP32 rounding); pi enters as the sum of two FP32 values.
__device__ __forceinline__ void sin_cos_pi(F2 x, F2 &s, F2 &c)
{
    const F2 z = f2_mul(x, x);
    F2 q = f2_fma(z, f2(-0.58901220979f), f2(2.54976104861f));
    q = f2_fma(z, q, f2(-5.16770768187f));
    q = f2_fma(z, q, f2(-9.7592573e-8f));                   // 3.14159264342 - 3.14159274101
    s = f2_fma(x, f2(3.14159274101f), f2_mul(x, q));
    F2 p = f2_fma(z, f2(0.231429548004f), f2(-1.33505846457f));
    p = f2_fma(z, p, f2(4.05870790448f));
    p = f2_fma(z, p, f2(-4.93480217341f));
    c = f2_fma(z, p, f2(1.f));
}

// The sine and cosine of the rest, turned by q quarters.
__device__ __forceinline__ void turned(uint32_t q, float sn, float cn, float &c, float &s)
{
    const float a = q & 1 ? sn : cn, b = q & 1 ? cn : sn;
    c = __uint_as_float(__float_as_uint(a) ^ (((q + 1) << 30) & 0x80000000u));
    s = __uint_as_float(__float_as_uint(b) ^ ((q << 30) & 0x80000000u));
}

// (Unrolled over the four axes, so that no section is looked up by a variable.)
__device__ __forceinline__ int column_axis(const RopeParams &p, int j)
{
    int a = 0, rest = j;
    if (p.mixed) {
        const int k = j % p.axes;
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (i == k && j < p.axes * p.sections[i]) a = i;
        return a;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (a == i && i + 1 < p.axes && rest >= p.sections[i]) {
            rest -= p.sections[i];
            a = i + 1;
        }
    return a;
}

// Each thread keeps N neighbouring columns and takes every (grid's)th token.
// Bound by the writes and, close behind, by the issue of about 34 instructions
// for a column's pair.
template <int N, bool POS64>
__global__ void __launch_bounds__(kThreads, kPerSm) k_rope(const RopeParams p)
{
    CRMSN_DEBUG_ENTER(p.dbg);
    const uint32_t groups = (uint32_t)p.half / N, id = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t lanes = gridDim.x * kThreads / groups;           // tokens in flight
    const int g = (int)(id % groups);
    int axis[N];
    bool one = true;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        axis[i] = column_axis(p, g * N + i);
        one = one && axis[i] == axis[0];
    }
    one = __all_sync(0xffffffffu, one);              // a warp takes one of the loops below
    const uint32_t first = id / groups;
    const bool any = first < lanes && first < p.T;
    int64_t at = (int64_t)axis[0] * p.ldp + first;
    grid_wait();
    uint64_t pos = one && any ? (uint64_t)ld_index(p.pos, POS64, at) : 0;
    __shared__ uint64_t column_turn[CRMSN_MAX_HEAD_DIM / 2];
    __shared__ float column_scale[CRMSN_MAX_HEAD_DIM / 2];   // the scaling, or NaN
    static_assert(CRMSN_MAX_HEAD_DIM / 2 <= kThreads, "a thread for each column");
    if ((int)threadIdx.x < p.half) {
        const float f = ld_f32_ro(p.freq + threadIdx.x);
        const bool ok = fabsf(f) < 0x1p40f;
        column_turn[threadIdx.x] = ok ? turn_fraction(f) : 0;
        column_scale[threadIdx.x] = ok ? p.scaling : __int_as_float(0x7fffffff);
    }
    __syncthreads();
    uint64_t F[N];
    float m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        F[i] = column_turn[g * N + i];
        m[i] = column_scale[g * N + i];
    }
    if (!any) return;
    // One loop for columns of one axis (one position a token), one for the
    // others.
    const int64_t by = (int64_t)lanes * p.ldo;
    float *row = p.out + first * p.ldo + g * N;
    const float *const end = p.out + p.T * p.ldo;
    const int half = p.half;
    auto emit = [&](const uint64_t (&turn)[N]) {
        float c[N], s[N], x[N];
        uint32_t q[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = quarter(turn[i], q[i]);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            F2 sn, cn;
            sin_cos_pi(f2(x[i], x[N > 1 ? i + 1 : i]), sn, cn);
            turned(q[i], f2_lo(sn), f2_lo(cn), c[i], s[i]);
            if (N > 1) turned(q[i + 1], f2_hi(sn), f2_hi(cn), c[i + 1], s[i + 1]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            c[i] = __fmul_rn(c[i], m[i]);
            s[i] = __fmul_rn(s[i], m[i]);
        }
        if constexpr (N == 4) {
            if (dbg_global(row, 16, true)) *reinterpret_cast<float4 *>(row) = make_float4(c[0], c[1], c[2], c[3]);
            if (dbg_global(row + half, 16, true))
                *reinterpret_cast<float4 *>(row + half) = make_float4(s[0], s[1], s[2], s[3]);
        } else {
            st_f32(row, c[0]);
            st_f32(row + half, s[0]);
        }
        row += by;
    };
    if (one) {
        // The next token's position is asked for while this one's is used.
        while (row < end) {
            uint64_t turn[N];
#pragma unroll
            for (int i = 0; i < N; ++i) turn[i] = pos * F[i];
            at += lanes;
            if (row + by < end) pos = (uint64_t)ld_index(p.pos, POS64, at);
            emit(turn);
        }
    } else {
        for (int64_t t = first; row < end; t += lanes) {
            uint64_t turn[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                turn[i] = (uint64_t)ld_index(p.pos, POS64, (int64_t)axis[i] * p.ldp + t) * F[i];
            emit(turn);
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, bool vec, int sms, cudaStream_t s)
{
    const int64_t groups = vec ? p.half / 4 : p.half;
    const int64_t want = (p.T * groups + kThreads - 1) / kThreads;
    static_assert(CRMSN_MAX_HEAD_DIM / 2 <= kThreads * kPerSm, "a token in flight at least");
    const int64_t most = (int64_t)sms * kPerSm;
    const dim3 grid((unsigned)(want < most ? want : most));
    const dim3 b(kThreads);
    if (vec) return p.pos64 ? launch_pdl(k_rope<4, true>, grid, b, 0, s, p) : launch_pdl(k_rope<4, false>, grid, b, 0, s, p);
    return p.pos64 ? launch_pdl(k_rope<1, true>, grid, b, 0, s, p) : launch_pdl(k_rope<1, false>, grid, b, 0, s, p);
}

}  // namespace crmsn
