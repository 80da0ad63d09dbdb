// rope.cu -- the cosines and sines of rotary positions on one or several axes.
//
//   out[t][j] = m cos(p f_j), out[t][R/2 + j] = m sin(p f_j),  p = pos[axis(j)][t]
//
// The angle is kept exact modulo a turn: f_j / 2 pi is turned once into a
// 64-bit fraction F of a turn, and p F modulo 2^64 (one wrapping integer
// product) is the fraction of p f_j / 2 pi, off by at most 2^-64 |p| turns:
// 2^-32 for any 32-bit position, where an FP32 product has lost every digit
// of the angle at p f = 2^24.
#include "heads.cuh"

namespace crmsn {

namespace {

constexpr int kThreads = 256;

// f / 2 pi modulo 1, as a 64-bit fraction (two's complement: -f gives -F);
// |f| < 2^40.
__device__ __forceinline__ uint64_t turn_fraction(float f)
{
    // 1 / 2 pi as the sum of two doubles.
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double x = fabs((double)f), p = x * kHi;
    const double e = __fma_rn(x, kLo, __fma_rn(x, kHi, -p));   // p + e = f / 2 pi
    const double whole = floor(p), frac = p - whole;           // exact
    const double up = floor(frac * 0x1p32), low = frac * 0x1p32 - up;
    const uint64_t F = ((uint64_t)(uint32_t)up << 32) + (uint64_t)__double2ull_rn(low * 0x1p32) +
                       (uint64_t)(int64_t)__double2ll_rn(e * 0x1p64);
    return f < 0.f ? 0 - F : F;
}

// Cosine and sine of a fraction of a turn.
__device__ __forceinline__ void turn_cos_sin(uint64_t u, float &c, float &s)
{
    // Nearest quarter turn and the signed rest, at most 1/8 turn.
    const uint32_t q = (uint32_t)((u + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(u - ((uint64_t)q << 62));
    float sn, cn;
    sincospif(__fmul_rn(__ll2float_rn(rest), 0x1p-63f), &sn, &cn);
    c = q & 1 ? sn : cn;
    s = q & 1 ? cn : sn;
    if (q == 1 || q == 2) c = -c;
    if (q & 2) s = -s;
}

__device__ __forceinline__ int column_axis(const RopeParams &p, int j)
{
    if (p.axes == 1) return 0;
    if (p.mixed) {
        const int a = j % p.axes;
        return j < p.axes * p.sections[a] ? a : 0;
    }
    int a = 0;
    while (a + 1 < p.axes && j >= p.sections[a]) j -= p.sections[a++];
    return a;
}

// Each thread keeps N neighbouring columns and takes every (grid's)th token.
template <int N>
__global__ void __launch_bounds__(kThreads) k_rope(const RopeParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    CRMSN_DEBUG_ENTER(p.dbg);
    const int groups = p.half / N;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t lanes = (int64_t)gridDim.x * kThreads / groups;   // tokens in flight
    const int g = (int)(id % groups);
    uint64_t F[N];
    int axis[N];
    bool ok[N], one = true;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float f = ld_f32_ro(p.freq + g * N + i);
        ok[i] = fabsf(f) < 0x1p40f;
        F[i] = ok[i] ? turn_fraction(f) : 0;
        axis[i] = column_axis(p, g * N + i);
        one = one && axis[i] == axis[0];
    }
    if (id / groups >= lanes) return;
    for (int64_t t = id / groups; t < p.T; t += lanes) {
        float c[N], s[N];
        uint64_t pos = (uint64_t)ld_index(p.pos, p.pos64, (int64_t)axis[0] * p.ldp + t);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!one && i > 0) pos = (uint64_t)ld_index(p.pos, p.pos64, (int64_t)axis[i] * p.ldp + t);
            turn_cos_sin(pos * F[i], c[i], s[i]);
            c[i] = ok[i] ? __fmul_rn(c[i], p.scaling) : __int_as_float(0x7fffffff);
            s[i] = ok[i] ? __fmul_rn(s[i], p.scaling) : __int_as_float(0x7fffffff);
        }
        float *row = p.out + t * p.ldo + g * N;
        if constexpr (N == 4) {
            if (dbg_global(row, 16, true))
                *reinterpret_cast<float4 *>(row) = make_float4(c[0], c[1], c[2], c[3]);
            if (dbg_global(row + p.half, 16, true))
                *reinterpret_cast<float4 *>(row + p.half) = make_float4(s[0], s[1], s[2], s[3]);
        } else {
            st_f32(row, c[0]);
            st_f32(row + p.half, s[0]);
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, bool vec, int sms, cudaStream_t s)
{
    const int64_t groups = vec ? p.half / 4 : p.half;
    const int64_t want = (p.T * groups + kThreads - 1) / kThreads;
    int64_t most = (int64_t)sms * 8;
    if (most * kThreads < groups) most = (groups + kThreads - 1) / kThreads;   // a token in flight at least
    const dim3 grid((unsigned)(want < most ? want : most));
    return vec ? launch_pdl(k_rope<4>, grid, dim3(kThreads), 0, s, p)
               : launch_pdl(k_rope<1>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace crmsn
