// heads_bwd.cuh -- the gradient of the per-head RMSNorm with rotation.
//
//   u = R(t)^T g:  u_a = g_a c + g_b s, u_b = g_b c - g_a s
//   dx = rstd (u w_eff - xhat mean(u w_eff xhat)),  xhat = x rstd
//   dw = sum over rows of u xhat
//
// rstd is computed again from x, which the row needs anyway, so the forward
// keeps nothing but its inputs.  dw: every warp adds its rows in registers in
// a fixed order, the CTA's warps are added in order into one partial row per
// CTA, and a second kernel adds the partial rows in a fixed order: the bits
// depend on the sizes, the access width and the number of SMs alone.  Each CTA
// works on q or on k, so that a lane keeps one weight and one set of sums.
#pragma once

#include <type_traits>

#include "heads.cuh"

namespace crmsn {

namespace {

constexpr int kBwdThreads = 128, kBwdWarps = kBwdThreads / 32, kBwdStages = 2 * kRun;
constexpr int kFold = 16;    // rows added plainly before they join the compensated sum

// A compensated sum as one value; an infinite or NaN sum has no low part.
__device__ __forceinline__ float joined(float h, float l) { return isfinite(h) ? __fadd_rn(h, l) : h; }

// Shared memory of a CTA: the ring of g and x pieces and, per thread, the
// compensated sums of its 16 columns, 4 to a 16-byte word.
struct BwdShared {
    uint4 ring[kBwdStages][4][kBwdThreads];
    float4 hi[4][kBwdThreads], lo[4][kBwdThreads];
};
struct BwdSharedPlain {
    uint4 ring[kBwdStages][2][kBwdThreads];
};

// The lane and the place among its 16 values of column j.
__device__ __forceinline__ void column_place(int j, int R, int D, int &l, int &i)
{
    const int first = j < R ? 0 : R, half = j < R ? R / 2 : (D - R + 15) / 16 * 8;
    const bool second = j - first >= half;
    const int k = j - first - (second ? half : 0);
    i = (k & 7) + (second ? 8 : 0);
    l = (j < R ? 0 : (R / 2 + 7) / 8) + (k >> 3);
}

// Four values (two packed pairs) join a compensated sum in shared memory.
__device__ __forceinline__ void fold4(float4 &hi, float4 &lo, F2 a, F2 b)
{
    if (!dbg_shared(&hi, 16) || !dbg_shared(&lo, 16)) return;
    float4 h = hi, l = lo;
    float e;
    two_sum(h.x, f2_lo(a), h.x, e);
    l.x = __fadd_rn(l.x, e);
    two_sum(h.y, f2_hi(a), h.y, e);
    l.y = __fadd_rn(l.y, e);
    two_sum(h.z, f2_lo(b), h.z, e);
    l.z = __fadd_rn(l.z, e);
    two_sum(h.w, f2_hi(b), h.w, e);
    l.w = __fadd_rn(l.w, e);
    hi = h;
    lo = l;
}

template <int N, bool WHOLE, int V, bool NORM, bool PAIRS>
__global__ void __launch_bounds__(kBwdThreads, kQkBwdCtasPerSm) k_qk_bwd(const QkBwdParams p)
{
    CRMSN_DEBUG_ENTER(p.dbg);
    using Shared = typename std::conditional<NORM, BwdShared, BwdSharedPlain>::type;
    Shared &sm = *reinterpret_cast<Shared *>(heads_smem);
    const int which = (int)blockIdx.x < p.share[0].blocks ? 0 : 1;
    const int block = (int)blockIdx.x - (which ? p.share[0].blocks : 0);
    const Lanes<N> L(p.lanes);
    const Pieces pc = lane_pieces<N, WHOLE>(L.l, p.R, p.D);
    const int H = p.g[which].H, tid = threadIdx.x, delta = pc.b - pc.a, P = p.cs_rows;
    const Share &sh = p.share[which];
    const LaneRows mine(sh, H, block * kBwdWarps + (tid >> 5), L.grp, L.rows());
    const int64_t t = mine.t;
    // x moves with g: its own strides, g's heads.
    Walk<const uint16_t> g = {p.g[which].p + t * p.g[which].ld + mine.h * p.g[which].hs + pc.a, mine.h};
    Walk<uint16_t> out = {const_cast<uint16_t *>(p.dx[which].p) + t * p.dx[which].ld + mine.h * p.dx[which].hs + pc.a,
                          mine.h};
    const uint16_t *x = NORM ? p.x[which].p + t * p.x[which].ld + mine.h * p.x[which].hs + pc.a : nullptr;
    grid_wait();
    int to_issue = mine.mine;
    auto issue = [&](int stage) {
        if (to_issue > 0) {
            copy_piece<N, WHOLE, V>(&sm.ring[stage][0][tid], g.p, pc.ca, p.l1);
            copy_piece<N, WHOLE, V>(&sm.ring[stage][1][tid], g.p + delta, pc.cb, p.l1);
            if constexpr (NORM) {
                copy_piece<N, WHOLE, V>(&sm.ring[stage][2][tid], x, pc.ca, p.l1);
                copy_piece<N, WHOLE, V>(&sm.ring[stage][3][tid], x + delta, pc.cb, p.l1);
            }
        }
        --to_issue;
        const int e = stage % kRun == kRun - 1;
        const bool over = g.step(sh.in[e], sh.dh[e], H);
        if constexpr (NORM) {
            x += sh.in2[e].step;
            if (over) x += sh.in2[e].wrap;
        }
    };
    // What a row's last pieces lack stays zero.
    if (N == 0 && (pc.ca < 8 || pc.cb < 8))
        for (int i = 0; i < kBwdStages; ++i)
            for (int k = 0; k < (NORM ? 4 : 2); ++k) sm.ring[i][k][tid] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kRun; ++i) issue(i);
    ring_commit();

    F2 wa[4], wb[4], ba[4], bb[4];                   // weights, sums of the last rows
    int filled = 0;
    if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ba[i] = bb[i] = f2(0.f);
            sm.hi[i][tid] = sm.lo[i][tid] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        ld_weights<V>(wa, p.w[which], p.w32, p.bias, pc.a, pc.ca);
        ld_weights<V>(wb, p.w[which], p.w32, p.bias, pc.b, pc.cb);
    }
    auto fold = [&] {
        if constexpr (NORM) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fold4(sm.hi[i][tid], sm.lo[i][tid], ba[2 * i], ba[2 * i + 1]);
                fold4(sm.hi[2 + i][tid], sm.lo[2 + i][tid], bb[2 * i], bb[2 * i + 1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) ba[i] = bb[i] = f2(0.f);
        }
        filled = 0;
    };
    int tc = (int)(t % P);
    Turn turn;
    if (pc.rot && mine.mine > 0) ld_turn<PAIRS, V>(turn, p.cs + (int64_t)tc * p.ldcs, L.l, p.R, pc);
    for (int i0 = 0; i0 < mine.most; i0 += kBwdStages) {
#pragma unroll
        for (int stage = 0; stage < kBwdStages; ++stage) {
            const int i = i0 + stage;
            if (i >= mine.most) break;
            if (stage % kRun == 0) {
#pragma unroll
                for (int k = 0; k < kRun; ++k) issue((stage + kRun + k) % kBwdStages);
                ring_commit();
                ring_wait<1>();
            }
            const bool on = i < mine.mine;
            const BVec<8> ga = ld_slot(&sm.ring[stage][0][tid]);
            const BVec<8> gb = ld_slot(&sm.ring[stage][1][tid]);
            F2 a[4], b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[k] = f2_bf16(ga.w[k]);
                b[k] = f2_bf16(gb.w[k]);
            }
            if (pc.rot) rotate<PAIRS, true>(a, b, turn);
            if constexpr (NORM) {
                const BVec<8> xa = ld_slot(&sm.ring[stage][2][tid]);
                const BVec<8> xb = ld_slot(&sm.ring[stage][3][tid]);
                F2 va[4], vb[4], ss = f2(0.f), m2 = f2(0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    va[k] = f2_bf16(xa.w[k]);
                    vb[k] = f2_bf16(xb.w[k]);
                    ss = f2_fma(va[k], va[k], ss);
                    ss = f2_fma(vb[k], vb[k], ss);
                    m2 = f2_fma(f2_mul(a[k], wa[k]), va[k], m2);
                    m2 = f2_fma(f2_mul(b[k], wb[k]), vb[k], m2);
                }
                float sum[2] = {f2_lo(ss) + f2_hi(ss), f2_lo(m2) + f2_hi(m2)};
                L.sum(sum);
                const float rstd = __frsqrt_rn(__fmaf_rn(sum[0], p.inv_d, p.eps));
                const F2 r2 = f2(on ? rstd : 0.f), n2 = f2(-__fmul_rn(__fmul_rn(sum[1], p.inv_d), rstd));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    va[k] = f2_mul(va[k], r2);
                    vb[k] = f2_mul(vb[k], r2);
                    if (on) {
                        ba[k] = f2_fma(a[k], va[k], ba[k]);
                        bb[k] = f2_fma(b[k], vb[k], bb[k]);
                    }
                    a[k] = f2_mul(r2, f2_fma(va[k], n2, f2_mul(a[k], wa[k])));
                    b[k] = f2_mul(r2, f2_fma(vb[k], n2, f2_mul(b[k], wb[k])));
                }
                if (++filled == kFold) fold();
            }
            if (on) {
                st_piece<V>(out.p, a, pc.ca);
                st_piece<V>(out.p + delta, b, pc.cb);
            }
            const int e = stage % kRun == kRun - 1;
            const bool over = out.step(sh.out[e], sh.dh[e], H);
            tc += sh.dtc[e] + over;
            if (tc >= P) tc -= P;
            if ((over || sh.dt[e] > 0) && i + 1 < mine.mine && pc.rot)
                ld_turn<PAIRS, V>(turn, p.cs + (int64_t)tc * p.ldcs, L.l, p.R, pc);
        }
    }
    if constexpr (NORM) {
        fold();
        // One partial row per CTA: each column over the warps and their row
        // groups, in order.
        __syncthreads();
        for (int j = tid; j < p.D; j += kBwdThreads) {
            int l, i;
            column_place(j, p.R, p.D, l, i);
            const float *hi = reinterpret_cast<const float *>(sm.hi[i >> 2]) + (i & 3);
            const float *lo = reinterpret_cast<const float *>(sm.lo[i >> 2]) + (i & 3);
            float h = 0.f, e = 0.f;
            for (int w = 0; w < kBwdWarps; ++w)
                for (int r = 0; r < L.rows(); ++r) {
                    const int k = 4 * (32 * w + r * L.n + l);
                    if (dbg_shared(hi + k, 4) && dbg_shared(lo + k, 4)) pair_acc(h, e, hi[k], lo[k]);
                }
            st_f32(p.part + (int64_t)blockIdx.x * p.D + j, joined(h, e));
        }
    }
}

template <int N, bool WHOLE, int V, bool NORM, bool PAIRS>
cudaError_t go_bwd(const QkBwdParams &p, dim3 grid, cudaStream_t s)
{
    constexpr size_t smem = NORM ? sizeof(BwdShared) : sizeof(BwdSharedPlain);
    static std::atomic<int> opted[kOptInDevices];
    if (cudaError_t e = opt_in_smem(k_qk_bwd<N, WHOLE, V, NORM, PAIRS>, smem, opted)) return e;
    return launch_pdl(k_qk_bwd<N, WHOLE, V, NORM, PAIRS>, grid, dim3(kBwdThreads), smem, s, p);
}

template <int N, bool WHOLE, int V>
cudaError_t go_bwd(const QkBwdParams &p, bool norm, dim3 grid, cudaStream_t s)
{
    if (norm) return p.pairs ? go_bwd<N, WHOLE, V, true, true>(p, grid, s) : go_bwd<N, WHOLE, V, true, false>(p, grid, s);
    return p.pairs ? go_bwd<N, WHOLE, V, false, true>(p, grid, s) : go_bwd<N, WHOLE, V, false, false>(p, grid, s);
}

}  // namespace

}  // namespace crmsn
