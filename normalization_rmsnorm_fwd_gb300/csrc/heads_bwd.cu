// heads_bwd.cu -- the gradient of the per-head RMSNorm with rotation.
//
//   u = R(t)^T g:  u_a = g_a c + g_b s, u_b = g_b c - g_a s
//   dx = rstd (u w_eff - xhat mean(u w_eff xhat)),  xhat = x rstd
//   dw = sum over rows of u xhat
//
// rstd is computed again from x, which the row needs anyway, so the forward
// keeps nothing but its inputs.  dw: every warp adds its rows in registers in
// a fixed order, the CTA's warps are added in order into one partial row per
// CTA, and a second kernel adds the partial rows in a fixed order: the bits
// depend on the sizes and the number of SMs alone.  Each CTA works on q or on
// k, so that a lane keeps one weight and one set of sums.
#include <type_traits>

#include "heads.cuh"

namespace crmsn {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32, kStages = 2 * kRun;
constexpr int kFold = 16;    // rows added plainly before they join the compensated sum

// A compensated sum as one value; an infinite or NaN sum has no low part.
__device__ __forceinline__ float joined(float h, float l) { return isfinite(h) ? __fadd_rn(h, l) : h; }

// The warps' pairs [kWarps][D] (high and low parts) -> one partial row.
__device__ __forceinline__ void store_partial(const float *hi, const float *lo, int D, float *part)
{
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += kThreads) {
        float h = 0.f, l = 0.f;
        for (int w = 0; w < kWarps; ++w) pair_acc(h, l, hi[w * D + j], lo[w * D + j]);
        st_f32(part + (int64_t)blockIdx.x * D + j, joined(h, l));
    }
}

// Shared memory of a CTA: the ring of g and x pieces and, per thread, the
// compensated sums of its 16 columns, 4 to a 16-byte word.
struct BwdShared {
    uint4 ring[kStages][4][kThreads];
    float4 hi[4][kThreads], lo[4][kThreads];
};
struct BwdSharedPlain {
    uint4 ring[kStages][2][kThreads];
};

// The lane and the place among its 16 values of column j.
__device__ __forceinline__ void column_place(int j, int R, int D, int &l, int &i)
{
    const int first = j < R ? 0 : R, half = j < R ? R / 2 : (D - R + 15) / 16 * 8;
    int k = j - first;
    i = k & 7;
    if (k >= half) {
        k -= half;
        i += 8;
    }
    l = first / 16 + (k >> 3);
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

template <int N, bool WHOLE, bool NORM, bool PAIRS>
__global__ void __launch_bounds__(kThreads, kQkBwdCtasPerSm) k_qk_bwd(const QkBwdParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    CRMSN_DEBUG_ENTER(p.dbg);
    using Shared = typename std::conditional<NORM, BwdShared, BwdSharedPlain>::type;
    Shared &sm = *reinterpret_cast<Shared *>(heads_smem);
    const int which = (int)blockIdx.x < p.share[0].blocks ? 0 : 1;
    const int block = (int)blockIdx.x - (which ? p.share[0].blocks : 0);
    const Lanes<N> L(p.lanes);
    const Pieces pc = lane_pieces<N, WHOLE>(L.l, p.R, p.D);
    const int H = p.g[which].H, tid = threadIdx.x, delta = pc.b - pc.a, P = p.cs_rows;
    const Share &sh = p.share[which];
    const LaneRows mine(sh, H, block * kWarps + (tid >> 5), L.grp, L.rows());
    const int64_t t = mine.t;
    // x moves with g: its own strides, g's heads.
    Walk<const uint16_t> g = {p.g[which].p + t * p.g[which].ld + mine.h * p.g[which].hs + pc.a, mine.h};
    Walk<uint16_t> out = {const_cast<uint16_t *>(p.dx[which].p) + t * p.dx[which].ld + mine.h * p.dx[which].hs + pc.a,
                          mine.h};
    const uint16_t *x = NORM ? p.x[which].p + t * p.x[which].ld + mine.h * p.x[which].hs + pc.a : nullptr;
    int to_issue = mine.mine;
    auto issue = [&](int stage) {
        if (to_issue > 0) {
            if (pc.va) cp_async16(&sm.ring[stage][0][tid], g.p);
            if (pc.vb) cp_async16(&sm.ring[stage][1][tid], g.p + delta);
            if constexpr (NORM) {
                if (pc.va) cp_async16(&sm.ring[stage][2][tid], x);
                if (pc.vb) cp_async16(&sm.ring[stage][3][tid], x + delta);
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
    // A piece that the row has not stays zero.
    if (N == 0 && !(pc.va && pc.vb))
        for (int i = 0; i < kStages; ++i)
            for (int k = 0; k < (NORM ? 4 : 2); ++k) sm.ring[i][k][tid] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kRun; ++i) issue(i);
    ring_commit();

    F2 wa[4], wb[4], ba[4], bb[4];                   // weights, sums of the last rows
    int filled = 0;
    if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            wa[i] = wb[i] = ba[i] = bb[i] = f2(0.f);
            sm.hi[i][tid] = sm.lo[i][tid] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (pc.va) ld_weight8(wa, p.w[which], p.w32, p.bias, pc.a);
        if (pc.vb) ld_weight8(wb, p.w[which], p.w32, p.bias, pc.b);
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
    if (pc.rot && mine.mine > 0) ld_turn<PAIRS>(turn, p.cs + (int64_t)tc * p.ldcs, L.l, p.R);
    for (int i0 = 0; i0 < mine.most; i0 += kStages) {
#pragma unroll
      for (int stage = 0; stage < kStages; ++stage) {
        const int i = i0 + stage;
        if (i >= mine.most) break;
        if (stage % kRun == 0) {
#pragma unroll
            for (int k = 0; k < kRun; ++k) issue((stage + kRun + k) % kStages);
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
        if (on && pc.va) st_f2x4(out.p, a);
        if (on && pc.vb) st_f2x4(out.p + delta, b);
        const int e = stage % kRun == kRun - 1;
        const bool over = out.step(sh.out[e], sh.dh[e], H);
        tc += sh.dtc[e] + over;
        if (tc >= P) tc -= P;
        if ((over || sh.dt[e] > 0) && i + 1 < mine.mine && pc.rot) ld_turn<PAIRS>(turn, p.cs + (int64_t)tc * p.ldcs, L.l, p.R);
      }
    }
    if constexpr (NORM) {
        fold();
        // One partial row per CTA: each column over the warps and their row
        // groups, in order.
        __syncthreads();
        for (int j = tid; j < p.D; j += kThreads) {
            int l, i;
            column_place(j, p.R, p.D, l, i);
            const float *hi = reinterpret_cast<const float *>(sm.hi[i >> 2]) + (i & 3);
            const float *lo = reinterpret_cast<const float *>(sm.lo[i >> 2]) + (i & 3);
            float h = 0.f, e = 0.f;
            for (int w = 0; w < kWarps; ++w)
                for (int r = 0; r < L.rows(); ++r) {
                    const int k = 4 * (32 * w + r * L.n + l);
                    if (dbg_shared(hi + k, 4) && dbg_shared(lo + k, 4)) pair_acc(h, e, hi[k], lo[k]);
                }
            st_f32(p.part + (int64_t)blockIdx.x * p.D + j, joined(h, e));
        }
    }
}

// The element-wise form: one warp per row.
__global__ void __launch_bounds__(kThreads) k_qk_bwd_any(const QkBwdParams p, bool norm)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    CRMSN_DEBUG_ENTER(p.dbg);
    constexpr int kUnits = CRMSN_MAX_HEAD_DIM / 64;
    __shared__ float sums[2 * kWarps * CRMSN_MAX_HEAD_DIM];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, units = p.D / 2;
    const int which = (int)blockIdx.x < p.share[0].blocks ? 0 : 1;
    const HeadView G = p.g[which], X = p.x[which], Y = p.dx[which];
    float h[kUnits][2], lo[kUnits][2];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) h[k][0] = h[k][1] = lo[k][0] = lo[k][1] = 0.f;
    const int64_t rows = (int64_t)p.T * X.H, nwarps = (int64_t)p.share[which].blocks * kWarps;
    const int block = (int)blockIdx.x - (which ? p.share[0].blocks : 0);
    for (int64_t r = (int64_t)block * kWarps + warp; r < rows; r += nwarps) {
        const int t = (int)(r / X.H), head = (int)(r - (int64_t)t * X.H);
        const uint16_t *g = G.p + (int64_t)t * G.ld + (int64_t)head * G.hs;
        const uint16_t *x = norm ? X.p + (int64_t)t * X.ld + (int64_t)head * X.hs : nullptr;
        uint16_t *y = const_cast<uint16_t *>(Y.p) + (int64_t)t * Y.ld + (int64_t)head * Y.hs;
        const float *cs = p.cs + (int64_t)(t % p.cs_rows) * p.ldcs;
        float u[kUnits][2], v[kUnits][2], ss = 0.f, m = 0.f;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int n = lane + 32 * k;
            u[k][0] = u[k][1] = v[k][0] = v[k][1] = 0.f;
            if (n >= units) continue;
            int i, j;
            unit_elems(n, p.R, p.pairs, i, j);
            float a = ld_bf16_1(g + i), b = ld_bf16_1(g + j);
            if (n < p.R / 2) {
                const float c = ld_f32_ro(cs + n), s = ld_f32_ro(cs + p.R / 2 + n);
                const float z = __fmaf_rn(a, c, __fmul_rn(b, s));
                b = __fmaf_rn(b, c, -__fmul_rn(a, s));
                a = z;
            }
            u[k][0] = a;
            u[k][1] = b;
            if (norm) {
                v[k][0] = ld_bf16_1(x + i);
                v[k][1] = ld_bf16_1(x + j);
                ss = __fmaf_rn(v[k][0], v[k][0], ss);
                ss = __fmaf_rn(v[k][1], v[k][1], ss);
                m = __fmaf_rn(__fmul_rn(a, weight_1(p.w[which], p.w32, p.bias, i)), v[k][0], m);
                m = __fmaf_rn(__fmul_rn(b, weight_1(p.w[which], p.w32, p.bias, j)), v[k][1], m);
            }
        }
        float rstd = 1.f, along = 0.f;
        if (norm) {
            rstd = __frsqrt_rn(__fadd_rn(__fmul_rn(warp_sum(ss), p.inv_d), p.eps));
            along = __fmul_rn(__fmul_rn(warp_sum(m), p.inv_d), rstd);
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int n = lane + 32 * k;
            if (n >= units) continue;
            int e[2];
            unit_elems(n, p.R, p.pairs, e[0], e[1]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float d = u[k][q];
                if (norm) {
                    const float xh = __fmul_rn(v[k][q], rstd);
                    d = __fmul_rn(rstd, __fmaf_rn(xh, -along, __fmul_rn(d, weight_1(p.w[which], p.w32, p.bias, e[q]))));
                    float s, err;
                    two_sum(h[k][q], __fmul_rn(u[k][q], xh), s, err);
                    h[k][q] = s;
                    lo[k][q] = __fadd_rn(lo[k][q], err);
                }
                st_bf16_1(y + e[q], d);
            }
        }
    }
    if (!norm) return;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int n = lane + 32 * k;
        if (n >= units) continue;
        int e[2];
        unit_elems(n, p.R, p.pairs, e[0], e[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            sums[warp * p.D + e[q]] = h[k][q];
            sums[(kWarps + warp) * p.D + e[q]] = lo[k][q];
        }
    }
    store_partial(sums, sums + kWarps * p.D, p.D, p.part);
}

// dw[j] = sum over the CTAs' partial rows, compensated, in a fixed order: a
// block covers 32 columns of dwq (blockIdx.y 0) or dwk, warp w a contiguous
// range of rows with up to kBatch loads in flight, then warp j adds the
// warps' pairs of column j in a butterfly.
constexpr int kReduceWarps = 16, kBatch = 16;

__global__ void __launch_bounds__(32 * kReduceWarps) k_qk_dw_reduce(const QkBwdParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    CRMSN_DEBUG_ENTER(p.dbg);
    __shared__ float sh[2][kReduceWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y;
    const int col = blockIdx.x * 32 + lane, n = p.share[which].blocks;
    const float *part = p.part + (which ? (int64_t)p.share[0].blocks * p.D : 0) + col;
    const int c0 = (int)((int64_t)warp * n / kReduceWarps), c1 = (int)((int64_t)(warp + 1) * n / kReduceWarps);
    float h = 0.f, l = 0.f;
    if (col < p.D) {
        for (int c = c0; c < c1; c += kBatch) {
            float v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                v[i] = c + i < c1 && dbg_global(part + (int64_t)(c + i) * p.D, 4, false)
                           ? __ldcg(part + (int64_t)(c + i) * p.D) : 0.f;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float s, e;
                two_sum(h, v[i], s, e);
                h = s;
                l = __fadd_rn(l, e);
            }
        }
    }
    sh[0][warp][lane] = h;
    sh[1][warp][lane] = l;
    __syncthreads();
    // Two columns a warp, 16 lanes each: lane i holds warp i's pair.
    const int j = 2 * warp + (lane >> 4);
    float a = sh[0][lane & 15][j], b = sh[1][lane & 15][j];
    for (int o = 8; o > 0; o >>= 1) {
        const float ch = __shfl_xor_sync(0xffffffffu, a, o), cl = __shfl_xor_sync(0xffffffffu, b, o);
        pair_acc(a, b, ch, cl);
    }
    const int out = blockIdx.x * 32 + j;
    if ((lane & 15) == 0 && out < p.D) st_f32(p.dw[which] + out, joined(a, b));
}

template <int N, bool WHOLE, bool NORM, bool PAIRS>
cudaError_t go(const QkBwdParams &p, dim3 grid, cudaStream_t s)
{
    constexpr size_t smem = NORM ? sizeof(BwdShared) : sizeof(BwdSharedPlain);
    static std::atomic<int> opted[kOptInDevices];
    if (cudaError_t e = opt_in_smem(k_qk_bwd<N, WHOLE, NORM, PAIRS>, smem, opted)) return e;
    return launch_pdl(k_qk_bwd<N, WHOLE, NORM, PAIRS>, grid, dim3(kThreads), smem, s, p);
}

template <int N, bool WHOLE>
cudaError_t go(const QkBwdParams &p, bool norm, dim3 grid, cudaStream_t s)
{
    if (norm) return p.pairs ? go<N, WHOLE, true, true>(p, grid, s) : go<N, WHOLE, true, false>(p, grid, s);
    return p.pairs ? go<N, WHOLE, false, true>(p, grid, s) : go<N, WHOLE, false, false>(p, grid, s);
}

}  // namespace

cudaError_t launch_qk_bwd(QkBwdParams p, bool norm, bool fast, int sms, cudaStream_t s)
{
    p.lanes = (p.D + 15) / 16;
    const int heads[2] = {p.g[0].H, p.g[1].H};
    // Runs of two steps (heads_fwd.cu): better up to D = 128 here (32 + 8
    // heads, T = 16384: 87.9 -> 80.0 us; D = 64, 16 + 16: 41.5 -> 38.0), worse
    // for wider heads (16 + 2 of 256 beside a gate, T = 8192: 55.1 -> 60.0).
    deal(p.share, heads, 2, p.T, p.cs_rows, fast ? 32 / p.lanes : 1, kWarps, sms * kQkBwdCtasPerSm, p.lanes <= 8);
    for (int i = 0; i < 2; ++i) {
        Share &sh = p.share[i];
        set_strides(sh.in, sh, heads[i], p.g[i].ld, p.g[i].hs);
        set_strides(sh.in2, sh, heads[i], p.x[i].ld, p.x[i].hs);
        set_strides(sh.out, sh, heads[i], p.dx[i].ld, p.dx[i].hs);
    }
    const dim3 grid((unsigned)(p.share[0].blocks + p.share[1].blocks)), block(kThreads);
    cudaError_t e;
    const bool whole = p.R == p.D;
    if (!fast) e = launch_pdl(k_qk_bwd_any, grid, block, 0, s, p, norm);
    else if (p.D == 64) e = whole ? go<4, true>(p, norm, grid, s) : go<4, false>(p, norm, grid, s);
    else if (p.D == 128) e = whole ? go<8, true>(p, norm, grid, s) : go<8, false>(p, norm, grid, s);
    else if (p.D == 256) e = whole ? go<16, true>(p, norm, grid, s) : go<16, false>(p, norm, grid, s);
    else e = go<0, false>(p, norm, grid, s);
    if (e != cudaSuccess || !norm) return e;
    return launch_pdl(k_qk_dw_reduce, dim3((unsigned)((p.D + 31) / 32), p.x[1].H > 0 ? 2 : 1),
                      dim3(32 * kReduceWarps), 0, s, p);
}

}  // namespace crmsn
