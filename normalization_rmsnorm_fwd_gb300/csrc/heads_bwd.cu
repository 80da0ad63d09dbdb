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
#include "heads.cuh"

namespace crmsn {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
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

template <bool NORM, bool PAIRS>
__global__ void __launch_bounds__(kThreads) k_qk_bwd(const QkBwdParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    CRMSN_DEBUG_ENTER(p.dbg);
    __shared__ float sums[NORM ? 2 * kWarps * CRMSN_MAX_HEAD_DIM : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lg = p.lg, l = lane & ((1 << lg) - 1), grp = lane >> lg, rpw = 32 >> lg;
    const Pieces pc = lane_pieces(l, p.R, p.D);
    const int which = (int)blockIdx.x < p.nblk[0] ? 0 : 1;
    const HeadView G = p.g[which], X = p.x[which], Y = p.dx[which];
    const int block = (int)blockIdx.x - (which ? p.nblk[0] : 0);
    const int chunks = p.chunks[which], steps = p.steps[which];
    F2 wa[4], wb[4];
    F2 ba[4], bb[4], ha[4], hb[4], la[4], lb[4];     // block sums, and the pairs they join
    int filled = 0;
    if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            wa[i] = wb[i] = ba[i] = bb[i] = ha[i] = hb[i] = la[i] = lb[i] = f2(0.f);
        if (pc.va) ld_weight8(wa, p.w[which], p.w32, p.bias, pc.a);
        if (pc.vb) ld_weight8(wb, p.w[which], p.w32, p.bias, pc.b);
    }
    auto fold = [&] {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s0, e0, s1, e1;
            two_sum(f2_lo(ha[i]), f2_lo(ba[i]), s0, e0);
            two_sum(f2_hi(ha[i]), f2_hi(ba[i]), s1, e1);
            ha[i] = f2(s0, s1);
            la[i] = f2_add(la[i], f2(e0, e1));
            two_sum(f2_lo(hb[i]), f2_lo(bb[i]), s0, e0);
            two_sum(f2_hi(hb[i]), f2_hi(bb[i]), s1, e1);
            hb[i] = f2(s0, s1);
            lb[i] = f2_add(lb[i], f2(e0, e1));
            ba[i] = bb[i] = f2(0.f);
        }
        filled = 0;
    };
    const uint32_t tasks = (uint32_t)p.T * (uint32_t)chunks;
    const uint32_t nwarps = (uint32_t)p.nblk[which] * kWarps;
    for (uint32_t task = (uint32_t)block * kWarps + warp; task < tasks; task += nwarps) {
        const int t = (int)(task / (uint32_t)chunks), chunk = (int)(task - (uint32_t)t * (uint32_t)chunks);
        Turn turn;
        if (pc.rot) ld_turn<PAIRS>(turn, p.cs + (int64_t)(t % p.cs_rows) * p.ldcs, l, p.R);
        const int h1 = min(X.H, (chunk + 1) * steps * rpw);
        for (int h0 = chunk * steps * rpw; h0 < h1; h0 += rpw) {
            const int h = h0 + grp;
            const bool on = h < h1;
            BVec<8> xa{}, xb{}, ga{}, gb{};
            if (on) {
                const uint16_t *g = G.p + (int64_t)t * G.ld + (int64_t)h * G.hs;
                if (pc.va) ga = ld_stream<8>(g + pc.a);
                if (pc.vb) gb = ld_stream<8>(g + pc.b);
                if constexpr (NORM) {
                    const uint16_t *x = X.p + (int64_t)t * X.ld + (int64_t)h * X.hs;
                    if (pc.va) xa = ld_stream<8>(x + pc.a);
                    if (pc.vb) xb = ld_stream<8>(x + pc.b);
                }
            }
            F2 a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = f2_bf16(ga.w[i]);
                b[i] = f2_bf16(gb.w[i]);
            }
            if (pc.rot) rotate<PAIRS, true>(a, b, turn);
            if constexpr (NORM) {
                float s0 = 0.f, s1 = 0.f;
                F2 m2 = f2(0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sq_acc_bf16x2(xa.w[i], s0, s1);
                    sq_acc_bf16x2(xb.w[i], s0, s1);
                    m2 = f2_fma(f2_mul(a[i], wa[i]), f2_bf16(xa.w[i]), m2);
                    m2 = f2_fma(f2_mul(b[i], wb[i]), f2_bf16(xb.w[i]), m2);
                }
                const float ss = row_lanes_sum(s0 + s1, lg);
                const float m = row_lanes_sum(f2_lo(m2) + f2_hi(m2), lg);
                const float rstd = __frsqrt_rn(__fadd_rn(__fmul_rn(ss, p.inv_d), p.eps));
                const float along = __fmul_rn(__fmul_rn(m, p.inv_d), rstd);
                const F2 r2 = f2(on ? rstd : 0.f), n2 = f2(-along);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 ya = f2_mul(f2_bf16(xa.w[i]), r2), yb = f2_mul(f2_bf16(xb.w[i]), r2);
                    const F2 ua = a[i], ub = b[i];
                    a[i] = f2_mul(r2, f2_fma(ya, n2, f2_mul(ua, wa[i])));
                    b[i] = f2_mul(r2, f2_fma(yb, n2, f2_mul(ub, wb[i])));
                    ba[i] = f2_fma(ua, ya, ba[i]);
                    bb[i] = f2_fma(ub, yb, bb[i]);
                }
                if (++filled == kFold) fold();
            }
            uint16_t *y = const_cast<uint16_t *>(Y.p) + (int64_t)t * Y.ld + (int64_t)h * Y.hs;
            BVec<8> v;
            if (on && pc.va) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v.w[i] = bf16_f2(a[i]);
                st_stream<8>(y + pc.a, v);
            }
            if (on && pc.vb) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v.w[i] = bf16_f2(b[i]);
                st_stream<8>(y + pc.b, v);
            }
        }
    }
    if constexpr (NORM) {
        fold();
        // The row groups of the warp hold the same columns.
        float *hi = sums + warp * p.D, *lo = sums + (kWarps + warp) * p.D;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float h0 = i & 1 ? f2_hi(ha[i / 2]) : f2_lo(ha[i / 2]), l0 = i & 1 ? f2_hi(la[i / 2]) : f2_lo(la[i / 2]);
            float h1 = i & 1 ? f2_hi(hb[i / 2]) : f2_lo(hb[i / 2]), l1 = i & 1 ? f2_hi(lb[i / 2]) : f2_lo(lb[i / 2]);
            for (int o = 1 << lg; o < 32; o <<= 1) {
                const float ch = __shfl_xor_sync(0xffffffffu, h0, o), cl = __shfl_xor_sync(0xffffffffu, l0, o);
                const float dh = __shfl_xor_sync(0xffffffffu, h1, o), dl = __shfl_xor_sync(0xffffffffu, l1, o);
                pair_acc(h0, l0, ch, cl);
                pair_acc(h1, l1, dh, dl);
            }
            if (grp == 0 && pc.va) {
                hi[pc.a + i] = h0;
                lo[pc.a + i] = l0;
            }
            if (grp == 0 && pc.vb) {
                hi[pc.b + i] = h1;
                lo[pc.b + i] = l1;
            }
        }
        store_partial(sums, sums + kWarps * p.D, p.D, p.part);
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
    const int which = (int)blockIdx.x < p.nblk[0] ? 0 : 1;
    const HeadView G = p.g[which], X = p.x[which], Y = p.dx[which];
    float h[kUnits][2], lo[kUnits][2];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) h[k][0] = h[k][1] = lo[k][0] = lo[k][1] = 0.f;
    const int64_t rows = (int64_t)p.T * X.H, nwarps = (int64_t)p.nblk[which] * kWarps;
    const int block = (int)blockIdx.x - (which ? p.nblk[0] : 0);
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
            rstd = __frsqrt_rn(__fadd_rn(__fmul_rn(row_lanes_sum(ss, 5), p.inv_d), p.eps));
            along = __fmul_rn(__fmul_rn(row_lanes_sum(m, 5), p.inv_d), rstd);
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
    const int col = blockIdx.x * 32 + lane, n = p.nblk[which];
    const float *part = p.part + (which ? (int64_t)p.nblk[0] * p.D : 0) + col;
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

}  // namespace

cudaError_t launch_qk_bwd(QkBwdParams p, bool norm, bool fast, int sms, cudaStream_t s)
{
    p.lg = 0;
    while ((16 << p.lg) < p.D) ++p.lg;
    const int rpw = fast ? 32 >> p.lg : 1, all = p.x[0].H + p.x[1].H;
    const int most = sms * kQkBwdCtasPerSm;
    for (int i = 0; i < 2; ++i) {
        const int H = p.x[i].H;
        p.nblk[i] = 0;
        p.chunks[i] = p.steps[i] = 1;
        if (H == 0) continue;
        // This tensor's share of the resident CTAs, and a token's heads split
        // over warps while they would leave some of them without work.
        int64_t share = i == 0 ? most : most - p.nblk[0];
        if (i == 0 && p.x[1].H > 0) {
            share = (int64_t)most * H / all;
            if (share < 1) share = 1;
            if (share > most - 1) share = most - 1;
        }
        const int total = (H + rpw - 1) / rpw;
        int64_t chunks = (share * kWarps + p.T - 1) / p.T;
        if (chunks > total) chunks = total;
        p.steps[i] = (int)((total + chunks - 1) / chunks);
        p.chunks[i] = (total + p.steps[i] - 1) / p.steps[i];
        const int64_t tasks = fast ? (int64_t)p.T * p.chunks[i] : (int64_t)p.T * H;
        const int64_t blocks = (tasks + kWarps - 1) / kWarps;
        p.nblk[i] = (int)(blocks < share ? blocks : share);
    }
    const dim3 grid((unsigned)(p.nblk[0] + p.nblk[1])), block(kThreads);
    cudaError_t e;
    if (!fast) e = launch_pdl(k_qk_bwd_any, grid, block, 0, s, p, norm);
    else if (norm) e = p.pairs ? launch_pdl(k_qk_bwd<true, true>, grid, block, 0, s, p)
                               : launch_pdl(k_qk_bwd<true, false>, grid, block, 0, s, p);
    else e = p.pairs ? launch_pdl(k_qk_bwd<false, true>, grid, block, 0, s, p)
                     : launch_pdl(k_qk_bwd<false, false>, grid, block, 0, s, p);
    if (e != cudaSuccess || !norm) return e;
    return launch_pdl(k_qk_dw_reduce, dim3((unsigned)((p.D + 31) / 32), p.x[1].H > 0 ? 2 : 1),
                      dim3(32 * kReduceWarps), 0, s, p);
}

}  // namespace crmsn
