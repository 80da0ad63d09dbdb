// heads_bwd.cu -- the launch of the query / key backward: its 16-byte form, its
// element-wise form, and the sum of the partial dw rows.
#include "heads_bwd.cuh"

namespace crmsn {

namespace {

// The warps' pairs [kBwdWarps][D] (high and low parts) -> one partial row.
__device__ __forceinline__ void store_partial(const float *hi, const float *lo, int D, float *part)
{
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += kBwdThreads) {
        float h = 0.f, l = 0.f;
        for (int w = 0; w < kBwdWarps; ++w) pair_acc(h, l, hi[w * D + j], lo[w * D + j]);
        st_f32(part + (int64_t)blockIdx.x * D + j, joined(h, l));
    }
}

// The element-wise form: one warp per row.
__global__ void __launch_bounds__(kBwdThreads) k_qk_bwd_any(const QkBwdParams p, bool norm)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    CRMSN_DEBUG_ENTER(p.dbg);
    constexpr int kUnits = CRMSN_MAX_HEAD_DIM / 64;
    __shared__ float sums[2 * kBwdWarps * CRMSN_MAX_HEAD_DIM];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, units = p.D / 2;
    const int which = (int)blockIdx.x < p.share[0].blocks ? 0 : 1;
    const HeadView G = p.g[which], X = p.x[which], Y = p.dx[which];
    float h[kUnits][2], lo[kUnits][2];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) h[k][0] = h[k][1] = lo[k][0] = lo[k][1] = 0.f;
    const int64_t rows = (int64_t)p.T * X.H, nwarps = (int64_t)p.share[which].blocks * kBwdWarps;
    const int block = (int)blockIdx.x - (which ? p.share[0].blocks : 0);
    for (int64_t r = (int64_t)block * kBwdWarps + warp; r < rows; r += nwarps) {
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
            sums[(kBwdWarps + warp) * p.D + e[q]] = lo[k][q];
        }
    }
    store_partial(sums, sums + kBwdWarps * p.D, p.D, p.part);
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

}  // namespace

cudaError_t launch_qk_bwd(QkBwdParams p, bool norm, int vec, int sms, cudaStream_t s)
{
    p.lanes = row_lanes(p.R, p.D);
    const int heads[2] = {p.g[0].H, p.g[1].H};
    // Runs of two steps (heads_fwd.cu): better up to D = 128 here (32 + 8
    // heads, T = 16384: 87.9 -> 80.0 us; D = 64, 16 + 16: 41.5 -> 38.0), worse
    // for wider heads (16 + 2 of 256 beside a gate, T = 8192: 55.1 -> 60.0).
    deal(p.share, heads, 2, p.T, p.cs_rows, vec > 0 ? 32 / p.lanes : 1, kBwdWarps, sms * kQkBwdCtasPerSm, p.lanes <= 8);
    for (int i = 0; i < 2; ++i) {
        Share &sh = p.share[i];
        set_strides(sh.in, sh, heads[i], p.g[i].ld, p.g[i].hs);
        set_strides(sh.in2, sh, heads[i], p.x[i].ld, p.x[i].hs);
        set_strides(sh.out, sh, heads[i], p.dx[i].ld, p.dx[i].hs);
    }
    const dim3 grid((unsigned)(p.share[0].blocks + p.share[1].blocks));
    cudaError_t e = vec == 8 ? run_qk_bwd(p, norm, grid, s)
                  : vec > 0  ? run_qk_bwd_narrow(p, norm, vec, grid, s)
                             : launch_pdl(k_qk_bwd_any, grid, dim3(kBwdThreads), 0, s, p, norm);
    if (e != cudaSuccess || !norm) return e;
    return launch_pdl(k_qk_dw_reduce, dim3((unsigned)((p.D + 31) / 32), p.g[1].H > 0 ? 2 : 1),
                      dim3(32 * kReduceWarps), 0, s, p);
}

cudaError_t run_qk_bwd(const QkBwdParams &p, bool norm, dim3 grid, cudaStream_t s)
{
    const bool whole = p.R == p.D;
    if (p.D == 64) return whole ? go_bwd<4, true, 8>(p, norm, grid, s) : go_bwd<4, false, 8>(p, norm, grid, s);
    if (p.D == 128) return whole ? go_bwd<8, true, 8>(p, norm, grid, s) : go_bwd<8, false, 8>(p, norm, grid, s);
    if (p.D == 256) return whole ? go_bwd<16, true, 8>(p, norm, grid, s) : go_bwd<16, false, 8>(p, norm, grid, s);
    return go_bwd<0, false, 8>(p, norm, grid, s);
}

}  // namespace crmsn
