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
// block covers 8 columns (a 32-byte sector of every row) of dwq (blockIdx.y 0)
// or dwk; thread r * 8 + c adds rows r, r + 64, ... of column c, its loads in
// flight together; lanes, then warps meet in fixed butterflies.  (32 columns a
// block, a warp to each contiguous range of rows: 11.6 instead of 10.5 us for
// the whole backward at T = 1024 with 32 + 8 heads of 128.)
constexpr int kReduceThreads = 512, kReduceRows = kReduceThreads / 8, kBatch = 10;

__device__ __forceinline__ void pair_xor(float &h, float &l, int o)
{
    const float ch = __shfl_xor_sync(0xffffffffu, h, o), cl = __shfl_xor_sync(0xffffffffu, l, o);
    pair_acc(h, l, ch, cl);
}

__global__ void __launch_bounds__(kReduceThreads) k_qk_dw_reduce(const QkBwdParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    CRMSN_DEBUG_ENTER(p.dbg);
    __shared__ float sh[2][8][kReduceThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y;
    const int col = blockIdx.x * 8 + (lane & 7), n = p.share[which].blocks;
    const float *part = p.part + (which ? (int64_t)p.share[0].blocks * p.D : 0) + col;
    float h = 0.f, l = 0.f;
    for (int r = threadIdx.x >> 3; r < n; r += kBatch * kReduceRows) {
        float v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int row = r + i * kReduceRows;
            v[i] = col < p.D && row < n && dbg_global(part + (int64_t)row * p.D, 4, false)
                       ? __ldcg(part + (int64_t)row * p.D) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float s, e;
            two_sum(h, v[i], s, e);
            h = s;
            l = __fadd_rn(l, e);
        }
    }
    pair_xor(h, l, 8);
    pair_xor(h, l, 16);
    if (lane < 8) {
        sh[0][lane][warp] = h;
        sh[1][lane][warp] = l;
    }
    __syncthreads();
    // Column c of the block: lanes 16 c .. 16 c + 15 hold its warps' pairs.
    if (warp >= 4) return;
    const int c = threadIdx.x >> 4, w = threadIdx.x & 15, out = blockIdx.x * 8 + c;
    h = sh[0][c][w];
    l = sh[1][c][w];
    for (int o = 8; o > 0; o >>= 1) pair_xor(h, l, o);
    if (w == 0 && out < p.D) st_f32(p.dw[which] + out, joined(h, l));
}

}  // namespace

cudaError_t launch_qk_bwd(QkBwdParams p, bool norm, int vec, int sms, cudaStream_t s)
{
    p.lanes = row_lanes(p.R, p.D);
    const int heads[2] = {p.g[0].H, p.g[1].H}, cost[2] = {1, 1};
    // Runs of two steps (heads.cu): better up to D = 128 here (32 + 8
    // heads, T = 16384: 87.9 -> 80.0 us; D = 64, 16 + 16: 41.5 -> 38.0), worse
    // for wider heads (16 + 2 of 256 beside a gate, T = 8192: 55.1 -> 60.0).
    deal(p.share, heads, cost, 2, p.T, p.cs_rows, vec > 0 ? 32 / p.lanes : 1, kBwdWarps, sms * kQkBwdCtasPerSm,
         p.lanes <= 8);
    for (int i = 0; i < 2; ++i) {
        Share &sh = p.share[i];
        set_strides(sh.in, sh, heads[i], p.g[i].ld, p.g[i].hs);
        set_strides(sh.in2, sh, heads[i], p.x[i].ld, p.x[i].hs);
        set_strides(sh.out, sh, heads[i], p.dx[i].ld, p.dx[i].hs);
    }
    p.l1 = split_sectors(p.R, p.D, p.g, 2) || (norm && split_sectors(p.R, p.D, p.x, 2));
    const dim3 grid((unsigned)(p.share[0].blocks + p.share[1].blocks));
    cudaError_t e = vec == 8 ? run_qk_bwd(p, norm, grid, s)
                  : vec > 0  ? run_qk_bwd_narrow(p, norm, vec, grid, s)
                             : launch_pdl(k_qk_bwd_any, grid, dim3(kBwdThreads), 0, s, p, norm);
    if (e != cudaSuccess || !norm) return e;
    return launch_pdl(k_qk_dw_reduce, dim3((unsigned)((p.D + 7) / 8), p.g[1].H > 0 ? 2 : 1), dim3(kReduceThreads), 0, s,
                      p);
}

cudaError_t run_qk_bwd(const QkBwdParams &p, bool norm, dim3 grid, cudaStream_t s)
{
    const bool whole = p.R == p.D;
    if (p.D == 64) return whole ? go_bwd<4, true, 8>(p, norm, grid, s) : go_bwd<4, false, 8>(p, norm, grid, s);
    if (p.D == 128) return whole ? go_bwd<8, true, 8>(p, norm, grid, s) : go_bwd<8, false, 8>(p, norm, grid, s);
    if (p.D == 256) return whole ? go_bwd<16, true, 8>(p, norm, grid, s) : go_bwd<16, false, 8>(p, norm, grid, s);
    if (p.D == 192) return whole ? go_bwd<12, true, 8>(p, norm, grid, s) : go_bwd<12, false, 8>(p, norm, grid, s);
    return go_bwd<0, false, 8>(p, norm, grid, s);
}

}  // namespace crmsn
