// heads.cu -- how the query / key kernels share out their rows, the launch of
// the forward and the append, and their element-wise form.
#include "heads_fwd.cuh"

namespace crmsn {

namespace {

constexpr int kWarps = kThreads / 32;

// One value to the cache.
__device__ __forceinline__ void st_cache1(void *base, int64_t off, int kind, float y, float inv)
{
    if (kind == CRMSN_CACHE_BF16) {
        st_bf16_1(static_cast<uint16_t *>(base) + off, y);
        return;
    }
    y = __fmul_rn(y, inv);
    st_u8_1(static_cast<uint8_t *>(base) + off, kind == CRMSN_CACHE_E4M3 ? pack_fp8<0>(y, 0.f) : pack_fp8<1>(y, 0.f));
}

// The element-wise form: one warp per row, any even D and R, any alignment.
__global__ void __launch_bounds__(kThreads) k_qk_fwd_any(const QkParams p, bool norm, bool append)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    CRMSN_DEBUG_ENTER(p.dbg);
    constexpr int kUnits = CRMSN_MAX_HEAD_DIM / 64;
    const int lane = threadIdx.x & 31;
    const int Hq = p.in[0].H, Hk = p.in[1].H, units = p.D / 2;
    const int64_t rows = (int64_t)p.T * p.heads, nwarps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows; r += nwarps) {
        const int t = (int)(r / p.heads), flat = (int)(r - (int64_t)t * p.heads);
        const int which = flat < Hq ? 0 : flat < Hq + Hk ? 1 : 2;
        const int h = flat - (which > 0 ? Hq : 0) - (which > 1 ? Hk : 0);
        int64_t base = 0;
        if (append && which > 0) base = cache_row(p, p.cache[which - 1], ld_index(p.slots, p.slot64, t));
        if (base < 0) continue;
        const uint16_t *x = p.in[which].p + (int64_t)t * p.in[which].ld + (int64_t)h * p.in[which].hs;
        float v[kUnits][2], ss = 0.f;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int u = lane + 32 * k;
            v[k][0] = v[k][1] = 0.f;
            if (u < units) {
                int i, j;
                unit_elems(u, p.R, p.pairs, i, j);
                v[k][0] = ld_bf16_1(x + i);
                v[k][1] = ld_bf16_1(x + j);
                ss = __fmaf_rn(v[k][0], v[k][0], ss);
                ss = __fmaf_rn(v[k][1], v[k][1], ss);
            }
        }
        float rstd = 1.f;
        if (norm) rstd = __frsqrt_rn(__fadd_rn(__fmul_rn(warp_sum(ss), p.inv_d), p.eps));
        const float *cs = p.cs + (int64_t)(t % p.cs_rows) * p.ldcs;
        float inv = 1.f;
        if (append && which > 0 && p.kind != CRMSN_CACHE_BF16) inv = scale_reciprocal(p.scale[which - 1]);
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int u = lane + 32 * k;
            if (u >= units) continue;
            int i, j;
            unit_elems(u, p.R, p.pairs, i, j);
            float a = v[k][0], b = v[k][1];
            if (which < 2) {
                if (norm) {
                    a = __fmul_rn(__fmul_rn(a, rstd), weight_1(p.w[which], p.w32, p.bias, i));
                    b = __fmul_rn(__fmul_rn(b, rstd), weight_1(p.w[which], p.w32, p.bias, j));
                }
                if (u < p.R / 2) {
                    const float c = ld_f32_ro(cs + u), s = ld_f32_ro(cs + p.R / 2 + u);
                    const float y = __fmaf_rn(a, c, -__fmul_rn(b, s));
                    b = __fmaf_rn(b, c, __fmul_rn(a, s));
                    a = y;
                }
            }
            if (append && which > 0) {
                const CacheView &cv = p.cache[which - 1];
                const int64_t off = base + (int64_t)h * cv.hs;
                st_cache1(cv.p, off + i, p.kind, a, inv);
                st_cache1(cv.p, off + j, p.kind, b, inv);
            } else {
                uint16_t *y = const_cast<uint16_t *>(p.out[which].p) + (int64_t)t * p.out[which].ld +
                              (int64_t)h * p.out[which].hs;
                st_bf16_1(y + i, a);
                st_bf16_1(y + j, b);
            }
        }
    }
}

}  // namespace

void deal(Share *s, const int *heads, const int *cost, int n, int64_t T, int cs_rows, int rows_per_step, int warps,
          int ctas, bool runs)
{
    int64_t all = 0, left = ctas;
    for (int i = 0; i < n; ++i) all += (int64_t)heads[i] * cost[i];
    for (int i = 0; i < n; ++i) {
        s[i] = Share{};
        if (heads[i] == 0) continue;
        // Every CTA of the launch has the same work, up to rounding.
        const int64_t part = (int64_t)heads[i] * cost[i];
        int64_t share = all == part ? left : (left * part + all / 2) / all;
        if (share < 1) share = 1;
        if (share > left - 2 && all != part) share = left - 2;      // at least one for each tensor to come
        s[i].rows = T * heads[i];
        const int64_t steps = (s[i].rows + rows_per_step - 1) / rows_per_step;
        const int64_t need = (steps + warps - 1) / warps;
        s[i].blocks = (int)(need < share ? need : share);
        const int64_t w = (int64_t)s[i].blocks * warps;
        s[i].run = runs && steps >= 4 * w ? kRun : 1;
        s[i].inc = w * s[i].run * rows_per_step;
        // A run's last step is its kRun-th, or each.
        const int64_t on[2] = {s[i].run > 1 ? rows_per_step : s[i].inc, s[i].inc - (s[i].run - 1) * rows_per_step};
        for (int e = 0; e < 2; ++e) {
            s[i].dt[e] = (int)(on[e] / heads[i]);
            s[i].dtc[e] = s[i].dt[e] % cs_rows;
            s[i].dh[e] = (int)(on[e] % heads[i]);
        }
        left -= share;
        all -= part;
    }
}

void set_strides(Stride (&d)[2], const Share &s, int H, int64_t ld, int64_t hs)
{
    for (int e = 0; e < 2; ++e) d[e] = {s.dt[e] * ld + s.dh[e] * hs, ld - H * hs};
}

bool split_sectors(int R, int D, const HeadView *v, int n)
{
    bool split = D % 16 || R / 2 % 16 || (D - R + 15) / 16 % 2;
    for (int i = 0; i < n; ++i)
        if (v[i].H > 0) split = split || v[i].ld % 16 || v[i].hs % 16 || (uintptr_t)v[i].p % 32;
    return split;
}

cudaError_t launch_qk_fwd(QkParams p, bool norm, bool append, int vec, int sms, cudaStream_t s)
{
    if (vec == 0) {
        const int64_t rows = (int64_t)p.T * p.heads;
        const int64_t blocks = (rows + kWarps - 1) / kWarps, most = (int64_t)sms * 24;
        return launch_pdl(k_qk_fwd_any, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, s, p, norm,
                          append);
    }
    p.lanes = row_lanes(p.R, p.D);
    // What a row of q, k and v costs: a key's row also finds its page, a
    // value's is only copied.  (With equal costs the CTAs of the keys end last:
    // a prompt of 8192 tokens, 32 + 8 heads of 128, 36.4 -> 33.7 us; 32 + 4
    // heads of 96, E4M3, T = 16000 53.5 -> 45.6.)
    const int cost[3] = {4, append ? 5 : 4, 3};
    const int heads[3] = {p.in[0].H, p.in[1].H, p.in[2].H}, n = append ? 3 : 2;
    // Runs of two steps load a token's cosines and sines half as often, which
    // narrow heads need (D = 64, T = 16384, 16 + 16 heads: 24.4 -> 21.2 us;
    // D = 96: 40.2 -> 37.3); single steps keep the memory that all warps
    // touch at a time closest together, which is worth more from D = 128 on
    // (32 + 8 heads: 60.1 -> 55.4 us; D = 256: 57.3 -> 49.5).
    deal(p.share, heads, cost, n, p.T, p.cs_rows, 32 / p.lanes, kWarps,
         sms * qk_fwd_ctas_per_sm(append, norm, !own_code(vec, p.D)), p.lanes < 8);
    int blocks = 0;
    for (int i = 0; i < n; ++i) {
        Share &sh = p.share[i];
        set_strides(sh.in, sh, heads[i], p.in[i].ld, p.in[i].hs);
        if (append && i > 0) set_strides(sh.out, sh, heads[i], 0, p.cache[i - 1].hs);
        else set_strides(sh.out, sh, heads[i], p.out[i].ld, p.out[i].hs);
        blocks += sh.blocks;
    }
    p.l1 = split_sectors(p.R, p.D, p.in, n);
    const dim3 grid((unsigned)blocks);
    if (vec < 8) return run_qk_narrow(p, norm, append, vec, grid, s);
    return append ? run_qk_append(p, norm, grid, s) : run_qk_fwd(p, norm, grid, s);
}

}  // namespace crmsn
