// heads_fwd.cu -- per-head RMSNorm with the position rotation of queries and
// keys in one pass, and the same pass with the keys and the values written to
// a paged cache.
//
//   n = x rstd w_eff (n = x without weights), rstd = 1 / sqrt(mean x^2 + eps)
//   y_a = n_a c - n_b s, y_b = n_b c + n_a s     on the rotated pairs
//
// everything in FP32, one rounding at the end.
#include "heads.cuh"

namespace crmsn {

namespace {

constexpr int kThreads = 128;

// Where a token's row of the cache begins (elements); false: not written.
__device__ __forceinline__ bool cache_slot(const QkParams &p, int t, uint32_t &page, uint32_t &row)
{
    const int64_t s = ld_index(p.slots, p.slot64, t);
    if (s < 0 || s >= p.num_slots) return false;
    page = (uint32_t)((uint64_t)s / (uint32_t)p.page_size);
    row = (uint32_t)((uint64_t)s - (uint64_t)page * (uint32_t)p.page_size);
    return true;
}

// 8 values to a cache of BF16 or, divided by the scale, FP8.
__device__ __forceinline__ void st_cache8(void *base, int64_t off, int kind, const F2 (&y)[4], float inv)
{
    if (kind == CRMSN_CACHE_BF16) {
        BVec<8> v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[i] = bf16_f2(y[i]);
        st_stream<8>(static_cast<uint16_t *>(base) + off, v);
        return;
    }
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __fmul_rn(f2_lo(y[i]), inv), hi = __fmul_rn(f2_hi(y[i]), inv);
        c[i] = kind == CRMSN_CACHE_E4M3 ? pack_fp8<0>(lo, hi) : pack_fp8<1>(lo, hi);
    }
    st_fp8<8>(static_cast<uint8_t *>(base) + off, c);
}

// The 16-byte form.  A warp takes a task: up to `steps` groups of 32 >> lg
// rows (heads) of one token, whose cosines and sines stay in registers.
template <bool NORM, bool PAIRS, bool APPEND>
__global__ void __launch_bounds__(kThreads) k_qk_fwd(const QkParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    CRMSN_DEBUG_ENTER(p.dbg);
    const int lane = threadIdx.x & 31, lg = p.lg, l = lane & ((1 << lg) - 1), grp = lane >> lg, rpw = 32 >> lg;
    const Pieces pc = lane_pieces(l, p.R, p.D);
    const int Hq = p.in[0].H, Hk = p.in[1].H;
    float inv[2] = {1.f, 1.f};
    if (APPEND && p.kind != CRMSN_CACHE_BF16) {
        inv[0] = __frcp_rn(ld_f32_ro(p.scale[0]));
        inv[1] = __frcp_rn(ld_f32_ro(p.scale[1]));
    }
    F2 wa[4], wb[4];
    int held = -1;                                   // the tensor whose weight is in registers
    const uint32_t tasks = (uint32_t)p.T * (uint32_t)p.chunks;
    const uint32_t nwarps = gridDim.x * (kThreads / 32);
    for (uint32_t task = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); task < tasks; task += nwarps) {
        const int t = (int)(task / (uint32_t)p.chunks), chunk = (int)(task - (uint32_t)t * (uint32_t)p.chunks);
        Turn turn;
        if (pc.rot) ld_turn<PAIRS>(turn, p.cs + (int64_t)(t % p.cs_rows) * p.ldcs, l, p.R);
        uint32_t page = 0, row = 0;
        const bool kept = APPEND ? cache_slot(p, t, page, row) : true;
        const int h1 = min(p.heads, (chunk + 1) * p.steps * rpw);
        for (int h0 = chunk * p.steps * rpw; h0 < h1; h0 += rpw) {
            const int flat = h0 + grp;
            const int which = flat < Hq ? 0 : flat < Hq + Hk ? 1 : 2;
            const int h = flat - (which > 0 ? Hq : 0) - (which > 1 ? Hk : 0);
            const bool on = flat < h1 && (which == 0 || kept);
            BVec<8> xa{}, xb{};
            if (on) {
                const uint16_t *x = p.in[which].p + (int64_t)t * p.in[which].ld + (int64_t)h * p.in[which].hs;
                if (pc.va) xa = ld_stream<8>(x + pc.a);
                if (pc.vb) xb = ld_stream<8>(x + pc.b);
            }
            F2 a[4], b[4];
            if constexpr (NORM) {
                if (on && which != held && which < 2) {
                    held = which;
                    if (pc.va) ld_weight8(wa, p.w[which], p.w32, p.bias, pc.a);
                    if (pc.vb) ld_weight8(wb, p.w[which], p.w32, p.bias, pc.b);
                }
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sq_acc_bf16x2(xa.w[i], s0, s1);
                    sq_acc_bf16x2(xb.w[i], s0, s1);
                }
                const float ss = row_lanes_sum(s0 + s1, lg);
                const float rstd = __frsqrt_rn(__fadd_rn(__fmul_rn(ss, p.inv_d), p.eps));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = f2_mul(f2_mul(f2_bf16(xa.w[i]), f2(rstd)), wa[i]);
                    b[i] = f2_mul(f2_mul(f2_bf16(xb.w[i]), f2(rstd)), wb[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = f2_bf16(xa.w[i]);
                    b[i] = f2_bf16(xb.w[i]);
                }
            }
            if (pc.rot) rotate<PAIRS, false>(a, b, turn);
            if (APPEND && which == 2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = f2_bf16(xa.w[i]);
                    b[i] = f2_bf16(xb.w[i]);
                }
            }
            if (on && APPEND && which > 0) {
                const CacheView &cv = p.cache[which - 1];
                const int64_t off = (int64_t)page * cv.ps + (int64_t)row * cv.ss + (int64_t)h * cv.hs;
                if (pc.va) st_cache8(cv.p, off + pc.a, p.kind, a, inv[which - 1]);
                if (pc.vb) st_cache8(cv.p, off + pc.b, p.kind, b, inv[which - 1]);
            } else if (on) {
                uint16_t *y = const_cast<uint16_t *>(p.out[which].p) + (int64_t)t * p.out[which].ld +
                              (int64_t)h * p.out[which].hs;
                BVec<8> v;
                if (pc.va) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v.w[i] = bf16_f2(a[i]);
                    st_stream<8>(y + pc.a, v);
                }
                if (pc.vb) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v.w[i] = bf16_f2(b[i]);
                    st_stream<8>(y + pc.b, v);
                }
            }
        }
    }
}

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
        uint32_t page = 0, row = 0;
        if (append && which > 0 && !cache_slot(p, t, page, row)) continue;
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
        if (norm) rstd = __frsqrt_rn(__fadd_rn(__fmul_rn(row_lanes_sum(ss, 5), p.inv_d), p.eps));
        const float *cs = p.cs + (int64_t)(t % p.cs_rows) * p.ldcs;
        float inv = 1.f;
        if (append && which > 0 && p.kind != CRMSN_CACHE_BF16) inv = __frcp_rn(ld_f32_ro(p.scale[which - 1]));
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
                const int64_t off = (int64_t)page * cv.ps + (int64_t)row * cv.ss + (int64_t)h * cv.hs;
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

template <bool NORM, bool APPEND>
cudaError_t go(const QkParams &p, dim3 grid, cudaStream_t s)
{
    return p.pairs ? launch_pdl(k_qk_fwd<NORM, true, APPEND>, grid, dim3(kThreads), 0, s, p)
                   : launch_pdl(k_qk_fwd<NORM, false, APPEND>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_qk_fwd(QkParams p, bool norm, bool append, bool fast, int sms, cudaStream_t s)
{
    constexpr int kWarps = kThreads / 32, kResident = 6;
    const int64_t room = (int64_t)sms * kResident * kWarps;      // warps of one resident grid
    if (!fast) {
        const int64_t rows = (int64_t)p.T * p.heads;
        const int64_t blocks = (rows + kWarps - 1) / kWarps, most = room / kWarps * 4;
        return launch_pdl(k_qk_fwd_any, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, s, p, norm,
                          append);
    }
    p.lg = 0;
    while ((16 << p.lg) < p.D) ++p.lg;
    const int rpw = 32 >> p.lg, total = (p.heads + rpw - 1) / rpw;
    // Few tokens: split a token's heads over warps until the grid is full.
    int64_t chunks = (room + p.T - 1) / p.T;
    if (chunks > total) chunks = total;
    p.steps = (int)((total + chunks - 1) / chunks);
    p.chunks = (total + p.steps - 1) / p.steps;
    const int64_t tasks = (int64_t)p.T * p.chunks, blocks = (tasks + kWarps - 1) / kWarps;
    const dim3 grid((unsigned)(blocks < sms * kResident ? blocks : sms * kResident));
    if (append) return norm ? go<true, true>(p, grid, s) : go<false, true>(p, grid, s);
    return norm ? go<true, false>(p, grid, s) : go<false, false>(p, grid, s);
}

}  // namespace crmsn
