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

constexpr int kThreads = 128, kPerSm = 6, kStages = 2 * kRun;

// Where a token's row of the cache begins (elements); -1: not written.
__device__ __forceinline__ int64_t cache_row(const QkParams &p, const CacheView &c, int64_t t)
{
    const int64_t s = ld_index(p.slots, p.slot64, t);
    if (s < 0 || s >= p.num_slots) return -1;                // num_slots < 2^31
    const uint32_t page = (uint32_t)s / (uint32_t)p.page_size, row = (uint32_t)s - page * (uint32_t)p.page_size;
    return (int64_t)page * c.ps + (int64_t)row * c.ss;
}

// 8 values to a cache of BF16 or, divided by the scale, FP8.
__device__ __forceinline__ void st_cache8(void *base, int64_t off, int kind, const F2 (&y)[4], float inv)
{
    if (kind == CRMSN_CACHE_BF16) {
        st_f2x4(static_cast<uint16_t *>(base) + off, y);
        return;
    }
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const F2 z = f2_mul(y[i], f2(inv));
        c[i] = kind == CRMSN_CACHE_E4M3 ? pack_fp8<0>(f2_lo(z), f2_hi(z)) : pack_fp8<1>(f2_lo(z), f2_hi(z));
    }
    st_fp8<8>(static_cast<uint8_t *>(base) + off, c);
}

enum Role { TO_HEADS, KEY_TO_CACHE, VALUE_TO_CACHE };

using Ring = uint4[kStages][2][kThreads];

// One warp's rows of tensor `which`.
template <int N, bool WHOLE, bool NORM, bool PAIRS, int ROLE>
__device__ __forceinline__ void walk_rows(const QkParams &p, int which, int block, Ring &ring)
{
    constexpr bool kRotate = ROLE != VALUE_TO_CACHE, kNorm = NORM && kRotate;
    const Lanes<N> L(p.lanes);
    const Pieces pc = lane_pieces<N, WHOLE>(L.l, p.R, p.D);
    const int H = p.in[which].H, tid = threadIdx.x, delta = pc.b - pc.a, P = p.cs_rows;
    const Share &sh = p.share[which];
    const LaneRows mine(sh, H, block * (kThreads / 32) + (tid >> 5), L.grp, L.rows());
    if (mine.most == 0) return;
    int64_t t = mine.t;
    Walk<const uint16_t> in = {p.in[which].p + t * p.in[which].ld + mine.h * p.in[which].hs + pc.a, mine.h};
    int to_issue = mine.mine;
    auto issue = [&](int stage) {
        if (to_issue > 0) {
            if (pc.va) cp_async16(&ring[stage][0][tid], in.p);
            if (pc.vb) cp_async16(&ring[stage][1][tid], in.p + delta);
        }
        --to_issue;
        const int e = stage % kRun == kRun - 1;
        in.step(sh.in[e], sh.dh[e], H);
    };
    // A piece that the row has not stays zero.
    if (N == 0 && !(pc.va && pc.vb))
        for (int i = 0; i < kStages; ++i) ring[i][0][tid] = ring[i][1][tid] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kRun; ++i) issue(i);
    ring_commit();

    F2 wa[4], wb[4];
    if constexpr (kNorm) {
        if (pc.va) ld_weight8(wa, p.w[which], p.w32, p.bias, pc.a);
        if (pc.vb) ld_weight8(wb, p.w[which], p.w32, p.bias, pc.b);
    }
    // Where the rows go: a heads tensor, or a head's place in a cache row.
    const bool fp8 = ROLE != TO_HEADS && p.kind != CRMSN_CACHE_BF16;
    float inv = 1.f;
    if (fp8) inv = __frcp_rn(ld_f32_ro(p.scale[which - 1]));
    Walk<uint16_t> out = {nullptr, mine.h};
    int64_t head = 0, base = 0;
    if constexpr (ROLE == TO_HEADS)
        out.p = const_cast<uint16_t *>(p.out[which].p) + t * p.out[which].ld + mine.h * p.out[which].hs + pc.a;
    else
        head = mine.h * p.cache[which - 1].hs + pc.a;
    int tc = (int)(t % P);                           // row of cos_sin
    Turn turn;
    if (kRotate && pc.rot && mine.mine > 0) ld_turn<PAIRS>(turn, p.cs + (int64_t)tc * p.ldcs, L.l, p.R);
    if constexpr (ROLE != TO_HEADS)
        if (mine.mine > 0) base = cache_row(p, p.cache[which - 1], t);
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
            const BVec<8> xa = ld_slot(&ring[stage][0][tid]), xb = ld_slot(&ring[stage][1][tid]);
            F2 a[4], b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[k] = f2_bf16(xa.w[k]);
                b[k] = f2_bf16(xb.w[k]);
            }
            if constexpr (kNorm) {
                F2 ss = f2_mul(a[0], a[0]), s2 = f2_mul(b[0], b[0]);
#pragma unroll
                for (int k = 1; k < 4; ++k) {
                    ss = f2_fma(a[k], a[k], ss);
                    s2 = f2_fma(b[k], b[k], s2);
                }
                ss = f2_add(ss, s2);
                float sum[1] = {f2_lo(ss) + f2_hi(ss)};
                L.sum(sum);
                const F2 rstd = f2(__frsqrt_rn(__fmaf_rn(sum[0], p.inv_d, p.eps)));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a[k] = f2_mul(f2_mul(a[k], rstd), wa[k]);
                    b[k] = f2_mul(f2_mul(b[k], rstd), wb[k]);
                }
            }
            if (kRotate && pc.rot) rotate<PAIRS, false>(a, b, turn);
            const bool on = i < mine.mine;
            if constexpr (ROLE == TO_HEADS) {
                if (on && pc.va) st_f2x4(out.p, a);
                if (on && pc.vb) st_f2x4(out.p + delta, b);
            } else if (on && base >= 0) {
                void *c = p.cache[which - 1].p;
                if (pc.va) st_cache8(c, base + head, p.kind, a, inv);
                if (pc.vb) st_cache8(c, base + head + delta, p.kind, b, inv);
            }
            // The lane's next row; what a new token needs is asked for now.
            const int e = stage % kRun == kRun - 1;
            bool over;
            if constexpr (ROLE == TO_HEADS) {
                over = out.step(sh.out[e], sh.dh[e], H);
            } else {
                head += sh.out[e].step;
                out.h += sh.dh[e];
                over = out.h >= H;
                if (over) {
                    out.h -= H;
                    head += sh.out[e].wrap;
                }
                t += sh.dt[e] + over;
            }
            tc += sh.dtc[e] + over;
            if (tc >= P) tc -= P;
            if ((over || sh.dt[e] > 0) && i + 1 < mine.mine) {
                if (kRotate && pc.rot) ld_turn<PAIRS>(turn, p.cs + (int64_t)tc * p.ldcs, L.l, p.R);
                if constexpr (ROLE != TO_HEADS) base = cache_row(p, p.cache[which - 1], t);
            }
        }
    }
}

template <int N, bool WHOLE, bool NORM, bool PAIRS, bool APPEND>
__global__ void __launch_bounds__(kThreads, kPerSm) k_qk_fwd(const QkParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    CRMSN_DEBUG_ENTER(p.dbg);
    Ring &ring = *reinterpret_cast<Ring *>(heads_smem);
    int block = blockIdx.x, which = 0;
    while (which < (APPEND ? 2 : 1) && block >= p.share[which].blocks) block -= p.share[which++].blocks;
    if (!APPEND || which == 0) walk_rows<N, WHOLE, NORM, PAIRS, TO_HEADS>(p, which, block, ring);
    else if (which == 1) walk_rows<N, WHOLE, NORM, PAIRS, KEY_TO_CACHE>(p, 1, block, ring);
    else walk_rows<N, WHOLE, NORM, PAIRS, VALUE_TO_CACHE>(p, 2, block, ring);
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
        int64_t base = 0;
        if (append && which > 0) base = cache_row(p, p.cache[which - 1], t);
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

template <int N, bool WHOLE, bool APPEND>
cudaError_t go(const QkParams &p, bool norm, dim3 grid, cudaStream_t s)
{
    const dim3 b(kThreads);
    if (norm) return p.pairs ? launch_pdl(k_qk_fwd<N, WHOLE, true, true, APPEND>, grid, b, sizeof(Ring), s, p)
                             : launch_pdl(k_qk_fwd<N, WHOLE, true, false, APPEND>, grid, b, sizeof(Ring), s, p);
    return p.pairs ? launch_pdl(k_qk_fwd<N, WHOLE, false, true, APPEND>, grid, b, sizeof(Ring), s, p)
                   : launch_pdl(k_qk_fwd<N, WHOLE, false, false, APPEND>, grid, b, sizeof(Ring), s, p);
}

template <bool APPEND>
cudaError_t go(const QkParams &p, bool norm, dim3 grid, cudaStream_t s)
{
    const bool whole = p.R == p.D;
    if (p.D == 64) return whole ? go<4, true, APPEND>(p, norm, grid, s) : go<4, false, APPEND>(p, norm, grid, s);
    if (p.D == 128) return whole ? go<8, true, APPEND>(p, norm, grid, s) : go<8, false, APPEND>(p, norm, grid, s);
    if (p.D == 256) return whole ? go<16, true, APPEND>(p, norm, grid, s) : go<16, false, APPEND>(p, norm, grid, s);
    return go<0, false, APPEND>(p, norm, grid, s);
}

}  // namespace

void deal(Share *s, const int *heads, int n, int64_t T, int cs_rows, int rows_per_step, int warps, int ctas,
          bool runs)
{
    int64_t all = 0, left = ctas;
    for (int i = 0; i < n; ++i) all += heads[i];
    for (int i = 0; i < n; ++i) {
        s[i] = Share{};
        if (heads[i] == 0) continue;
        // Every CTA of the launch has the same number of rows, up to rounding.
        int64_t share = all == heads[i] ? left : (left * heads[i] + all / 2) / all;
        if (share < 1) share = 1;
        if (share > left - 2 && all != heads[i]) share = left - 2;      // at least one for each tensor to come
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
        all -= heads[i];
    }
}

void set_strides(Stride (&d)[2], const Share &s, int H, int64_t ld, int64_t hs)
{
    for (int e = 0; e < 2; ++e) d[e] = {s.dt[e] * ld + s.dh[e] * hs, ld - H * hs};
}

cudaError_t launch_qk_fwd(QkParams p, bool norm, bool append, bool fast, int sms, cudaStream_t s)
{
    constexpr int kWarps = kThreads / 32;
    if (!fast) {
        const int64_t rows = (int64_t)p.T * p.heads;
        const int64_t blocks = (rows + kWarps - 1) / kWarps, most = (int64_t)sms * 4 * kPerSm;
        return launch_pdl(k_qk_fwd_any, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, s, p, norm,
                          append);
    }
    p.lanes = (p.D + 15) / 16;
    const int heads[3] = {p.in[0].H, p.in[1].H, p.in[2].H}, n = append ? 3 : 2;
    // Runs of two steps load a token's cosines and sines half as often, which
    // narrow heads need (D = 64, T = 16384, 16 + 16 heads: 24.4 -> 21.2 us;
    // D = 96: 40.2 -> 37.3); single steps keep the memory that all warps
    // touch at a time closest together, which is worth more from D = 128 on
    // (32 + 8 heads: 60.1 -> 55.4 us; D = 256: 57.3 -> 49.5).
    deal(p.share, heads, n, p.T, p.cs_rows, 32 / p.lanes, kWarps, sms * kPerSm, p.lanes < 8);
    int blocks = 0;
    for (int i = 0; i < n; ++i) {
        Share &sh = p.share[i];
        set_strides(sh.in, sh, heads[i], p.in[i].ld, p.in[i].hs);
        if (append && i > 0) set_strides(sh.out, sh, heads[i], 0, p.cache[i - 1].hs);
        else set_strides(sh.out, sh, heads[i], p.out[i].ld, p.out[i].hs);
        blocks += sh.blocks;
    }
    const dim3 grid((unsigned)blocks);
    return append ? go<true>(p, norm, grid, s) : go<false>(p, norm, grid, s);
}

}  // namespace crmsn
