// heads_fwd.cuh -- per-head RMSNorm with the position rotation of queries and
// keys in one pass, and the same pass with the keys and the values written to
// a paged cache.
//
//   n = x rstd w_eff (n = x without weights), rstd = 1 / sqrt(mean x^2 + eps)
//   y_a = n_a c - n_b s, y_b = n_b c + n_a s     on the rotated pairs
//
// everything in FP32, one rounding at the end.  Bound by HBM where the sizes
// are large: 180 instructions for a step of 1 KB in and 1 KB out.
#pragma once

#include <cfloat>

#include "heads.cuh"

namespace crmsn {

namespace {

constexpr int kThreads = 128, kStages = 2 * kRun;

// Where the row of a cache slot begins (elements); -1: not written.
__device__ __forceinline__ int64_t cache_row(const QkParams &p, const CacheView &c, int64_t s)
{
    if (s < 0 || s >= p.num_slots) return -1;                // num_slots < 2^31
    const uint32_t page = (uint32_t)s / (uint32_t)p.page_size, row = (uint32_t)s - page * (uint32_t)p.page_size;
    return (int64_t)page * c.ps + (int64_t)row * c.ss;
}

// What the values of an FP8 cache are multiplied by: RN(1 / scale), at most
// the largest FP32 value (infinite, from a scale up to 2^-128, it would turn
// zeros into NaN).
__device__ __forceinline__ float scale_reciprocal(const float *scale)
{
    const float inv = __frcp_rn(ld_f32_ro(scale));
    return inv > FLT_MAX ? FLT_MAX : inv;
}

// A piece of `count` values to a cache of BF16 or, divided by the scale, FP8.
template <int V>
__device__ __forceinline__ void st_cache(void *base, int64_t off, int kind, const F2 (&y)[4], float inv, int count)
{
    if (kind == CRMSN_CACHE_BF16) {
        st_piece<V>(static_cast<uint16_t *>(base) + off, y, count);
        return;
    }
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const F2 z = f2_mul(y[i], f2(inv));
        c[i] = (kind == CRMSN_CACHE_E4M3 ? pack_fp8<0>(f2_lo(z), f2_hi(z)) : pack_fp8<1>(f2_lo(z), f2_hi(z))) & 0xffffu;
    }
    uint8_t *q = static_cast<uint8_t *>(base) + off;
#pragma unroll
    for (int e = 0; e < 8; e += V) {
        if (e >= count || !dbg_global(q + e, V, true)) continue;
        const uint32_t four = c[e / 2] | (V > 2 ? c[(e / 2 + 1) & 3] << 16 : 0u);
        if constexpr (V == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(four, c[2] | c[3] << 16);
        else if constexpr (V == 4) *reinterpret_cast<uint32_t *>(q + e) = four;
        else *reinterpret_cast<uint16_t *>(q + e) = (uint16_t)four;
    }
}

enum Role { TO_HEADS, KEY_TO_CACHE, VALUE_TO_CACHE };

using Ring = uint4[kStages][2][kThreads];

// One warp's rows of tensor `which`.
template <int N, bool WHOLE, int V, bool NORM, bool PAIRS, int ROLE>
__device__ __forceinline__ void walk_rows(const QkParams &p, int which, int block, Ring &ring)
{
    constexpr bool kRotate = ROLE != VALUE_TO_CACHE, kNorm = NORM && kRotate;
    const Lanes<N> L(p.lanes);
    const Pieces pc = lane_pieces<N, WHOLE>(L.l, p.R, p.D);
    const int H = p.in[which].H, tid = threadIdx.x, delta = pc.b - pc.a, P = p.cs_rows;
    const Share &sh = p.share[which];
    const LaneRows mine(sh, H, block * (kThreads / 32) + (tid >> 5), L.grp, L.rows());
    int64_t t = mine.t;
    Walk<const uint16_t> in = {p.in[which].p + t * p.in[which].ld + mine.h * p.in[which].hs + pc.a, mine.h};
    grid_wait();
    if (mine.most == 0) return;
    int to_issue = mine.mine;
    auto issue = [&](int stage) {
        if (to_issue > 0) {
            copy_piece<N, WHOLE, V>(&ring[stage][0][tid], in.p, pc.ca, p.l1);
            copy_piece<N, WHOLE, V>(&ring[stage][1][tid], in.p + delta, pc.cb, p.l1);
        }
        --to_issue;
        const int e = stage % kRun == kRun - 1;
        in.step(sh.in[e], sh.dh[e], H);
    };
    // What a row's last pieces lack stays zero.
    if (N == 0 && (pc.ca < 8 || pc.cb < 8))
        for (int i = 0; i < kStages; ++i) ring[i][0][tid] = ring[i][1][tid] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kRun; ++i) issue(i);
    ring_commit();

    F2 wa[4], wb[4];
    if constexpr (kNorm) {
        ld_weights<V>(wa, p.w[which], p.w32, p.bias, pc.a, pc.ca);
        ld_weights<V>(wb, p.w[which], p.w32, p.bias, pc.b, pc.cb);
    }
    // Where the rows go: a heads tensor, or a head's place in a cache row.
    const bool fp8 = ROLE != TO_HEADS && p.kind != CRMSN_CACHE_BF16;
    float inv = 1.f;
    if (fp8) inv = scale_reciprocal(p.scale[which - 1]);
    Walk<uint16_t> out = {nullptr, mine.h};
    int64_t head = 0, base = 0;
    if constexpr (ROLE == TO_HEADS)
        out.p = const_cast<uint16_t *>(p.out[which].p) + t * p.out[which].ld + mine.h * p.out[which].hs + pc.a;
    else
        head = mine.h * p.cache[which - 1].hs + pc.a;
    int tc = (int)(t % P);                           // row of cos_sin
    Turn turn;
    if (kRotate && pc.rot && mine.mine > 0) ld_turn<PAIRS, V>(turn, p.cs + (int64_t)tc * p.ldcs, L.l, p.R, pc);
    // A token's slot is asked for a step before it is looked at.
    int64_t slot = -1;
    bool fresh = true;
    if constexpr (ROLE != TO_HEADS)
        if (mine.mine > 0) slot = ld_index(p.slots, p.slot64, t);
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
                if (on) {
                    st_piece<V>(out.p, a, pc.ca);
                    st_piece<V>(out.p + delta, b, pc.cb);
                }
            } else if (on) {
                if (fresh) base = cache_row(p, p.cache[which - 1], slot);
                void *c = p.cache[which - 1].p;
                const int ca = base < 0 ? 0 : pc.ca, cb = base < 0 ? 0 : pc.cb;
                st_cache<V>(c, base + head, p.kind, a, inv, ca);
                st_cache<V>(c, base + head + delta, p.kind, b, inv, cb);
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
            fresh = over || sh.dt[e] > 0;
            if (fresh && i + 1 < mine.mine) {
                if (kRotate && pc.rot) ld_turn<PAIRS, V>(turn, p.cs + (int64_t)tc * p.ldcs, L.l, p.R, pc);
                if constexpr (ROLE != TO_HEADS) slot = ld_index(p.slots, p.slot64, t);
            }
        }
    }
}

template <int N, bool WHOLE, int V, bool NORM, bool PAIRS, bool APPEND>
__global__ void __launch_bounds__(kThreads, qk_fwd_ctas_per_sm(APPEND, NORM, N == 0)) k_qk_fwd(const QkParams p)
{
    CRMSN_DEBUG_ENTER(p.dbg);
    Ring &ring = *reinterpret_cast<Ring *>(heads_smem);
    int block = blockIdx.x, which = 0;
    while (which < (APPEND ? 2 : 1) && block >= p.share[which].blocks) block -= p.share[which++].blocks;
    if (!APPEND || which == 0) walk_rows<N, WHOLE, V, NORM, PAIRS, TO_HEADS>(p, which, block, ring);
    else if (which == 1) walk_rows<N, WHOLE, V, NORM, PAIRS, KEY_TO_CACHE>(p, 1, block, ring);
    else walk_rows<N, WHOLE, V, NORM, PAIRS, VALUE_TO_CACHE>(p, 2, block, ring);
}

template <int N, bool WHOLE, int V, bool APPEND>
cudaError_t go(const QkParams &p, bool norm, dim3 grid, cudaStream_t s)
{
    const dim3 b(kThreads);
    if (norm) return p.pairs ? launch_pdl(k_qk_fwd<N, WHOLE, V, true, true, APPEND>, grid, b, sizeof(Ring), s, p)
                             : launch_pdl(k_qk_fwd<N, WHOLE, V, true, false, APPEND>, grid, b, sizeof(Ring), s, p);
    return p.pairs ? launch_pdl(k_qk_fwd<N, WHOLE, V, false, true, APPEND>, grid, b, sizeof(Ring), s, p)
                   : launch_pdl(k_qk_fwd<N, WHOLE, V, false, false, APPEND>, grid, b, sizeof(Ring), s, p);
}

// The 16-byte form: head sizes 64, 128, 192 and 256 have code of their own,
// with the lanes of a row (and, if all of it is rotated, the distance of its
// two pieces) known.  Measured with the general code: D = 128 (32 + 8 heads,
// T = 16384) 60.8 -> 56.2 us; an append of D = 192 (32 + 4 heads, T = 8797)
// 71.4 -> 54.7 (50.2 with its CTAs dealt by cost), its backward 86.1 -> 81.7.
// (D = 80 and 96: 3 %, not kept.)
template <bool APPEND>
cudaError_t go(const QkParams &p, bool norm, dim3 grid, cudaStream_t s)
{
    const bool whole = p.R == p.D;
    if (p.D == 64) return whole ? go<4, true, 8, APPEND>(p, norm, grid, s) : go<4, false, 8, APPEND>(p, norm, grid, s);
    if (p.D == 128) return whole ? go<8, true, 8, APPEND>(p, norm, grid, s) : go<8, false, 8, APPEND>(p, norm, grid, s);
    if (p.D == 256) return whole ? go<16, true, 8, APPEND>(p, norm, grid, s) : go<16, false, 8, APPEND>(p, norm, grid, s);
    if (p.D == 192) return whole ? go<12, true, 8, APPEND>(p, norm, grid, s) : go<12, false, 8, APPEND>(p, norm, grid, s);
    return go<0, false, 8, APPEND>(p, norm, grid, s);
}

}  // namespace

}  // namespace crmsn
