// attn_combine.cu -- joins the parts of the tiles that several CTAs shared:
// with a part's maximum M_i, sum L_i and values O_i (relative to M_i),
//   M = max M_i,  L = sum L_i 2^(M_i - M),  o = sum O_i 2^(M_i - M) / L.
//
// CTA column c looks at the tile in which the work of CTA Hk + c of the
// attention kernel began, and joins it where its group is the first such one.
// Parts are added in the order of their keys, a row by a warp.  (Two rows a warp
// in tiled calls: 24 packed prompts 475 us against 476, 64 texts 47.3 against
// 47.3, a small chunk 43.3 against 42.5.)
#include "attn.cuh"

namespace crmsn {
namespace {

constexpr int kWarps = 8;

// CTAs of an SM, which the registers of the rare call would cost.  (Limits of 3
// to 5 by head size, as many registers as that call wants, against 5: a chunk in
// E5M2 with heads of 64 42.9 against 42.5 us, a window with heads of 256 190.0
// against 187.3.  6: 43.0, 187.8.)
constexpr int kCtas = 5;

template <int KIND, int DP>
__global__ void __launch_bounds__(kWarps * 32, kCtas) k_attn_combine(const __grid_constant__ AttnParams p, int rows)
{
    constexpr int NV = DP / 64;              // pairs of columns of a lane
    CRMSN_DEBUG_ENTER(p.dbg);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = (int)blockIdx.x + p.Hk, g = c / p.Hk;
    AttnHeader *at = reinterpret_cast<AttnHeader *>(p.ws) + c;
    if (!dbg_global(at, (int)sizeof(AttnHeader), false)) return;
    const AttnHeader hd = *at;
    if (!hd.tile || first_unit(hd.units, hd.groups, g - 1) > hd.first) return;
    const int nrows = hd.ntok * p.group.d, lane = threadIdx.x & 31;
    const int r = (int)blockIdx.y * kWarps + (int)(threadIdx.x >> 5);
    if (r >= nrows) return;
    const int n = unit_owner(hd.units, hd.groups, hd.last - 1) - g + 2;
    const float vs = KIND == KV_BF16 ? 1.f : ld_f32_ro(p.scale[1]);
    // The part of the group before is its second (the tile begins there), that of the others their first.
    const auto part = [&](int i) { return part_of(p.ws, c + (i - 1) * p.Hk, i == 0, rows, DP); };
    float M = -INFINITY, L = 0.f;
    F2 o[NV];
    for (int k = 0; k < NV; ++k) o[k] = f2(0.f);
    for (int base = 0; base < n; base += 32) {
        float m = -INFINITY, l = 0.f;
        if (base + lane < n) {
            const float *ml = part(base + lane) + 2 * r;
            if (dbg_global(ml, 8, false)) {
                m = ml[0];
                l = ml[1];
            }
        }
        float top = m;
        for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        top = fmaxf(top, M);
        const float ref = top == -INFINITY ? 0.f : top;
        const float keep = exp2f(M - ref), mine = exp2f(m - ref);
        M = top;
        L *= keep;
        for (int k = 0; k < NV; ++k) o[k] = f2_mul(o[k], f2(keep));
        const int here = min(32, n - base);
#pragma unroll 4
        for (int i = 0; i < here; ++i) {
            const float w = __shfl_sync(0xffffffffu, mine, i);
            L = fmaf(__shfl_sync(0xffffffffu, l, i), w, L);
            const float *v = part(base + i) + 2 * rows + (int64_t)r * DP + 2 * lane;
            for (int k = 0; k < NV; ++k)
                if (dbg_global(v + 64 * k, 8, false))
                    o[k] = f2_fma(*reinterpret_cast<const float2 *>(v + 64 * k), f2(w), o[k]);
        }
    }
    const int i = p.group.div(r), hq = hd.h * p.group.d + (r - i * p.group.d);
    const int64_t t = hd.tok + i;
    const float inv = vs / L;
    uint16_t *out = const_cast<uint16_t *>(p.out.p) + t * p.out.ld + hq * p.out.hs + 2 * lane;
    bool odd = false;
    for (int k = 0; k < NV; ++k) {
        const F2 y = L == 0.f ? f2(0.f) : f2_mul(o[k], f2(inv));    // no key: zeros, whatever 0 times the values was
        odd = odd || (2 * lane + 64 * k < p.D && (suspect(y.x, L) || suspect(y.y, L)));
        if (2 * lane + 64 * k < p.D && dbg_global(out + 64 * k, 4, true))
            *reinterpret_cast<uint32_t *>(out + 64 * k) = bf16_f2(y);
    }
    if (p.lse && lane == 0) st_f32(p.lse + t * p.out.H + hq, L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718f);
    if (__any_sync(0xffffffffu, odd)) work_out_again<KIND, DP / 32>(p, hd.b, hd.h, hd.tok, hd.ntok, (int)t, hq, lane == 0);
}

template <int KIND>
cudaError_t run(const AttnParams &p, int rows, int DP, dim3 grid, cudaStream_t s)
{
    const dim3 block(kWarps * 32);
    switch (DP) {
        case 64: return launch_pdl(k_attn_combine<KIND, 64>, grid, block, 0, s, p, rows);
        case 128: return launch_pdl(k_attn_combine<KIND, 128>, grid, block, 0, s, p, rows);
        case 192: return launch_pdl(k_attn_combine<KIND, 192>, grid, block, 0, s, p, rows);
        default: return launch_pdl(k_attn_combine<KIND, 256>, grid, block, 0, s, p, rows);
    }
}

}  // namespace

cudaError_t launch_attn_combine(const AttnParams &p, int rows, int DP, int groups, cudaStream_t s)
{
    if (groups < 2) return cudaSuccess;
    const dim3 grid((groups - 1) * p.Hk, (rows + kWarps - 1) / kWarps);
    switch (p.kind) {
        case KV_BF16: return run<KV_BF16>(p, rows, DP, grid, s);
        case KV_E4M3: return run<KV_E4M3>(p, rows, DP, grid, s);
        default: return run<KV_E5M2>(p, rows, DP, grid, s);
    }
}

}  // namespace crmsn
