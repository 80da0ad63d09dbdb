// attn_row.cu -- attention with one warp for each row: the form for head sizes
// and layouts that the tiled kernels do not take.  Every key is read once for
// every row, so its rate is that of the L1 and L2 caches.
#include "attn.cuh"

namespace crmsn {
namespace {

constexpr int kWarps = 4;

template <int KIND, int NE>
__global__ void __launch_bounds__(kWarps * 32) k_attn_row(const __grid_constant__ AttnParams p)
{
    CRMSN_DEBUG_ENTER(p.dbg);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t rows = (int64_t)p.T * p.q.H;
    for (int64_t r = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; r < rows; r += (int64_t)gridDim.x * kWarps) {
        const int t = (int)(r / p.q.H), hq = (int)(r - (int64_t)t * p.q.H);
        int b;
        if (p.starts) {
            // The last sequence that starts at t or before it.
            int lo = 0, hi = p.B;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (ld_index(p.starts + mid) <= t) lo = mid + 1;
                else hi = mid;
            }
            b = lo - 1;
            if (b < 0) continue;
        } else {
            b = t / p.n;
        }
        const Seq s = sequence(p, b);
        if (t < s.first || t - s.first >= s.n) continue;       // a row of no sequence stays as it is
        attend_row<KIND, NE, NE <= 8 ? 4 : 2>(p, b, s, t - s.first, hq, true);
    }
}

template <int KIND>
cudaError_t run(const AttnParams &p, int sms, cudaStream_t s)
{
    const int64_t rows = (int64_t)p.T * p.q.H, want = (rows + kWarps - 1) / kWarps, most = (int64_t)sms * 64;
    const dim3 grid((unsigned)(want < most ? want : most)), block(kWarps * 32);
    if (p.D <= 128) return launch_pdl(k_attn_row<KIND, 4>, grid, block, 0, s, p);
    if (p.D <= 256) return launch_pdl(k_attn_row<KIND, 8>, grid, block, 0, s, p);
    return launch_pdl(k_attn_row<KIND, 16>, grid, block, 0, s, p);
}

}  // namespace

cudaError_t launch_attn_row(const AttnParams &p, int sms, cudaStream_t s)
{
    switch (p.kind) {
        case KV_BF16: return run<KV_BF16>(p, sms, s);
        case KV_E4M3: return run<KV_E4M3>(p, sms, s);
        default: return run<KV_E5M2>(p, sms, s);
    }
}

}  // namespace crmsn
