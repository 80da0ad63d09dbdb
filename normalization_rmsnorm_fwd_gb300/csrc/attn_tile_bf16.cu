// attn_tile_bf16.cu -- the tiled attention over BF16 keys and values.
#include "attn_tile.cuh"

namespace crmsn {

cudaError_t launch_attn_tile_bf16(const AttnParams &p, int sms, cudaStream_t s)
{
    switch (attn_padded(p.D)) {
        case 64: return run_attn_tile<KV_BF16, 64>(p, sms, s);
        case 128: return run_attn_tile<KV_BF16, 128>(p, sms, s);
        case 192: return run_attn_tile<KV_BF16, 192>(p, sms, s);
        default: return run_attn_tile<KV_BF16, 256>(p, sms, s);
    }
}

cudaError_t take_given_up_bf16(unsigned int &n) { return take_given_up(n); }

}  // namespace crmsn
