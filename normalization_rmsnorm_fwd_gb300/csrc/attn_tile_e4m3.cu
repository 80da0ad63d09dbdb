// attn_tile_e4m3.cu -- the tiled attention over E4M3 keys and values.
#include "attn_tile.cuh"

namespace crmsn {

cudaError_t launch_attn_tile_e4m3(const AttnParams &p, int sms, cudaStream_t s)
{
    switch (attn_padded(p.D)) {
        case 64: return run_attn_tile<KV_E4M3, 64>(p, sms, s);
        case 128: return run_attn_tile<KV_E4M3, 128>(p, sms, s);
        case 192: return run_attn_tile<KV_E4M3, 192>(p, sms, s);
        default: return run_attn_tile<KV_E4M3, 256>(p, sms, s);
    }
}

cudaError_t take_given_up_e4m3(unsigned int &n) { return take_given_up(n); }

}  // namespace crmsn
