// heads_narrow.cu -- the forward and the append with 8- and 4-byte accesses.
#include "heads_fwd.cuh"

namespace crmsn {

cudaError_t run_qk_narrow(const QkParams &p, bool norm, bool append, int vec, dim3 grid, cudaStream_t s)
{
    if (append) return vec == 4 ? go<0, false, 4, true>(p, norm, grid, s) : go<0, false, 2, true>(p, norm, grid, s);
    return vec == 4 ? go<0, false, 4, false>(p, norm, grid, s) : go<0, false, 2, false>(p, norm, grid, s);
}

}  // namespace crmsn
