// heads_bwd_narrow.cu -- the query / key backward with 8- and 4-byte accesses.
#include "heads_bwd.cuh"

namespace crmsn {

cudaError_t run_qk_bwd_narrow(const QkBwdParams &p, bool norm, int vec, dim3 grid, cudaStream_t s)
{
    return vec == 4 ? go_bwd<0, false, 4>(p, norm, grid, s) : go_bwd<0, false, 2>(p, norm, grid, s);
}

}  // namespace crmsn
