// heads_fwd.cu -- the 16-byte form of the query / key forward.
#include "heads_fwd.cuh"

namespace crmsn {

cudaError_t run_qk_fwd(const QkParams &p, bool norm, dim3 grid, cudaStream_t s) { return go<false>(p, norm, grid, s); }

}  // namespace crmsn
