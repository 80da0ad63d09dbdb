// heads_append.cu -- the 16-byte form of the append to a paged cache.
#include "heads_fwd.cuh"

namespace crmsn {

cudaError_t run_qk_append(const QkParams &p, bool norm, dim3 grid, cudaStream_t s) { return go<true>(p, norm, grid, s); }

}  // namespace crmsn
