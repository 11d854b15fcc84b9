// Cache in 4 bits on tcgen05: bf16.
#include "q4_tc.cuh"

namespace kve {
template cudaError_t launch_q4_tc<__nv_bfloat16>(const PgDims &D, const Q4Shape &Q, const PgAttn &A, bool own, cudaStream_t st);
}  // namespace kve
