// The tensor-core kernel's projection with an epilogue.
#include "q2k_ffn_tc_kernel.cuh"

namespace q2k {

template cudaError_t launch_tc<Tc::kLinear, __nv_bfloat16, false>(TcArgs, const Plan&, uint8_t*, const void*, const void*,
                                                       int, int, int, cudaStream_t, int);
template cudaError_t launch_tc<Tc::kLinear, float, false>(TcArgs, const Plan&, uint8_t*, const void*, const void*,
                                                       int, int, int, cudaStream_t, int);

}  // namespace q2k
