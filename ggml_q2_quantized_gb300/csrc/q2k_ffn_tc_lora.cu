// The tensor-core kernel's projection with adapters.
#include "q2k_ffn_tc_kernel.cuh"

namespace q2k {

template cudaError_t launch_tc<Tc::kLora, __nv_bfloat16, false>(TcArgs, const Plan&, uint8_t*, const void*, const void*,
                                                       int, int, int, cudaStream_t, int);
template cudaError_t launch_tc<Tc::kLora, float, false>(TcArgs, const Plan&, uint8_t*, const void*, const void*,
                                                       int, int, int, cudaStream_t, int);

}  // namespace q2k
