// The tensor-core kernel's gated block.
#include "q2k_ffn_tc_kernel.cuh"

namespace q2k {

template cudaError_t launch_tc<Tc::kGated, __nv_bfloat16, false>(TcArgs, const Plan&, uint8_t*, const void*, const void*,
                                                       int, int, int, cudaStream_t, int);
template cudaError_t launch_tc<Tc::kGated, float, false>(TcArgs, const Plan&, uint8_t*, const void*, const void*,
                                                       int, int, int, cudaStream_t, int);

}  // namespace q2k
