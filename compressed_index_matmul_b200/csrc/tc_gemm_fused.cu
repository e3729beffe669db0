// The tensor-core forward with its fused epilogue (the kernel: tc_gemm.cuh).
#include "tc_gemm.cuh"

namespace vq {

cudaError_t launch_tc_fused(const LayerArgs& a, const Plan& pl, float* scratch, uint32_t* tickets, uint32_t* err,
                            cudaStream_t s) {
  return launch_tc_f<true>(a, pl, scratch, tickets, err, s);
}

}  // namespace vq
