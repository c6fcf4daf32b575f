// packed_gemm_bf16.cu -- the packed product's tensor-core kernels for bf16 activations.
#include "packed_gemm_launch.cuh"

namespace admmq {

int packed_gemm_bf16(const PackedArgs& p, cudaStream_t st) { return packed_gemm<__nv_bfloat16>(p, st); }
extern const GaveUp packed_bf16_gave_up = {take_gave_up, launch_give_up};

}  // namespace admmq
