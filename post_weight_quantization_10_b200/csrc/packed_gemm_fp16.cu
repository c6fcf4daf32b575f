// packed_gemm_fp16.cu -- the packed product's tensor-core kernels for fp16 activations.
#include "packed_gemm_launch.cuh"

namespace admmq {

int packed_gemm_fp16(const PackedArgs& p, cudaStream_t st) { return packed_gemm<__half>(p, st); }
extern const GaveUp packed_fp16_gave_up = {take_gave_up, launch_give_up};

}  // namespace admmq
