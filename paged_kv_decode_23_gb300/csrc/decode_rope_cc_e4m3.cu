// decode_rope_cc_e4m3.cu -- the CUDA-core decode kernels with ROPE_LLAMA for e4m3 KV (f16 or
// bf16 q): each K row is widened to fp32 and rotated in registers.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_rope_cc_e4m3(std::vector<DecodeKernel>& out) {
  cuda_core_e4m3<__half, kUnbounded, true>(out);
  cuda_core_e4m3<__nv_bfloat16, kUnbounded, true>(out);
}

}  // namespace pkd
