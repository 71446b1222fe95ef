// decode_rope_cc.cu -- the CUDA-core decode kernels with ROPE_LLAMA (plan's pos_encoding_mode
// with use_tensor_cores off), 16-bit KV: q rotated per tile, every K row in fp32 registers.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_rope_cc(std::vector<DecodeKernel>& out) {
  cuda_core_16<__half, kUnbounded, true>(out);
  cuda_core_16<__nv_bfloat16, kUnbounded, true>(out);
}

}  // namespace pkd
