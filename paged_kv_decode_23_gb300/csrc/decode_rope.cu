// decode_rope.cu -- the tensor-core decode kernels with ROPE_LLAMA (plan's pos_encoding_mode):
// q and every K row are rotated in registers before the QK MMAs (in fp16), for each q / KV
// dtype pair and head_dim the plain kernels are built for.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_rope(std::vector<DecodeKernel>& out) {
  tensor_core_16<__half, kUnbounded, true>(out);
  tensor_core_16<__nv_bfloat16, kUnbounded, true>(out);
  tensor_core_e4m3<__half, kUnbounded, true>(out);
  tensor_core_e4m3<__nv_bfloat16, kUnbounded, true>(out);
}

}  // namespace pkd
