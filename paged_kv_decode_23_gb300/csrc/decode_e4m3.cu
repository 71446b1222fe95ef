// decode_e4m3.cu -- instantiations of the paged decode kernels for fp8 e4m3 K/V with fp16 or
// bf16 q / o.
// Both variants widen e4m3 to fp16 in registers (exact: every e4m3 value is an fp16 value);
// the tensor-core variant runs fp16 MMAs on operands built straight from the fp8 bytes.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_e4m3(std::vector<DecodeKernel>& out) {
  tensor_core_e4m3<__half, kUnbounded>(out);
  tensor_core_e4m3<__nv_bfloat16, kUnbounded>(out);
  cuda_core_e4m3<__half, kUnbounded>(out);
  cuda_core_e4m3<__nv_bfloat16, kUnbounded>(out);
}

}  // namespace pkd
