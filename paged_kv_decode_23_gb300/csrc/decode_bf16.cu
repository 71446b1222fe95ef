// decode_bf16.cu -- instantiations of the paged decode kernels for bf16 q / K / V / o.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_bf16(std::vector<DecodeKernel>& out) {
  tensor_core_16<__nv_bfloat16, kUnbounded>(out);
  cuda_core_16<__nv_bfloat16, kUnbounded>(out);
}

}  // namespace pkd
