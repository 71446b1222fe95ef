// decode_e2m1.cu -- instantiations of the 4-bit decode kernel, fp16 or bf16 q / o.
#include "decode_e2m1_kernels.cuh"

namespace pkd {

void register_decode_e2m1(std::vector<DecodeKernel>& out) {
  register_e2m1_geometries<__half, kUnbounded>(out, kF16);
  register_e2m1_geometries<__nv_bfloat16, kUnbounded>(out, kBF16);
}

}  // namespace pkd
