// decode_e2m1.cu -- instantiations of the 4-bit decode kernel, fp16 or bf16 q / o.
#include "decode_e2m1_kernels.cuh"

namespace pkd {

void register_decode_e2m1(std::vector<DecodeKernel>& out) {
  out.push_back(make_decode_e2m1<__half, 64, 128, 8>(kF16));
  out.push_back(make_decode_e2m1<__half, 128, 128, 5>(kF16));
  out.push_back(make_decode_e2m1<__half, 256, 64, 5>(kF16));
  out.push_back(make_decode_e2m1<__nv_bfloat16, 64, 128, 8>(kBF16));
  out.push_back(make_decode_e2m1<__nv_bfloat16, 128, 128, 5>(kBF16));
  out.push_back(make_decode_e2m1<__nv_bfloat16, 256, 64, 5>(kBF16));
}

}  // namespace pkd
