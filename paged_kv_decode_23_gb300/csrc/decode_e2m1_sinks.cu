// decode_e2m1_sinks.cu -- the 4-bit decode kernels that take sinks beside a window.
#include "decode_e2m1_kernels.cuh"

namespace pkd {

void register_decode_e2m1_sinks(std::vector<DecodeKernel>& out) {
  register_e2m1_geometries<__half, kSinks>(out, kF16);
  register_e2m1_geometries<__nv_bfloat16, kSinks>(out, kBF16);
}

}  // namespace pkd
