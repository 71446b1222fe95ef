// decode_e2m1_weights.cu -- the 4-bit decode kernels that also leave every attended key's score (the
// first half of a plan with key weights), in the geometries of decode_e2m1.cu.
#include "decode_e2m1_kernels.cuh"

namespace pkd {

void register_decode_e2m1_weights(std::vector<DecodeKernel>& out) {
  register_e2m1_geometries<__half, true>(out, kF16);
  register_e2m1_geometries<__nv_bfloat16, true>(out, kBF16);
}

}  // namespace pkd
