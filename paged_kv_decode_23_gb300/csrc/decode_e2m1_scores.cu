// decode_e2m1_scores.cu -- the 4-bit decode kernels that also leave every attended key's score
// (the first half of a plan with key weights; key_weights.cu is the second), with or without sinks.
#include "decode_e2m1_kernels.cuh"

namespace pkd {

void register_decode_e2m1_scores(std::vector<DecodeKernel>& out) {
  register_e2m1_geometries<__half, kScores>(out, kF16);
  register_e2m1_geometries<__nv_bfloat16, kScores>(out, kBF16);
}

}  // namespace pkd
