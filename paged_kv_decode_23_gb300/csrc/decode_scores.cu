// decode_scores.cu -- the tensor-core decode kernels that also leave every attended key's score
// (the first half of a plan with key weights; key_weights.cu is the second), with or without sinks;
// 16-bit and e4m3 caches.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_scores(std::vector<DecodeKernel>& out) {
  tensor_core_16<__half, kScores>(out);
  tensor_core_16<__nv_bfloat16, kScores>(out);
  tensor_core_e4m3<__half, kScores>(out);
  tensor_core_e4m3<__nv_bfloat16, kScores>(out);
}

}  // namespace pkd
