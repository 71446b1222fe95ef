// decode_sinks_rope_cc_e4m3.cu -- the CUDA-core decode kernels with ROPE_LLAMA that take sinks beside a
// window; e4m3 caches.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_sinks_rope_cc_e4m3(std::vector<DecodeKernel>& out) {
  cuda_core_e4m3<__half, kSinks, true>(out);
  cuda_core_e4m3<__nv_bfloat16, kSinks, true>(out);
}

}  // namespace pkd
