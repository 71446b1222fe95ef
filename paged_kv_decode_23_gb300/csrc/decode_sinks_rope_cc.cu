// decode_sinks_rope_cc.cu -- the CUDA-core decode kernels with ROPE_LLAMA that take sinks beside a window;
// 16-bit caches.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_sinks_rope_cc(std::vector<DecodeKernel>& out) {
  cuda_core_16<__half, kSinks, true>(out);
  cuda_core_16<__nv_bfloat16, kSinks, true>(out);
}

}  // namespace pkd
