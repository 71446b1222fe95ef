// decode_sinks_cc.cu -- the CUDA-core decode kernels that take sinks beside a window; 16-bit and e4m3
// caches.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_sinks_cc(std::vector<DecodeKernel>& out) {
  cuda_core_16<__half, kSinks>(out);
  cuda_core_16<__nv_bfloat16, kSinks>(out);
  cuda_core_e4m3<__half, kSinks>(out);
  cuda_core_e4m3<__nv_bfloat16, kSinks>(out);
}

}  // namespace pkd
