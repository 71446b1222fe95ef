// decode_sinks.cu -- the tensor-core decode kernels that take sinks beside a window, without and with
// ROPE_LLAMA; 16-bit and e4m3 caches.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_sinks(std::vector<DecodeKernel>& out) {
  tensor_core_16<__half, kSinks>(out);
  tensor_core_16<__nv_bfloat16, kSinks>(out);
  tensor_core_e4m3<__half, kSinks>(out);
  tensor_core_e4m3<__nv_bfloat16, kSinks>(out);
  tensor_core_16<__half, kSinks, true>(out);
  tensor_core_16<__nv_bfloat16, kSinks, true>(out);
  tensor_core_e4m3<__half, kSinks, true>(out);
  tensor_core_e4m3<__nv_bfloat16, kSinks, true>(out);
}

}  // namespace pkd
