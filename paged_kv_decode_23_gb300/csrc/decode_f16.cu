// decode_f16.cu -- instantiations of the paged decode kernels for f16 q / K / V / o.
#include "decode_geometries.cuh"

namespace pkd {

void register_decode_f16(std::vector<DecodeKernel>& out) {
  tensor_core_16<__half, kUnbounded>(out);
  cuda_core_16<__half, kUnbounded>(out);
}

}  // namespace pkd
