// decode_sinks.cu -- the tensor-core decode kernels that take sinks beside a window;
// 16-bit and e4m3 caches, in the geometries of decode_f16.cu, decode_bf16.cu and decode_e4m3.cu.
#include "decode_kernels.cuh"

namespace pkd {

namespace {
template <typename TQ, bool KV_FP8, int D, int TS>
DecodeKernel bounded(int q, int kv) {
  return make_decode_kernel<TQ, KV_FP8, D, TS, 3, kTensorCore, 8, false, kSinks>(q, kv);
}
}  // namespace

void register_decode_sinks(std::vector<DecodeKernel>& out) {
  out.push_back(bounded<__half, false, 64, 128>(kF16, kF16));
  out.push_back(bounded<__half, false, 128, 64>(kF16, kF16));
  out.push_back(bounded<__half, false, 256, 32>(kF16, kF16));
  out.push_back(bounded<__nv_bfloat16, false, 64, 128>(kBF16, kBF16));
  out.push_back(bounded<__nv_bfloat16, false, 128, 64>(kBF16, kBF16));
  out.push_back(bounded<__nv_bfloat16, false, 256, 32>(kBF16, kBF16));
  out.push_back(bounded<__half, true, 128, 128>(kF16, kE4M3));
  out.push_back(bounded<__half, true, 256, 64>(kF16, kE4M3));
  out.push_back(bounded<__nv_bfloat16, true, 128, 128>(kBF16, kE4M3));
  out.push_back(bounded<__nv_bfloat16, true, 256, 64>(kBF16, kE4M3));
}

}  // namespace pkd
