// decode_geometries.cuh -- the geometries in which the decode kernels over 16-bit and e4m3 caches are
// built, for the files that instantiate them: plain, taking sinks (kSinks) or leaving scores (kScores).
// Tiles are sized so one pipeline stage (K + V) is 32 KiB: 16 bits, head_dim 64 -> 128 tokens, 128 -> 64,
// 256 -> 32; e4m3, 128 -> 128 tokens, 256 -> 64.  Three stages per CTA, two CTAs per SM; where the
// CUDA-core kernels' rotated q buffers would leave room for only one CTA per SM, two stages.
#ifndef PKD_DECODE_GEOMETRIES_CUH_
#define PKD_DECODE_GEOMETRIES_CUH_

#include <type_traits>

#include "decode_kernels.cuh"

namespace pkd {

template <typename TQ>
constexpr int kCode = std::is_same<TQ, __half>::value ? kF16 : kBF16;

// Plans without sinks run instances of their own: on the CUDA cores and with ROPE_LLAMA those that take
// sinks are up to 4.9 % slower (us without and with, 64 rows of 512 to 4,096 keys, 8 kv heads: fp16, head_dim
// 64, 4 qo heads, rotating 98.3 and 103.2; head_dim 128, 1 head, rotating 115.5 and 120.6; e4m3, 256, tensor
// cores, rotating 63.0 and 65.4).  In these geometries they measured 1 to 6 % faster instead and serve plain
// plans as well (fp16, 128, 8 heads 215.0 and 212.4, rotating 335.5 and 326.0; e4m3, 128, 4 heads 119.4 and
// 118.1, rotating 193.7 and 182.0; e4m3, 256, 2 heads, rotating 175.8 and 170.2).
constexpr bool sinks_serve_plain(int kind, bool kv_fp8, int d, int heads, bool rope) {
  if (kind != kCudaCore) return false;
  if (kv_fp8) return (d == 128 && heads == 4) || (d == 256 && heads == 2 && rope);
  return heads == 8 && (d == 128 || (d == 256 && !rope));
}

template <typename TQ, bool KV_FP8, int D, int TS, int NSTAGES, int KIND, int GP, bool ROPE, int BOUNDED>
void add(std::vector<DecodeKernel>& out) {
  if constexpr (BOUNDED != kUnbounded || !sinks_serve_plain(KIND, KV_FP8, D, GP, ROPE))
    out.push_back(make_decode_kernel<TQ, KV_FP8, D, TS, NSTAGES, KIND, GP, ROPE, BOUNDED>(
        kCode<TQ>, KV_FP8 ? (int)kE4M3 : (int)kCode<TQ>));
}

template <typename TQ, int BOUNDED, bool ROPE = false>
void tensor_core_16(std::vector<DecodeKernel>& out) {
  add<TQ, false, 64, 128, 3, kTensorCore, 8, ROPE, BOUNDED>(out);
  add<TQ, false, 128, 64, 3, kTensorCore, 8, ROPE, BOUNDED>(out);
  add<TQ, false, 256, 32, 3, kTensorCore, 8, ROPE, BOUNDED>(out);
}

template <typename TQ, int BOUNDED, bool ROPE = false>
void tensor_core_e4m3(std::vector<DecodeKernel>& out) {
  add<TQ, true, 128, 128, 3, kTensorCore, 8, ROPE, BOUNDED>(out);
  add<TQ, true, 256, 64, 3, kTensorCore, 8, ROPE, BOUNDED>(out);
}

template <typename TQ, int BOUNDED, bool ROPE = false>
void cuda_core_16(std::vector<DecodeKernel>& out) {
  add<TQ, false, 64, 128, 3, kCudaCore, 1, ROPE, BOUNDED>(out);
  add<TQ, false, 64, 128, 3, kCudaCore, 2, ROPE, BOUNDED>(out);
  add<TQ, false, 64, 128, 3, kCudaCore, 4, ROPE, BOUNDED>(out);
  add<TQ, false, 64, 128, 3, kCudaCore, 8, ROPE, BOUNDED>(out);
  add<TQ, false, 128, 64, 3, kCudaCore, 1, ROPE, BOUNDED>(out);
  add<TQ, false, 128, 64, 3, kCudaCore, 2, ROPE, BOUNDED>(out);
  add<TQ, false, 128, 64, 3, kCudaCore, 4, ROPE, BOUNDED>(out);
  add<TQ, false, 128, 64, ROPE ? 2 : 3, kCudaCore, 8, ROPE, BOUNDED>(out);
  add<TQ, false, 256, 32, 3, kCudaCore, 1, ROPE, BOUNDED>(out);
  add<TQ, false, 256, 32, 3, kCudaCore, 2, ROPE, BOUNDED>(out);
  add<TQ, false, 256, 32, ROPE ? 2 : 3, kCudaCore, 4, ROPE, BOUNDED>(out);
  add<TQ, false, 256, 32, ROPE ? 2 : 3, kCudaCore, 8, ROPE, BOUNDED>(out);
}

template <typename TQ, int BOUNDED, bool ROPE = false>
void cuda_core_e4m3(std::vector<DecodeKernel>& out) {
  add<TQ, true, 128, 128, 3, kCudaCore, 1, ROPE, BOUNDED>(out);
  add<TQ, true, 128, 128, 3, kCudaCore, 2, ROPE, BOUNDED>(out);
  add<TQ, true, 128, 128, 3, kCudaCore, 4, ROPE, BOUNDED>(out);
  add<TQ, true, 128, 128, 3, kCudaCore, 8, ROPE, BOUNDED>(out);
  add<TQ, true, 256, 64, 3, kCudaCore, 1, ROPE, BOUNDED>(out);
  add<TQ, true, 256, 64, ROPE ? 2 : 3, kCudaCore, 2, ROPE, BOUNDED>(out);
  add<TQ, true, 256, 64, ROPE ? 2 : 3, kCudaCore, 4, ROPE, BOUNDED>(out);
  add<TQ, true, 256, 64, ROPE ? 2 : 3, kCudaCore, 8, ROPE, BOUNDED>(out);
}

}  // namespace pkd

#endif  // PKD_DECODE_GEOMETRIES_CUH_
