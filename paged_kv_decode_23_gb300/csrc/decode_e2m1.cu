// decode_e2m1.cu -- instantiations of the 4-bit decode kernel, fp16 or bf16 q / o, for tasks of up
// to 4 or up to 8 qo heads: 4 where a kv head has no more.  Groups of 4 heads through the 8-head
// instance took 52.1 us for 45.4 (64 contexts of 512 to 4,096, head_dim 128), and 123 for 113 (4 of
// 131,072).  At head_dim 64 these cases take 30.3 and 75.9 us.
#include "decode_e2m1_kernels.cuh"

namespace pkd {

template <typename TQ>
void register_t(std::vector<DecodeKernel>& out, int q) {
  //                                  D  heads warps slices stages  CTAs per SM
  out.push_back(make_decode_e2m1<TQ, E2m1Geom<64, 4, 4, 2, 5>, 4>(q));
  out.push_back(make_decode_e2m1<TQ, E2m1Geom<128, 4, 4, 2, 3>, 4>(q));
  out.push_back(make_decode_e2m1<TQ, E2m1Geom<256, 4, 4, 2, 3>, 2>(q));
  out.push_back(make_decode_e2m1<TQ, E2m1Geom<64, 8, 4, 2, 4>, 4>(q));
  out.push_back(make_decode_e2m1<TQ, E2m1Geom<128, 8, 4, 2, 4>, 3>(q));
  out.push_back(make_decode_e2m1<TQ, E2m1Geom<256, 8, 4, 2, 3>, 2>(q));
}

void register_decode_e2m1(std::vector<DecodeKernel>& out) {
  register_t<__half>(out, kF16);
  register_t<__nv_bfloat16>(out, kBF16);
}

}  // namespace pkd
