// decode_e2m1.cu -- instantiations of the 4-bit decode kernel, fp16 or bf16 q / o, for tasks of up
// to 4 or up to 8 qo heads.
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
