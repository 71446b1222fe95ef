// cache_ops.cuh -- types shared by the page-cache operators' kernels and their C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pkd.h"

namespace pkd {

// Launchers (cache_append.cu, cache_gather.cu, cache_copy.cu); arguments are checked.
cudaError_t launch_append(const pkd_append_args& a, cudaStream_t s);
cudaError_t launch_gather(const pkd_gather_args& a, cudaStream_t s);

// One pool of a page copy: page p is the `bytes` bytes at base + p * stride.
struct CopyPool {
  char* base;
  int64_t stride;
  int64_t bytes;
};
cudaError_t launch_copy_pages(const CopyPool* pools, int n_pools, const int32_t* src,
                              const int32_t* dst, int64_t n_pairs, cudaStream_t s);

// A launch as a programmatic dependent of the stream's previous kernel: the kernel waits
// (griddepcontrol.wait) before it touches anything, so only the launch gap is hidden.
template <typename P>
inline cudaError_t launch_pdl(void (*kernel)(P), const P& prm, unsigned grid, unsigned threads,
                              cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<P*>(&prm)};
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), args);
}

}  // namespace pkd
