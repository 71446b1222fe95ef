// cache_copy.cu -- pages copied inside each of many pools in one launch (pkd_copy_pages).
//
// The pool table and the page pairs travel as kernel parameters: no upload, no staging memory,
// and a captured launch holds its own lists.  A CTA copies one 16 KiB piece of one page of one
// pool; pieces of all pools count up within a pair, so that pools of different page sizes (codes
// and scales) mix.  The lists' 24 KB cost nothing that shows: with a second instance for lists of
// up to 64 pools and pairs, a copy of 4 pages in 16 pools took the same time on the host
// (16 to 17 us, most of it spent on looking at the tensors) and in a replayed graph (4.15 us).
// Bound: bytes.  786 MB of pages, read and written: 229 us, 6.87 TB/s, what a plain copy reaches.
#include "cache_ops.cuh"

namespace pkd {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kPiece = kThreads * kUnroll * 16;

struct CopyParams {
  CopyPool pools[PKD_COPY_POOLS];
  // first piece of each pool within a pair; the last entry: all pieces
  int32_t piece0[PKD_COPY_POOLS + 1];
  int32_t src[PKD_COPY_PAIRS];
  int32_t dst[PKD_COPY_PAIRS];
  int32_t n_pools;
};
static_assert(sizeof(CopyParams) <= 32764, "kernel parameters end at 32,764 bytes");

__global__ void __launch_bounds__(kThreads)
    copy_pages_kernel(const __grid_constant__ CopyParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t per_pair = (uint32_t)p.piece0[p.n_pools];
  const uint32_t pair = blockIdx.x / per_pair;
  const int piece = (int)(blockIdx.x - pair * per_pair);
  int lo = 0, hi = p.n_pools;  // piece0[lo] <= piece < piece0[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.piece0[mid] <= piece) lo = mid;
    else hi = mid;
  }
  const CopyPool pool = p.pools[lo];
  const int64_t off = (int64_t)(piece - p.piece0[lo]) * kPiece;
  const char* src = pool.base + p.src[pair] * pool.stride + off;
  char* dst = pool.base + p.dst[pair] * pool.stride + off;
  const int64_t left = pool.bytes - off;
  const int n = left < kPiece ? (int)left : kPiece;
  if (((reinterpret_cast<uintptr_t>(pool.base) | (uintptr_t)pool.stride | (uintptr_t)pool.bytes) & 15) == 0) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int at = (u * kThreads + threadIdx.x) * 16;
      if (at < n) v[u] = *reinterpret_cast<const uint4*>(src + at);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int at = (u * kThreads + threadIdx.x) * 16;
      if (at < n) *reinterpret_cast<uint4*>(dst + at) = v[u];
    }
  } else {  // pools of odd sizes or places: byte by byte
    for (int at = threadIdx.x; at < n; at += kThreads) dst[at] = src[at];
  }
}

cudaError_t launch_some(const CopyPool* pools, int n_pools, const int32_t* src, const int32_t* dst,
                        int n_pairs, cudaStream_t s) {
  CopyParams p;
  int64_t at = 0;
  for (int j = 0; j < n_pools; ++j) {
    p.pools[j] = pools[j];
    p.piece0[j] = (int32_t)at;
    at += (pools[j].bytes + kPiece - 1) / kPiece;
    if (at > INT32_MAX) return cudaErrorInvalidValue;
  }
  p.piece0[n_pools] = (int32_t)at;
  p.n_pools = n_pools;
  // at most 2^31 - 1 CTAs a launch
  const int64_t most = INT32_MAX / at;
  for (int i0 = 0; i0 < n_pairs;) {
    const int n = n_pairs - i0 < most ? n_pairs - i0 : (int)most;
    for (int i = 0; i < n; ++i) {
      p.src[i] = src[i0 + i];
      p.dst[i] = dst[i0 + i];
    }
    cudaError_t e = launch_pdl(copy_pages_kernel, p, (unsigned)(n * at), kThreads, s);
    if (e != cudaSuccess) return e;
    i0 += n;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_copy_pages(const CopyPool* pools, int n_pools, const int32_t* src,
                              const int32_t* dst, int64_t n_pairs, cudaStream_t s) {
  for (int j = 0; j < n_pools; j += PKD_COPY_POOLS) {
    const int np = n_pools - j < PKD_COPY_POOLS ? n_pools - j : PKD_COPY_POOLS;
    for (int64_t i = 0; i < n_pairs; i += PKD_COPY_PAIRS) {
      const int n = (int)(n_pairs - i < PKD_COPY_PAIRS ? n_pairs - i : PKD_COPY_PAIRS);
      cudaError_t e = launch_some(pools + j, np, src + i, dst + i, n, s);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace pkd
