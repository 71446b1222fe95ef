// cache_gather.cu -- listed token rows of a paged cache back as 16-bit rows (pkd_gather).
//
// A row of one head is spread over head_dim / 8 lanes, eight values each: 16, 8 or 4 bytes in,
// 16 bytes out.  A group of lanes takes R rows of one token (its K and V heads), all loaded
// before the first is used.  Nothing is computed but the widening and one multiply: bytes bound.
#include <type_traits>

#include "cache_rows.cuh"

namespace pkd {
namespace {

using namespace rows;

struct GatherParams {
  pkd_gather_args a;
  int64_t token0;
  uint32_t items;
  uint32_t chunks;
  int heads;  // kv heads of K and of V together (of the one that is asked for)
  int page_log;
};

constexpr int kThreads = 256;

template <typename T, int KV>
__device__ __forceinline__ void widen8(const uint4& raw, uint32_t scale, float (&x)[8]) {
  if constexpr (KV == kSame16) {
    unpack8<T>(raw, x);
  } else if constexpr (KV == kFp8) {
    uint32_t h[4];
    dev::e4m3x4_to_half2x2(raw.x, h[0], h[1]);
    dev::e4m3x4_to_half2x2(raw.y, h[2], h[3]);
    unpack8<__half>(make_uint4(h[0], h[1], h[2], h[3]), x);
  } else {
    uint4 h;
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h.x), "=r"(h.y), "=r"(h.z), "=r"(h.w)
        : "r"(raw.x));
    unpack8<__half>(h, x);
    const float s = e4m3_value(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= s;  // at most 6 bits: exact
  }
}

template <typename T, int KV, int D, int R>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ GatherParams p) {
  constexpr int LANES = D / 8;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const pkd_gather_args& a = p.a;
  const int gl = threadIdx.x & (LANES - 1);
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  if (item >= p.items) return;
  const uint32_t tok = item / p.chunks;
  const int c0 = (int)(item - tok * p.chunks);
  const int64_t t = p.token0 + tok;
  const int b = __ldg(a.batch_indices + t);
  if (b < 0) return;
  const Slot slot = find_slot(a.pool, p.page_log, b, __ldg(a.positions + t));
  if (slot.status) {
    if (gl == 0 && a.status) atomicOr(a.status, slot.status);
    return;
  }
  const int hkv = a.pool.num_kv_heads;
  uint4 raw[R];
  uint32_t sf[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int r = c0 + j * (int)p.chunks;
    raw[j] = make_uint4(0, 0, 0, 0);
    sf[j] = 0;
    if (r < p.heads) {
      const bool is_v = a.k_out == nullptr || r >= hkv;
      const int head = r >= hkv ? r - hkv : r;
      const char* src = row_addr<KV>(is_v ? a.pool.v : a.pool.k, a.pool.strides, slot, head, gl);
      if constexpr (KV == kSame16) raw[j] = *reinterpret_cast<const uint4*>(src);
      else if constexpr (KV == kFp8) {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        raw[j].x = v.x;
        raw[j].y = v.y;
      } else {
        raw[j].x = *reinterpret_cast<const uint32_t*>(src);
        sf[j] = *scale_addr(is_v ? a.pool.v_scales : a.pool.k_scales, a.pool.scale_strides, slot,
                            head, gl);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int r = c0 + j * (int)p.chunks;
    if (r >= p.heads) continue;
    const bool is_v = a.k_out == nullptr || r >= hkv;
    const int head = r >= hkv ? r - hkv : r;
    const float unit = is_v ? a.pool.v_scale : a.pool.k_scale;
    float x[8];
    widen8<T, KV>(raw[j], sf[j], x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= unit;
    T* dst = is_v ? static_cast<T*>(a.v_out) + t * a.v_out_strides[0] + head * a.v_out_strides[1]
                  : static_cast<T*>(a.k_out) + t * a.k_out_strides[0] + head * a.k_out_strides[1];
    *(reinterpret_cast<uint4*>(dst) + gl) = pack8<T>(x);
  }
}

template <typename T, int KV, int D, int R>
cudaError_t launch_r(const pkd_gather_args& a, cudaStream_t s) {
  constexpr int LANES = D / 8;
  GatherParams p;
  p.a = a;
  p.heads = a.pool.num_kv_heads * ((a.k_out != nullptr) + (a.v_out != nullptr));
  p.chunks = (uint32_t)(p.heads + R - 1) / R;
  p.page_log = __builtin_ctz((unsigned)a.pool.page_size);
  const int64_t slab = (int64_t(1) << 30) / p.chunks;  // tokens a launch counts in 32 bits
  for (int64_t t0 = 0; t0 < a.num_tokens; t0 += slab) {
    const int64_t n = a.num_tokens - t0 < slab ? a.num_tokens - t0 : slab;
    p.token0 = t0;
    p.items = (uint32_t)(n * p.chunks);
    const unsigned grid = (p.items + kThreads / LANES - 1) / (kThreads / LANES);
    cudaError_t e = launch_pdl(gather_kernel<T, KV, D, R>, p, grid, kThreads, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int KV>
cudaError_t launch_kv(const pkd_gather_args& a, cudaStream_t s) {
  switch (a.pool.head_dim) {
    case 64: return launch_r<T, KV, 64, 4>(a, s);
    case 128: return launch_r<T, KV, 128, 4>(a, s);
    default: return launch_r<T, KV, 256, 4>(a, s);
  }
}

template <typename T>
cudaError_t launch_t(const pkd_gather_args& a, cudaStream_t s) {
  switch (a.pool.dtype) {
    case PKD_DTYPE_E4M3: return launch_kv<T, kFp8>(a, s);
    case PKD_DTYPE_E2M1: return launch_kv<T, kFp4>(a, s);
    default: return launch_kv<T, kSame16>(a, s);
  }
}

}  // namespace

cudaError_t launch_gather(const pkd_gather_args& a, cudaStream_t s) {
  return a.out_dtype == PKD_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<__half>(a, s);
}

}  // namespace pkd
