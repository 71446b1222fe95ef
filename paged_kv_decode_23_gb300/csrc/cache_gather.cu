// cache_gather.cu -- listed token rows of a paged cache back as 16-bit rows (pkd_gather).
//
// A row of one head is spread over head_dim / 16 lanes, sixteen values each (of a 4-bit cache one
// block: eight code bytes and its scale): 32, 16 or 8 bytes in, 32 bytes out.  A group of lanes
// takes up to R neighbouring heads of one token's K or V, all loaded before the first is used.
// Nothing is computed but the widening and one product, rounded once: bytes bound.  345 MB of prefixes out of a
// 4-bit cache (HND, 8 heads of 128): 54.8 us, 6.3 TB/s; a call of some MB is latency, 3 us.
#include <cstring>
#include <type_traits>

#include "cache_rows.cuh"

namespace pkd {
namespace {

using namespace rows;

struct GatherParams {
  pkd_gather_args a;
  int64_t token0;
  uint32_t items;   // (token, chunk of heads) pairs of this launch
  uint32_t chunks;  // chunks of a token: hc of each of K and V that is asked for
  int hc;
  int page_log;
  int wide;         // the outputs' rows are 32-byte aligned: one store a lane
  int rounding[2];  // of K's and V's products
};

constexpr int kThreads = 64;

// How a product x * unit reaches T with one rounding; x has at most 11 bits.
//   kExact  unit has at most 12 bits: the 32-bit product is exact.
//   kSticky unit has more: no product is then a border of T (a border's odd part is below 2^12 and unit's
//           odd part divides the product's), so that the product cut off to 32 bits with its last bit set
//           rounds as the exact one does.
//   kWide   a unit of few bits that can take a bf16 value's product below 2^-149: 64 bits.
// The prefixes above out of 4 bits, e4m3 and bf16: 55.1, 62.5 and 80.7 us with kExact, 55.2, 63.7 and
// 88.0 with kSticky.  Every product's rest from an FMA, one way for all units, took 72.7 and 118 (4 bits, bf16).
enum Rounding { kExact = 0, kSticky = 1, kWide = 2 };

Rounding rounding_of(float unit, bool bf16_values) {
  uint32_t bits;
  std::memcpy(&bits, &unit, sizeof bits);  // (a normal number)
  const int zeros = __builtin_ctz((bits & 0x7fffffu) | 0x800000u);
  if (24 - zeros > 12) return kSticky;
  return bf16_values && (int)(bits >> 23) - 127 - (23 - zeros) < -16 ? kWide : kExact;
}

// Eight values of raw (of an e2m1 block: its codes' values without the scale).
template <typename T, int KV>
__device__ __forceinline__ void widen8(const uint4& raw, float (&x)[8]) {
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
  }
}

// x with its last bit set; an infinity (of a 16-bit cache) is itself.
template <int KV>
__device__ __forceinline__ float sticky(float x) {
  return KV == kSame16 && !(fabsf(x) < __int_as_float(0x7f800000)) ? x : __uint_as_float(__float_as_uint(x) | 1u);
}

template <typename T, int KV, int D, int R>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ GatherParams p) {
  constexpr int LANES = D / 16;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const pkd_gather_args& a = p.a;
  const int gl = threadIdx.x & (LANES - 1);
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  if (item >= p.items) return;
  const uint32_t tok = item / p.chunks;
  int c = (int)(item - tok * p.chunks);
  const int64_t t = p.token0 + tok;
  const int b = __ldg(a.batch_indices + t);
  if (b < 0) return;
  const Slot slot = find_slot(a.pool, p.page_log, b, __ldg(a.positions + t));
  if (slot.status) {
    if (gl == 0 && a.status) atomicOr(a.status, slot.status);
    return;
  }
  const bool is_v = a.k_out == nullptr || c >= p.hc;
  if (c >= p.hc) c -= p.hc;
  const int h0 = c * R, n = min(R, a.pool.num_kv_heads - h0);
  // heads follow each other at fixed strides
  const char* src = row_addr<KV>(is_v ? a.pool.v : a.pool.k, a.pool.strides, slot, h0, 16 * gl);
  const int64_t step = a.pool.strides[2] * (KV == kSame16 ? 2 : 1);
  uint4 raw[R][KV == kSame16 ? 2 : 1];
  uint32_t sf[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (j < n) {
      if constexpr (KV == kSame16) {
        raw[j][0] = reinterpret_cast<const uint4*>(src + j * step)[0];
        raw[j][1] = reinterpret_cast<const uint4*>(src + j * step)[1];
      } else if constexpr (KV == kFp8) {
        raw[j][0] = *reinterpret_cast<const uint4*>(src + j * step);
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(src + j * step);
        raw[j][0] = make_uint4(v.x, v.y, 0, 0);
      }
    }
  }
  if constexpr (KV == kFp4) {
    const uint8_t* at = scale_addr(is_v ? a.pool.v_scales : a.pool.k_scales, a.pool.scale_strides, slot, h0, 16 * gl);
#pragma unroll
    for (int j = 0; j < R; ++j) sf[j] = j < n ? at[j * a.pool.scale_strides[2]] : 0u;
  }
  constexpr bool bf16_values = KV == kSame16 && std::is_same<T, __nv_bfloat16>::value;
  const float unit = is_v ? a.pool.v_scale : a.pool.k_scale;
  const int rounding = p.rounding[is_v];
  const int64_t o0 = is_v ? a.v_out_strides[0] : a.k_out_strides[0];
  const int64_t o1 = is_v ? a.v_out_strides[1] : a.k_out_strides[1];
  T* dst = static_cast<T*>(is_v ? a.v_out : a.k_out) + t * o0 + h0 * o1 + 16 * gl;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (j >= n) break;
    // (an e2m1 value times its scale has at most 6 bits and is exact)
    const float s = KV == kFp4 ? e4m3_value(sf[j]) : 1.f;
    uint4 v16[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (KV == kSame16 && unit == 1.f) {
        v16[i] = raw[j][KV == kSame16 ? i : 0];
        continue;
      }
      float x[8];
      if constexpr (KV == kSame16) widen8<T, KV>(raw[j][i], x);
      else if constexpr (KV == kFp8) widen8<T, KV>(i ? make_uint4(raw[j][0].z, raw[j][0].w, 0, 0) : raw[j][0], x);
      else widen8<T, KV>(i ? make_uint4(raw[j][0].y, 0, 0, 0) : raw[j][0], x);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float2 v = make_float2(x[e], x[e + 1]);
        if constexpr (KV == kFp4) v = __fmul2_rn(v, make_float2(s, s));
        if (rounding == kExact) {
          v = __fmul2_rn(v, make_float2(unit, unit));
        } else if (bf16_values && rounding == kWide) {
          v = make_float2(to_odd((double)v.x * unit), to_odd((double)v.y * unit));
        } else {
          const float2 w = __fmul2_rz(v, make_float2(unit, unit));
          v = make_float2(sticky<KV>(w.x), sticky<KV>(w.y));
        }
        x[e] = v.x;
        x[e + 1] = v.y;
      }
      v16[i] = pack8<T>(x);
    }
    if (p.wide) {
      // whole sectors: two stores of 16 bytes would each write half of every sector
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + j * o1),
                   "r"(v16[0].x), "r"(v16[0].y), "r"(v16[0].z), "r"(v16[0].w), "r"(v16[1].x),
                   "r"(v16[1].y), "r"(v16[1].z), "r"(v16[1].w)
                   : "memory");
    } else {
      reinterpret_cast<uint4*>(dst + j * o1)[0] = v16[0];
      reinterpret_cast<uint4*>(dst + j * o1)[1] = v16[1];
    }
  }
}

template <typename T, int KV, int D, int R>
cudaError_t launch_r(const pkd_gather_args& a, cudaStream_t s) {
  constexpr int LANES = D / 16;
  GatherParams p;
  p.a = a;
  uint64_t bits = 0;  // of every address a row can start at, in bytes
  if (a.k_out) bits |= (uint64_t)a.k_out | (uint64_t)(2 * a.k_out_strides[0]) | (uint64_t)(2 * a.k_out_strides[1]);
  if (a.v_out) bits |= (uint64_t)a.v_out | (uint64_t)(2 * a.v_out_strides[0]) | (uint64_t)(2 * a.v_out_strides[1]);
  p.wide = (bits & 31) == 0;  // (those 345 MB take 62.7 us with two 16-byte stores a lane, 54.8 with one)
  constexpr bool bf16_values = KV == kSame16 && std::is_same<T, __nv_bfloat16>::value;
  p.rounding[0] = rounding_of(a.pool.k_scale, bf16_values);
  p.rounding[1] = rounding_of(a.pool.v_scale, bf16_values);
  p.hc = (a.pool.num_kv_heads + R - 1) / R;
  p.chunks = (uint32_t)(p.hc * ((a.k_out != nullptr) + (a.v_out != nullptr)));
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
