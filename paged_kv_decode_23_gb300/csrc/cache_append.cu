// cache_append.cu -- token rows into a paged cache, with the norm of each query and key head and
// the position rotation in the same pass (pkd_append).
//
// A row of one head is spread over head_dim / 8 lanes, eight values (16 bytes) each: the sum of
// squares is a shuffle tree over those lanes, the rotation partner of the half-split form is the
// value of another lane (one shuffle), that of the interleaved form is in the lane itself, and a
// block of the 4-bit cache is two lanes.  A group of lanes takes R heads of one token, R of them
// loaded before the first is used; cos and sin are read once for them.
//
// Codes.  A cache of 8 or 4 bits stores the code nearest to the exact quotient, so that neither
// the order of a sum nor the lanes' roundings can show in it.  t, the quotient in 32 bits, comes
// with a bound e on its error; where the codes of t - e and t + e agree (all but about one value
// in 1e5) that is the code.  Otherwise: a value that comes straight from the input (v; k without
// norm, outside the rotated dims) is exact, and an FMA against the border between the two codes
// settles it, ties included; a computed value sends its warp through the row once more in 64 bits.
//
// Bound: bytes.  Every input byte is read once and every output byte written once; see the
// figures at the launcher.
#include <type_traits>

#include "cache_rows.cuh"

namespace pkd {
namespace {

using namespace rows;

struct AppendParams {
  pkd_append_args a;
  int64_t token0;    // first token of this launch
  uint32_t items;    // (token, chunk of heads) pairs of this launch
  uint32_t chunks;   // chunks of a token
  int heads;         // Hq + 2 Hkv
  int page_log;
};

// Relative error bound of a computed value against the terms it is summed from: sums of squares
// over 256 values (12 roundings, halved by the root), rsqrt (2 ulp), two products, and the
// rotation's product and FMA stay below 16 units of 2^-24.
constexpr float kValueErr = 9.5367431640625e-07f;  // 2^-20
// ... and of a quotient against the value it is computed from (three roundings, doubled).
constexpr float kQuotErr = 4.76837158203125e-07f;  // 2^-21

constexpr int kThreads = 256;

__device__ __forceinline__ void load_weight8(const void* w, int f32, int gl, bool bf16, float (&out)[8]) {
  if (f32) {
    const float4* f = static_cast<const float4*>(w) + 2 * gl;
    const float4 a = __ldg(f), b = __ldg(f + 1);
    out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
    out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
  } else {
    const uint4 v = __ldg(static_cast<const uint4*>(w) + gl);
    if (bf16) unpack8<__nv_bfloat16>(v, out);
    else unpack8<__half>(v, out);
  }
}

struct Codes {
  uint32_t lo, hi;   // e4m3: eight bytes; e2m1: eight nibbles in lo
  uint32_t scale;    // e2m1: the block's scale byte
};

// The codes of a computed key row, in 64 bits throughout.  Called by whole warps; `src` null for
// lanes that have no such row.
template <typename T, int KV, int D>
__device__ __noinline__ Codes exact_codes(const T* src, const void* weight, int weight_f32,
                                          const float* cs, int rotary, int interleaved, double eps,
                                          float unit) {
  constexpr int LANES = D / 8;
  const int lane = threadIdx.x & 31, gl = lane & (LANES - 1);
  float xf[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (src) unpack8<T>(*(reinterpret_cast<const uint4*>(src) + gl), xf);
  double x[8];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = xf[i];
    ss += x[i] * x[i];
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) ss += __shfl_xor_sync(~0u, ss, o);
  if (weight != nullptr && src) {
    float w[8];
    load_weight8(weight, weight_f32, gl, std::is_same<T, __nv_bfloat16>::value, w);
    const double r = 1.0 / sqrt(ss / D + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  }
  if (rotary) {
    const int half = rotary / 2;
    const bool turned = 8 * gl < rotary && src != nullptr;
    if (interleaved) {
      if (turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double c = cs[4 * gl + i], s = cs[half + 4 * gl + i];
          const double u = x[2 * i], v = x[2 * i + 1];
          x[2 * i] = u * c - v * s;
          x[2 * i + 1] = v * c + u * s;
        }
      }
    } else {
      const bool first = 8 * gl < half;
      const int from = (lane - gl) + ((first ? gl + half / 8 : gl - half / 8) & (LANES - 1));
      const int i0 = first ? 8 * gl : 8 * gl - half;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double other = __shfl_sync(~0u, x[i], from);
        if (turned) {
          const double c = cs[i0 + i], s = cs[half + i0 + i];
          x[i] = first ? x[i] * c - other * s : x[i] * c + other * s;
        }
      }
    }
  }
  Codes out{0, 0, 0};
  double by = unit;
  if constexpr (KV == kFp4) {
    double top = 0.0;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top = fmax(top, fabs(x[i]));
      nan |= x[i] != x[i];
    }
    top = fmax(top, __shfl_xor_sync(~0u, top, 1));
    nan |= __shfl_xor_sync(~0u, (int)nan, 1) != 0;
    const float t = to_odd(top / (6.0 * unit));
    out.scale = nan ? 0x7fu : codes2<kFp8>(t, t) & 0xffu;
    by = (double)e4m3_value(out.scale) * unit;
    if (!(by > 0.0)) return out;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = to_odd(fabs(x[i]) / by);
    const uint32_t sign = x[i] < 0.0 ? 1u : 0u;
    if constexpr (KV == kFp8) {
      const uint32_t c = (codes2<kFp8>(t, t) & 0xffu) | sign << 7;
      if (i < 4) out.lo |= c << (8 * i);
      else out.hi |= c << (8 * (i - 4));
    } else {
      out.lo |= ((codes2<kFp4>(t, t) & 0xfu) | sign << 3) << (4 * i);
    }
  }
  return out;
}

// The codes of a row from its values y in 32 bits, each with the sum `err` of the terms it was
// computed from (unused where `exact`).  Whole warps; *doubt: some code needs exact_codes.
template <int KV>
__device__ __forceinline__ Codes quick_codes(const float (&y)[8], const float (&err)[8], bool exact,
                                             float unit, bool* doubt) {
  Codes out{0, 0, 0};
  float m = 1.f, inv = 1.f / unit;
  if constexpr (KV == kFp4) {
    float top = 0.f, off = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top = fmaxf(top, fabsf(y[i]));
      off = fmaxf(off, err[i]);
      nan |= y[i] != y[i];
    }
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
    off = fmaxf(off, __shfl_xor_sync(~0u, off, 1));
    nan |= __shfl_xor_sync(~0u, (int)nan, 1) != 0;
    const float t = top * (inv * 0.16666667f);
    const float e = t * kQuotErr + (exact ? 0.f : off * (inv * 0.16666667f) * kValueErr);
    out.scale = nan ? 0x7fu : nearest_code<kFp8>(top, t, e, 6.f, unit, exact, doubt);
    m = e4m3_value(out.scale);
    if (!(m > 0.f)) return out;  // a block of zeros (or a NaN's): all codes 0
    inv = 1.f / (m * unit);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(y[i]);
    const float t = a * inv;
    const float e = t * kQuotErr + (exact ? 0.f : err[i] * inv * kValueErr);
    const uint32_t c = nearest_code<KV>(a, t, e, m, unit, exact, doubt);
    const uint32_t sign = __float_as_uint(y[i]) >> 31;
    if constexpr (KV == kFp8) {
      if (i < 4) out.lo |= (c | sign << 7) << (8 * i);
      else out.hi |= (c | sign << 7) << (8 * (i - 4));
    } else {
      out.lo |= (c | sign << 3) << (4 * i);
    }
  }
  return out;
}

template <typename T, int KV, int D, int R>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LANES = D / 8;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const pkd_append_args& a = p.a;
  const int lane = threadIdx.x & 31, gl = lane & (LANES - 1);
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const bool in = item < p.items;
  const uint32_t tok = in ? item / p.chunks : 0;
  const int c0 = in ? (int)(item - tok * p.chunks) : 0;
  const int64_t t = p.token0 + tok;
  const int hq = a.num_qo_heads, hkv = a.pool.num_kv_heads;
  const int rotary = a.rotary_dim;

  const int b = in ? __ldg(a.batch_indices + t) : -1;
  const int pos = in ? __ldg(a.positions + t) : 0;
  const int rpos = rotary && a.rope_positions && in ? __ldg(a.rope_positions + t) : pos;
  const bool turnable = !rotary || (rpos >= 0 && rpos < a.cos_sin_rows);
  const bool live = b >= 0 && turnable;

  // this group's heads c0, c0 + chunks, ...: neighbouring groups read neighbouring rows
  const T* src[R];
  uint4 raw[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int r = c0 + j * (int)p.chunks;
    src[j] = nullptr;
    raw[j] = make_uint4(0, 0, 0, 0);
    if (live && r < p.heads) {
      if (r < hq) src[j] = static_cast<const T*>(a.q) + t * a.q_strides[0] + r * a.q_strides[1];
      else if (r < hq + hkv) src[j] = static_cast<const T*>(a.k) + t * a.k_strides[0] + (r - hq) * a.k_strides[1];
      else src[j] = static_cast<const T*>(a.v) + t * a.v_strides[0] + (r - hq - hkv) * a.v_strides[1];
      raw[j] = *(reinterpret_cast<const uint4*>(src[j]) + gl);
    }
  }
  Slot slot{0, 0, 0};
  if (live && c0 + (R - 1) * (int)p.chunks >= hq && hkv > 0) slot = find_slot(a.pool, p.page_log, b, pos);
  if (gl == 0 && a.status) {
    const uint32_t bits = (b >= 0 && !turnable ? PKD_STATUS_BAD_TOKEN : 0u) | slot.status;
    if (bits) atomicOr(a.status, bits);
  }
  float cs[8], sn[8];
  const int half = rotary / 2;
  const bool turned = live && 8 * gl < rotary;
  const bool first = 8 * gl < half;
  const float* cs_row = a.cos_sin + (turned || live ? (int64_t)rpos * rotary : 0);
  if (turned) {
    if (a.interleaved) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(cs_row + 4 * gl));
      const float4 s = __ldg(reinterpret_cast<const float4*>(cs_row + half + 4 * gl));
      cs[0] = cs[1] = c.x; cs[2] = cs[3] = c.y; cs[4] = cs[5] = c.z; cs[6] = cs[7] = c.w;
      sn[0] = sn[1] = s.x; sn[2] = sn[3] = s.y; sn[4] = sn[5] = s.z; sn[6] = sn[7] = s.w;
    } else {
      const int i0 = first ? 8 * gl : 8 * gl - half;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(cs_row + i0) + i);
        const float4 s = __ldg(reinterpret_cast<const float4*>(cs_row + half + i0) + i);
        cs[4 * i] = c.x; cs[4 * i + 1] = c.y; cs[4 * i + 2] = c.z; cs[4 * i + 3] = c.w;
        sn[4 * i] = s.x; sn[4 * i + 1] = s.y; sn[4 * i + 2] = s.z; sn[4 * i + 3] = s.w;
      }
    }
  }
  const int from = (lane - gl) + ((first ? gl + half / 8 : gl - half / 8) & (LANES - 1));

#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int r = c0 + j * (int)p.chunks;
    const bool is_v = r >= hq + hkv;
    const void* w = is_v ? nullptr : r < hq ? a.q_weight : a.k_weight;
    float y[8];
    unpack8<T>(raw[j], y);
    // ---- norm (both weights are given or one of them: the shuffles are the warp's)
    if (a.q_weight || a.k_weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) ss += __shfl_xor_sync(~0u, ss, o);
      if (w && src[j]) {
        float wv[8];
        load_weight8(w, a.weight_f32, gl, kBf16, wv);
        const float rn = rsqrtf(fmaf(ss, 1.f / D, (float)a.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * rn * wv[i];
      }
    }
    // ---- rotation
    float err[8];  // |terms| that a value is the sum of
#pragma unroll
    for (int i = 0; i < 8; ++i) err[i] = fabsf(y[i]);
    if (rotary) {
      float other[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) other[i] = a.interleaved ? y[i ^ 1] : __shfl_sync(~0u, y[i], from);
      if (turned && !is_v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool minus = a.interleaved ? (i & 1) == 0 : first;
          const float os = other[i] * (minus ? -sn[i] : sn[i]);
          err[i] = fabsf(y[i] * cs[i]) + fabsf(os);
          y[i] = fmaf(y[i], cs[i], os);
        }
      }
    }
    // ---- q out
    if (src[j] && r < hq) {
      T* dst = static_cast<T*>(a.q_out) + t * a.q_out_strides[0] + r * a.q_out_strides[1];
      *(reinterpret_cast<uint4*>(dst) + gl) = pack8<T>(y);
    }
    // ---- k and v into their slots
    const bool store = src[j] && r >= hq && slot.status == 0;
    const int head = is_v ? r - hq - hkv : r - hq;
    if constexpr (KV == kSame16) {
      if (store)
        *reinterpret_cast<uint4*>(row_addr<KV>(is_v ? a.pool.v : a.pool.k, a.pool.strides, slot, head, gl)) =
            pack8<T>(y);
    } else {
      if (__any_sync(~0u, store)) {
        const float unit = is_v ? a.pool.v_scale : a.pool.k_scale;
        const bool exact = is_v || (!w && !turned);
        bool doubt = false;
        Codes c = quick_codes<KV>(y, err, exact, unit, &doubt);
        if (__any_sync(~0u, doubt && store)) {
          const Codes e = exact_codes<T, KV, D>(store && !is_v ? src[j] : nullptr, w, a.weight_f32,
                                                cs_row, rotary, a.interleaved, a.eps, unit);
          if (!exact) c = e;
        }
        if (store) {
          char* dst = row_addr<KV>(is_v ? a.pool.v : a.pool.k, a.pool.strides, slot, head, gl);
          if constexpr (KV == kFp8) *reinterpret_cast<uint2*>(dst) = make_uint2(c.lo, c.hi);
          else *reinterpret_cast<uint32_t*>(dst) = c.lo;
          if (KV == kFp4 && (gl & 1) == 0)
            *scale_addr(is_v ? a.pool.v_scales : a.pool.k_scales, a.pool.scale_strides, slot, head, gl) =
                (uint8_t)c.scale;
        }
      }
    }
  }
}

template <typename T, int KV, int D, int R>
cudaError_t launch_r(const pkd_append_args& a, cudaStream_t s) {
  constexpr int LANES = D / 8;
  AppendParams p;
  p.a = a;
  p.heads = a.num_qo_heads + 2 * a.pool.num_kv_heads;
  p.chunks = (uint32_t)(p.heads + R - 1) / R;
  p.page_log = __builtin_ctz((unsigned)a.pool.page_size);
  const int64_t slab = (int64_t(1) << 30) / p.chunks;  // tokens a launch counts in 32 bits
  for (int64_t t0 = 0; t0 < a.num_tokens; t0 += slab) {
    const int64_t n = a.num_tokens - t0 < slab ? a.num_tokens - t0 : slab;
    p.token0 = t0;
    p.items = (uint32_t)(n * p.chunks);
    const unsigned grid = (p.items + kThreads / LANES - 1) / (kThreads / LANES);
    cudaError_t e = launch_pdl(append_kernel<T, KV, D, R>, p, grid, kThreads, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int KV, int D>
cudaError_t launch_d(const pkd_append_args& a, cudaStream_t s) {
  // Heads a lane group takes: one while the call leaves SMs idle (a decode step is latency), four
  // once there is work for every SM several times over.
  const int64_t rows = a.num_tokens * (a.num_qo_heads + 2 * (int64_t)a.pool.num_kv_heads);
  if (rows * (D / 8) >= 4 * 152 * 2048) return launch_r<T, KV, D, 4>(a, s);
  return launch_r<T, KV, D, 1>(a, s);
}

template <typename T, int KV>
cudaError_t launch_kv(const pkd_append_args& a, cudaStream_t s) {
  switch (a.pool.head_dim) {
    case 64: return launch_d<T, KV, 64>(a, s);
    case 128: return launch_d<T, KV, 128>(a, s);
    default: return launch_d<T, KV, 256>(a, s);
  }
}

template <typename T>
cudaError_t launch_t(const pkd_append_args& a, cudaStream_t s) {
  switch (a.pool.dtype) {
    case PKD_DTYPE_E4M3: return launch_kv<T, kFp8>(a, s);
    case PKD_DTYPE_E2M1: return launch_kv<T, kFp4>(a, s);
    default: return launch_kv<T, kSame16>(a, s);
  }
}

}  // namespace

cudaError_t launch_append(const pkd_append_args& a, cudaStream_t s) {
  return a.in_dtype == PKD_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<__half>(a, s);
}

}  // namespace pkd
