// cache_append.cu -- token rows into a paged cache, with the norm of each query and key head and
// the position rotation in the same pass (pkd_append).
//
// A row of one head is spread over a group of head_dim / 8 lanes, eight values (16 bytes) each: the
// sum of squares is a shuffle tree over the group, the rotation partner of the half-split form is
// the value of another lane (one shuffle), that of the interleaved form is in the lane itself, and
// a block of the 4-bit cache is two lanes.  A warp takes one token's neighbouring heads, all q, all
// k or all v, up to R for each of its groups, and loads them before it uses the first; weights,
// cosines and sines are read once for them, and all that depends on the token is the same in every
// lane, so that every shuffle is the whole warp's (one over a part of it costs four instructions
// more).  Pairs of values go through the packed 32-bit FMA.
//
// Codes.  A cache of 8 or 4 bits stores the code nearest to the exact quotient, so that neither
// the order of a sum nor the lanes' roundings can show in it.  A value that comes straight from
// the input (v; k without norm, outside the rotated dims) is exact: its quotient is rounded to odd
// and that to the code.  Ties are common there, one value in eight with a scale of few bits.  A
// computed value's quotient t has an error bound e: where the codes of t - e and t + e agree (all
// but about one value in 1e5) that is the code, else its warp goes through its rows once more in
// 64 bits.
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
  int64_t token0;     // first token of this launch
  uint32_t items;     // (token, chunk of heads) pairs of this launch, a warp each
  uint32_t chunks;    // chunks of a token: qc of q, kc of k, kc of v
  int qc, kc;
  int page_log;
  float eps;          // a.eps in 32 bits (a conversion per row would take the 64-bit pipe)
  float k_inv, v_inv;  // 1 / k_scale, 1 / v_scale
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

// The codes of a computed key row, in 64 bits throughout.  Called by whole warps.
template <typename T, int KV, int D>
__device__ __noinline__ Codes exact_codes(const T* src, const void* weight, int weight_f32,
                                          const float* cs, int rotary,
                                          int interleaved, double eps, float unit) {
  constexpr int LANES = D / 8;
  const int lane = threadIdx.x & 31, gl = lane & (LANES - 1);
  float xf[8];
  unpack8<T>(*(reinterpret_cast<const uint4*>(src) + gl), xf);
  double x[8];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = xf[i];
    ss += x[i] * x[i];
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) ss += __shfl_xor_sync(~0u, ss, o);
  if (weight != nullptr) {
    float w[8];
    load_weight8(weight, weight_f32, gl, std::is_same<T, __nv_bfloat16>::value, w);
    const double r = 1.0 / sqrt(ss / D + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  }
  if (rotary) {
    const int half = rotary / 2;
    const bool turned = 8 * gl < rotary;
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
// computed from (unused where `exact`); inv about 1 / unit.  Whole warps, whose lanes may differ in
// `exact`; *doubt: some code needs exact_codes.
template <int KV>
__device__ __forceinline__ Codes quick_codes(const float (&y)[8], const float (&err)[8],
                                             bool exact, float unit, float inv, bool* doubt) {
  Codes out{0, 0, 0};
  float d = unit, dl = 0.f;  // the divisor and what its rounding left
  if constexpr (KV == kFp4) {
    float top = 0.f, off = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top = fmaxf(top, fabsf(y[i]));
      nan |= y[i] != y[i];
      if (!exact) off = fmaxf(off, err[i]);
    }
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
    off = fmaxf(off, __shfl_xor_sync(~0u, off, 1));  // (lanes differ in exact)
    nan |= __shfl_xor_sync(~0u, (int)nan, 1) != 0;
    const float sixth = inv * 0.16666667f;
    if (exact) {
      const float six = 6.f * unit, t = odd_quotient(top, six, fmaf(6.f, unit, -six), sixth);
      out.scale = codes2<kFp8>(t, t) & 0xffu;
    } else {
      const float t = top * sixth, e = off * sixth * (kValueErr + kQuotErr);
      const uint32_t c = codes2<kFp8>(t - e, t + e);
      out.scale = c & 0xffu;
      *doubt = out.scale != c >> 8;
    }
    if (nan) out.scale = 0x7fu;
    const float m = e4m3_value(out.scale);
    if (!(m > 0.f)) return out;  // a block of zeros (or a NaN's): all codes 0
    d = m * unit;
    dl = fmaf(m, unit, -d);
    inv = rcp(d);
  }
  if (exact) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = odd_quotient(y[i], d, dl, inv);
    const uint2 c = codes8<KV>(t);
    out.lo = c.x;
    out.hi = c.y;
  } else {
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // (+ 0: a negative zero, from a zero head and a negative weight, is no doubt)
      const float t = fmaf(y[i], inv, 0.f), e = err[i] * inv * (kValueErr + kQuotErr);
      lo[i] = t - e;
      hi[i] = t + e;
    }
    const uint2 a = codes8<KV>(lo), b = codes8<KV>(hi);
    out.lo = a.x;
    out.hi = a.y;
    *doubt |= a.x != b.x || a.y != b.y;
  }
  return out;
}

template <typename T, int KV, int D, int R>
__global__ void __launch_bounds__(kThreads, KV == kSame16 ? 3 : 2) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LANES = D / 8;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const pkd_append_args& a = p.a;
  constexpr int GROUPS = 32 / LANES;
  const int lane = threadIdx.x & 31, gl = lane & (LANES - 1);
  const uint32_t item = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (item >= p.items) return;  // whole warps from here on, until their last row is stored
  const uint32_t tok = item / p.chunks;
  int c = (int)(item - tok * p.chunks);
  const int64_t t = p.token0 + tok;

  // this warp's heads [h0, heads) of q, k or v: its group g takes h0 + g, h0 + g + GROUPS, ...
  const int kind = c < p.qc ? 0 : c < p.qc + p.kc ? 1 : 2;
  c -= kind == 0 ? 0 : kind == 1 ? p.qc : p.qc + p.kc;
  const int heads = kind == 0 ? a.num_qo_heads : a.pool.num_kv_heads;
  const int h0 = c * R * GROUPS + lane / LANES;
  const int64_t st0 = kind == 0 ? a.q_strides[0] : kind == 1 ? a.k_strides[0] : a.v_strides[0];
  const int64_t st1 = kind == 0 ? a.q_strides[1] : kind == 1 ? a.k_strides[1] : a.v_strides[1];
  const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + t * st0;
  const int b = __ldg(a.batch_indices + t);
  const int pos = __ldg(a.positions + t);
  const int rotary = a.rotary_dim;
  const int rpos = rotary && a.rope_positions ? __ldg(a.rope_positions + t) : pos;
  uint4 raw[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {  // (a padding row's values are read and dropped; no head: zeros)
    const int h = h0 + j * GROUPS;
    raw[j] = h < heads ? *(reinterpret_cast<const uint4*>(src + h * st1) + gl) : make_uint4(0, 0, 0, 0);
  }
  if (b < 0) return;
  if (rotary && (rpos < 0 || rpos >= a.cos_sin_rows)) {
    if (lane == 0 && a.status) atomicOr(a.status, PKD_STATUS_BAD_TOKEN);
    return;
  }
  Slot slot{0, 0, 0};
  if (kind != 0) {
    slot = find_slot(a.pool, p.page_log, b, pos);
    if (slot.status) {
      if (lane == 0 && a.status) atomicOr(a.status, slot.status);
      return;
    }
  }
  const bool turned = kind != 2 && 8 * gl < rotary;
  const void* w = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
  const float unit = kind == 2 ? a.pool.v_scale : a.pool.k_scale, inv = kind == 2 ? p.v_inv : p.k_inv;
  const int half = rotary / 2;
  const bool first = 8 * gl < half;
  const float* cs_row = rotary ? a.cos_sin + (int64_t)rpos * rotary : nullptr;
  // cosines, and sines with the sign that this lane's values take their partners with
  float cs[8], sn[8], wv[8];
  if (turned) {
    if (a.interleaved) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(cs_row + 4 * gl));
      const float4 s = __ldg(reinterpret_cast<const float4*>(cs_row + half + 4 * gl));
      cs[0] = cs[1] = u.x; cs[2] = cs[3] = u.y; cs[4] = cs[5] = u.z; cs[6] = cs[7] = u.w;
      sn[1] = s.x; sn[3] = s.y; sn[5] = s.z; sn[7] = s.w;
      sn[0] = -s.x; sn[2] = -s.y; sn[4] = -s.z; sn[6] = -s.w;
    } else {
      const int i0 = first ? 8 * gl : 8 * gl - half;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(cs_row + i0) + i);
        const float4 s = __ldg(reinterpret_cast<const float4*>(cs_row + half + i0) + i);
        cs[4 * i] = u.x; cs[4 * i + 1] = u.y; cs[4 * i + 2] = u.z; cs[4 * i + 3] = u.w;
        sn[4 * i] = s.x; sn[4 * i + 1] = s.y; sn[4 * i + 2] = s.z; sn[4 * i + 3] = s.w;
      }
      if (first)
#pragma unroll
        for (int i = 0; i < 8; ++i) sn[i] = -sn[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  }
  if (w) load_weight8(w, a.weight_f32, gl, kBf16, wv);
  const int from = (lane - gl) + ((first ? gl + half / 8 : gl - half / 8) & (LANES - 1));

#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int h = h0 + j * GROUPS;
    if (h0 - lane / LANES + j * GROUPS >= heads) break;  // the warp's last heads are done
    const bool live = h < heads;
    float y[8], err[8];  // err: |terms| that a value is the sum of
    unpack8<T>(raw[j], y);
    // ---- norm
    if (w) {
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; i += 2) ss = __ffma2_rn(make_float2(y[i], y[i + 1]), make_float2(y[i], y[i + 1]), ss);
      float sum = ss.x + ss.y;
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
      const float rn = rsqrtf(fmaf(sum, 1.f / D, p.eps));
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 v = __fmul2_rn(__fmul2_rn(make_float2(y[i], y[i + 1]), make_float2(rn, rn)), make_float2(wv[i], wv[i + 1]));
        y[i] = v.x;
        y[i + 1] = v.y;
      }
    }
    // ---- rotation
    if (KV != kSame16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) err[i] = fabsf(y[i]);
    }
    if (rotary && kind != 2) {
      float other[8];
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = y[i ^ 1];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(~0u, y[i], from);
      }
      if (turned) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 os = __fmul2_rn(make_float2(other[i], other[i + 1]), make_float2(sn[i], sn[i + 1]));
          const float2 cc = make_float2(cs[i], cs[i + 1]);
          const float2 v = __ffma2_rn(make_float2(y[i], y[i + 1]), cc, os);
          if (KV != kSame16) {
            err[i] = fabsf(y[i] * cc.x) + fabsf(os.x);
            err[i + 1] = fabsf(y[i + 1] * cc.y) + fabsf(os.y);
          }
          y[i] = v.x;
          y[i + 1] = v.y;
        }
      }
    }
    // ---- out
    if (kind == 0) {
      T* dst = static_cast<T*>(a.q_out) + t * a.q_out_strides[0] + h * a.q_out_strides[1];
      if (live) *(reinterpret_cast<uint4*>(dst) + gl) = pack8<T>(y);
      continue;
    }
    char* dst = row_addr<KV>(kind == 2 ? a.pool.v : a.pool.k, a.pool.strides, slot, h, gl);
    if constexpr (KV == kSame16) {
      if (live) *reinterpret_cast<uint4*>(dst) = kind == 2 ? raw[j] : pack8<T>(y);
    } else {
      const bool exact = kind == 2 || (!w && !turned);
      bool doubt = false;
      Codes cd = quick_codes<KV>(y, err, exact, unit, inv, &doubt);
      if (__any_sync(~0u, doubt && live)) {
        // (a group without a head goes along on the warp's first one)
        const T* row = src + (live ? h : h0 - lane / LANES) * st1;
        const Codes e = exact_codes<T, KV, D>(row, w, a.weight_f32, cs_row, rotary, a.interleaved, a.eps, unit);
        if (!exact) cd = e;
      }
      if (live) {
        if constexpr (KV == kFp8) *reinterpret_cast<uint2*>(dst) = make_uint2(cd.lo, cd.hi);
        else *reinterpret_cast<uint32_t*>(dst) = cd.lo;
        if (KV == kFp4 && (gl & 1) == 0)
          *scale_addr(kind == 2 ? a.pool.v_scales : a.pool.k_scales, a.pool.scale_strides, slot, h, gl) =
              (uint8_t)cd.scale;
      }
    }
  }
}

template <typename T, int KV, int D, int R>
cudaError_t launch_r(const pkd_append_args& a, cudaStream_t s) {
  constexpr int PER = R * 32 / (D / 8);  // heads of a warp
  AppendParams p;
  p.a = a;
  p.eps = (float)a.eps;
  p.k_inv = 1.f / a.pool.k_scale;
  p.v_inv = 1.f / a.pool.v_scale;
  p.qc = (a.num_qo_heads + PER - 1) / PER;
  p.kc = (a.pool.num_kv_heads + PER - 1) / PER;
  p.chunks = (uint32_t)(p.qc + 2 * p.kc);
  p.page_log = a.pool.page_size > 0 ? __builtin_ctz((unsigned)a.pool.page_size) : 0;
  const int64_t slab = (int64_t(1) << 30) / p.chunks;  // tokens a launch counts in 32 bits
  for (int64_t t0 = 0; t0 < a.num_tokens; t0 += slab) {
    const int64_t n = a.num_tokens - t0 < slab ? a.num_tokens - t0 : slab;
    p.token0 = t0;
    p.items = (uint32_t)(n * p.chunks);
    const unsigned grid = (p.items + kThreads / 32 - 1) / (kThreads / 32);
    cudaError_t e = launch_pdl(append_kernel<T, KV, D, R>, p, grid, kThreads, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int KV, int D>
cudaError_t launch_d(const pkd_append_args& a, cudaStream_t s) {
  // Heads a group takes: one while the call leaves SMs idle (a decode step is latency), several
  // once there is work for every SM several times over.
  const int64_t rows = a.num_tokens * (a.num_qo_heads + 2 * (int64_t)a.pool.num_kv_heads);
  if (rows * (D / 8) >= 4 * 152 * 2048) return launch_r<T, KV, D, KV == kSame16 ? 4 : 2>(a, s);
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
