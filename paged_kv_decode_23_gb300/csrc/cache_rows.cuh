// cache_rows.cuh -- device code shared by the kernels that write and read rows of a paged cache: a
// row of one head lies over head_dim / 16 lanes, two pieces of eight consecutive values a lane.
#pragma once

#include "cache_ops.cuh"
#include "pkd_device.cuh"

namespace pkd {
namespace rows {

using dev::pack2;
using dev::unpack2;

enum CacheKind { kSame16 = 0, kFp8 = 1, kFp4 = 2 };

// Bytes of eight values in a cache of kind KV.
template <int KV>
__host__ __device__ constexpr int bytes8() { return KV == kSame16 ? 16 : KV == kFp8 ? 8 : 4; }

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const float2 a = unpack2<T>(v.x), b = unpack2<T>(v.y), c = unpack2<T>(v.z), d = unpack2<T>(v.w);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]),
                    pack2<T>(x[6], x[7]));
}

// Where a token's rows live: the page id and the slot in it.
struct Slot {
  int64_t page;
  int slot;
  uint32_t status;  // 0, or the PKD_STATUS_* bit that says why there is none
};

// Bounds-checked walk of the page table; reads nothing outside indptr[0 .. batch] and
// indices[0 .. num_indices).
__device__ __forceinline__ Slot find_slot(const pkd_paged_pool& p, int page_log, int b, int pos) {
  Slot s{0, pos & ((1 << page_log) - 1), PKD_STATUS_BAD_TOKEN};
  if (b < 0 || b >= p.batch || pos < 0) return s;
  const int64_t first = __ldg(p.indptr + b), end = __ldg(p.indptr + b + 1);
  const int64_t at = first + (pos >> page_log);
  if (first < 0 || at >= end || at >= p.num_indices) return s;
  s.page = __ldg(p.indices + at);
  s.status = s.page >= 0 && s.page < p.num_pages ? 0u : PKD_STATUS_BAD_PAGE;
  return s;
}

// Address of dim d (a multiple of 8) of one head's row in the K or V pool ...
template <int KV>
__device__ __forceinline__ char* row_addr(void* base, const int64_t (&st)[3], const Slot& s, int head, int d) {
  constexpr int kUnit = KV == kSame16 ? 2 : 1;  // bytes a stride unit
  return static_cast<char*>(base) +
         (s.page * st[0] + (int64_t)s.slot * st[1] + (int64_t)head * st[2]) * kUnit + d / 8 * bytes8<KV>();
}
// ... and of the scale byte of its block of a 4-bit cache.
__device__ __forceinline__ uint8_t* scale_addr(void* base, const int64_t (&st)[3], const Slot& s, int head, int d) {
  return static_cast<uint8_t*>(base) + s.page * st[0] + (int64_t)s.slot * st[1] + (int64_t)head * st[2] + d / 16;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

// Codes of two values, nearest with ties to even, at most the type's largest, with their signs: of
// `lo` in the low half of the result, of `hi` above it (8 bits each in e4m3, 4 in e2m1).
template <int KV>
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  if constexpr (KV == kFp8) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    uint32_t r;
    asm("{\n\t.reg .b8 t, z;\n\tmov.b16 {z, t}, 0;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
        "mov.b32 %0, {t, z, z, z};\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
  }
}
// ... and of eight, in order: eight bytes, or eight nibbles in w.x.
template <int KV>
__device__ __forceinline__ uint2 codes8(const float (&v)[8]) {
  if constexpr (KV == kFp8) {
    return make_uint2(codes2<KV>(v[0], v[1]) | codes2<KV>(v[2], v[3]) << 16,
                      codes2<KV>(v[4], v[5]) | codes2<KV>(v[6], v[7]) << 16);
  } else {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return make_uint2(r, 0u);
  }
}
// A double as a float whose last bit is set if anything was cut off (rounding to odd): a further
// rounding to nearest, to a type of at most 22 bits, then gives what the double itself rounds to.
__device__ __forceinline__ float to_odd(double x) {
  const float f = __double2float_rz(x);
  return (double)f != x && f == f && fabsf(f) < __int_as_float(0x7f800000)
             ? __uint_as_float(__float_as_uint(f) | 1u)
             : f;
}

// a / d rounded to odd (as to_odd), for any a and normal d in [2^-64, 2^64].  The remainder of a
// correctly rounded quotient is a float; small values are scaled so that it stays in range.
__device__ __forceinline__ float odd_quotient(float a, float d) {
  const float q = __fdiv_rn(a, d), z = fabsf(a) < 1.f ? 0x1p64f : 1.f;
  const float r = fmaf(-(q * z), d, a * z);
  uint32_t bits = __float_as_uint(q);
  if (fabsf(q) < __int_as_float(0x7f800000) && r != 0.f) {  // truncated, the last bit set
    bits -= (__float_as_uint(r) ^ __float_as_uint(a)) >> 31;
    bits |= 1u;
  }
  return __uint_as_float(bits);
}

// 1 / x within one unit in the last place, for normal x.
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// a / (d + dl) rounded to odd, so that one more rounding to a type of few bits is that of the exact
// quotient, for two values: d + dl the exact divisor as a float and the rest it leaves, inv about 1 / d.
// One Newton step makes t faithful; the remainder then keeps its sign through its two FMAs.
__device__ __forceinline__ float2 odd_quotients(float a, float b, float d, float dl, float inv) {
  // (what passes 2^20 has no code left to decide on; min.NaN keeps a NaN, and an infinity out)
  auto clamp = [&](float v) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(v)), "f"(d * 0x1p20f));
    return r;
  };
  const float2 x = make_float2(clamp(a), clamp(b)), by = make_float2(inv, inv);
  const float2 nd = make_float2(-d, -d), ndl = make_float2(-dl, -dl);
  float2 t = __fmul2_rn(x, by);
  float2 r = __ffma2_rn(t, ndl, __ffma2_rn(t, nd, x));
  t = __ffma2_rn(r, by, t);
  r = __ffma2_rn(t, ndl, __ffma2_rn(t, nd, x));
  // truncated (one unit less where t is above the quotient), with what was cut off kept in the last bit
  auto odd = [](float t, float r, float sign) {
    uint32_t bits = __float_as_uint(t) + (uint32_t)(__float_as_int(r) >> 31);
    if (r != 0.f) bits |= 1u;
    return __uint_as_float(bits | (__float_as_uint(sign) & 0x80000000u));
  };
  return make_float2(odd(t.x, r.x, a), odd(t.y, r.y, b));
}

}  // namespace rows
}  // namespace pkd
