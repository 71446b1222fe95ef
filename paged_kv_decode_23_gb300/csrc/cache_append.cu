// cache_append.cu -- token rows into a paged cache, with the norm of each query and key head and
// the position rotation in the same pass (pkd_append).
//
// A row of one head is spread over a group of head_dim / 16 lanes, two pieces of eight values (16
// bytes) each: where pairs (i, i + rotary_dim / 2) turn, a lane holds both pieces of its pairs, else
// 16 values on end, so that no rotation needs another lane's values.  The sum of squares is a
// shuffle tree over the group; a block of the 4-bit cache is two pieces, wherever they are.  A warp
// takes one token's neighbouring heads, all q, all k or all v, up to R for each of its groups;
// weights, cosines and sines are read once for them, and all that depends on the token is the same
// in every lane, so that every shuffle is the whole warp's.  Warps stay for several items where a
// call has more than fit, the next item's rows under way while the current ones are worked on; into
// a 16-bit cache a warp's items are all of one chunk of heads, whose weights it keeps (65.2 -> 62.9 us
// for the prompts below; codes take the registers that this needs, and cost unlike q).
// Pairs of values go through the packed 32-bit FMA.
//
// Codes.  A cache of 8 or 4 bits stores the code nearest to the exact quotient, so that neither
// the order of a sum nor the lanes' roundings can show in it.  A value that comes straight from
// the input (v; k without norm, outside the rotated dims) is exact: its quotient is rounded to odd
// and that to the code.  Ties are common there, one value in eight with a scale of few bits.  A
// computed value's quotient t has an error bound e: where the codes of t - e and t + e agree (all
// but about one value in 1e5) that is the code, else that value is computed once more in 64 bits;
// so are the largest values of a block whose scale is in doubt.  (The 64-bit pipe is far too slow for
// whole rows.)
//
// Bound: every input byte is read once and every output byte written once.  A 16-bit cache comes
// near that: 8,190 tokens of 64 + 2 * 8 heads of 128, fp16, norm and rotation, 340 MB: 63 us, 5.4 TB/s.
// Into 8 or 4 bits no pipe is full: the same rows take 96 us into e4m3 (issue 0.57 per cycle and
// scheduler, ALU pipe 38 %) and 137 us into 4 bits (0.48, 30 %), 4,095 tokens of 16 + 2 * 2 heads of 256
// from bf16 into e4m3, 81 MB, 33 us (0.53, 44 %).  What bounds them is latency at 16 warps an SM: 128
// registers a thread are all that four CTAs leave, instances for codes spill (launch_d), and each
// instruction waits for its warp's last.  The instructions themselves are two conversions a computed
// value and the products rounded to odd of the others.  A decode step's call is latency: 3.5 us (4.8 us
// a replayed graph of one call).
#include <type_traits>

#include "cache_rows.cuh"

namespace pkd {
namespace {

using namespace rows;

struct AppendParams {
  pkd_append_args a;
  int64_t token0;     // first token of this launch
  uint32_t items;     // (token, chunk of heads) pairs of this launch, a warp each
  uint32_t warps;     // warps of this launch; warp i takes items i, i + warps, ...
  uint32_t parallel;  // 16-bit caches: tokens that lie between a warp's items
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

constexpr int kThreads = 128;
constexpr int kCtas = 4;  // per SM

// A 16-bit cache whose scales are not 1: every value is divided and rounded once.  Instances of their
// own, since the division's registers cost the others (8,190 tokens of the prompts above with scales of
// 1: 66.1 us where one instance does both, 62.9 in two; 108 us with other scales).
constexpr int kOver16 = kFp4 + 1;
template <int KV>
__host__ __device__ constexpr bool is16() { return KV == kSame16 || KV == kOver16; }

// The dims of a lane's two pieces, and where a piece's other half of its 16-value block is.
struct Place {
  int d[2];        // first dim of each piece
  bool turned;     // the lane's values are rotated
  bool split;      // ... as pairs (d[0] + i, d[1] + i)
  int lane[2];     // lane (of the warp) and piece that hold dims d[i] ^ 8 ..
  int piece[2];
};
template <int D>
__device__ __forceinline__ Place place_of(int lane, int rotary, int interleaved) {
  constexpr int LANES = D / 16;
  const int gl = lane & (LANES - 1), half = rotary / 2;
  Place p;
  p.turned = 16 * gl < rotary;
  p.split = p.turned && !interleaved;
  p.d[0] = p.split ? 8 * gl : 16 * gl;
  p.d[1] = p.split ? half + 8 * gl : 16 * gl + 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int o = p.d[i] ^ 8;
    const bool pair = !interleaved && o < rotary;
    p.lane[i] = (lane - gl) + (pair ? (o < half ? o : o - half) / 8 : o / 16);
    p.piece[i] = pair ? o >= half : (o >> 3) & 1;
  }
  return p;
}

// Eight weights as floats.
template <typename T>
__device__ __forceinline__ void load_weight8(const void* w, int f32, int d, float (&out)[8]) {
  if (f32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(w) + d);
    const float4 a = __ldg(f), b = __ldg(f + 1);
    out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
    out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
  } else {
    unpack8<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(w) + d)), out);
  }
}

struct Codes {
  uint2 c[2];         // of each piece: e4m3: eight bytes; e2m1: eight nibbles in x
  uint2 alt[2];       // quick_codes: where it differs from c the code is in doubt
  uint32_t scale[2];  // e2m1: the scale byte of the piece's block
};

// Mean square of z times a row, a power of 2; a, b: this lane's 16 values.  Whole warps.
template <typename T, int D>
__device__ __noinline__ float scaled_mean(uint4 a, uint4 b, float z) {
  float x[16], sum = 0.f;
  unpack8<T>(a, *reinterpret_cast<float(*)[8]>(x));
  unpack8<T>(b, *reinterpret_cast<float(*)[8]>(x + 8));
#pragma unroll
  for (int e = 0; e < 16; ++e) sum = fmaf(x[e] * z, x[e] * z, sum);
#pragma unroll
  for (int o = 1; o < D / 16; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
  return sum * (1.f / D);
}

// 1 / sqrt(mean(x^2) + eps) of a row in 64 bits; x: this lane's 16 values.  The squares of 16-bit
// values are exact in 32 bits and are summed with their rounding errors kept (Knuth's two-sum), so
// that the 64-bit pipe, 16 cycles an instruction, has only the root to do: one Newton step from
// the 32-bit root, good to 2^-42.  (bf16 rows of magnitudes whose squares would leave the 32-bit
// range are scaled by a power of 2 first.)  Whole warps.
template <typename T, int D>
__device__ __forceinline__ double exact_rnorm(const uint4 (&raw)[2], double eps) {
  constexpr int LANES = D / 16;
  float z = 1.f;
  if (std::is_same<T, __nv_bfloat16>::value) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[8];
      unpack8<T>(raw[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    z = top > 0x1p55f ? 0x1p-70f : top < 0x1p-45f ? 0x1p80f : 1.f;
  }
  float s = 0.f, low = 0.f;
  auto add = [&](float x) {
    const float t = s + x, b = t - s;
    low += (s - (t - b)) + (x - b);
    s = t;
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float x[8];
    unpack8<T>(raw[i], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) add((x[e] * z) * (x[e] * z));
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    const float os = __shfl_xor_sync(~0u, s, o), ol = __shfl_xor_sync(~0u, low, o);
    add(os);
    low += ol;
  }
  const double m = ((double)s + low) * (1.0 / D) / ((double)z * z) + eps;
  if (!(m > 0x1p-100 && m < 0x1p120)) return 1.0 / sqrt(m);
  const double r = rsqrtf((float)m);
  return r * (1.5 - 0.5 * m * r * r);
}

// One value (dim d) of a computed key row in 64 bits, over its divisor, rounded to odd.
template <typename T>
__device__ __noinline__ float exact_quotient(const T* src, const void* weight, int weight_f32, const float* cs,
                                             int rotary, int interleaved, double rn, int d, float m, float unit) {
  auto value = [&](int at) {
    double x = (double)(float)src[at];
    if (weight)
      x = x * rn * (double)(weight_f32 ? static_cast<const float*>(weight)[at] : (float)static_cast<const T*>(weight)[at]);
    return x;
  };
  double x = value(d);
  if (d < rotary) {
    const int half = rotary / 2, pair = interleaved ? d >> 1 : d < half ? d : d - half;
    const bool first = interleaved ? !(d & 1) : d < half;
    const double o = value(interleaved ? d ^ 1 : first ? d + half : d - half);
    const double c = cs[pair], s = cs[half + pair];
    x = first ? x * c - o * s : x * c + o * s;
  }
  return to_odd(x / ((double)m * unit));
}

// The codes of a row from its values y in 32 bits, each with the sum `err` of the terms it was
// computed from (unused where `exact`); inv about 1 / unit.  exact_at(rn, i, e, m): value e of piece
// i over m * unit, to odd, given rn = exact_norm().  Whole warps, whose lanes may differ in `exact`;
// *doubt: some code is in doubt (alt differs from c).
template <int KV, class Norm, class At>
__device__ __forceinline__ Codes quick_codes(const Place& pl, const float (&y)[2][8],
                                             const float (&err)[2][8], bool exact, bool all_exact,
                                             float unit, float inv, bool live, Norm exact_norm,
                                             At exact_at, bool* doubt) {
  Codes out;
  float d[2] = {unit, unit}, dl[2] = {0.f, 0.f}, inv2[2] = {inv, inv};  // divisors, what their rounding left
  if constexpr (KV == kFp4) {
    // largest magnitude of each block, by its bits: a NaN's are above all others
    uint32_t top[2] = {0, 0}, both[2];
    float off[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) top[i] = max(top[i], __float_as_uint(y[i][e]) & 0x7fffffffu);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t t0 = __shfl_sync(~0u, top[0], pl.lane[i]), t1 = __shfl_sync(~0u, top[1], pl.lane[i]);
      both[i] = max(top[i], pl.piece[i] ? t1 : t0);
    }
    if (!all_exact) {  // (the same in the whole warp)
      float mine[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) mine[i] = fmaxf(mine[i], exact ? 0.f : err[i][e]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float t0 = __shfl_sync(~0u, mine[0], pl.lane[i]), t1 = __shfl_sync(~0u, mine[1], pl.lane[i]);
        off[i] = fmaxf(mine[i], pl.piece[i] ? t1 : t0);
      }
    }
    bool unsure[2] = {false, false};
    const float six = 6.f * unit, six_l = fmaf(6.f, unit, -six), sixth = inv * 0.16666667f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = __uint_as_float(both[i]);
      if (exact) {
        const float t = odd_quotients(a, a, six, six_l, sixth).x;
        out.scale[i] = codes2<kFp8>(t, t) & 0xffu;
      } else {
        const float t = a * sixth, e = off[i] * sixth * (kValueErr + kQuotErr);
        const uint32_t c = codes2<kFp8>(t - e, t + e);
        out.scale[i] = c & 0xffu;
        unsure[i] = out.scale[i] != c >> 8;
      }
    }
    if (!all_exact && __any_sync(~0u, (unsure[0] || unsure[1]) && live)) {
      // the scale again, from the exact values of those that can be the block's largest
      const double rn = exact_norm();
      float best[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t which = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          which |= (uint32_t) !(fabsf(y[i][e]) + 2.f * off[i] * kValueErr < __uint_as_float(both[i])) << e;
        if (!unsure[i] || !live) which = 0;
        for (; which; which &= which - 1) best[i] = fmaxf(best[i], fabsf(exact_at(rn, i, __ffs(which) - 1, 6.f)));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float t0 = __shfl_sync(~0u, best[0], pl.lane[i]), t1 = __shfl_sync(~0u, best[1], pl.lane[i]);
        const float t = fmaxf(best[i], pl.piece[i] ? t1 : t0);
        if (unsure[i]) out.scale[i] = codes2<kFp8>(t, t) & 0xffu;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (both[i] > 0x7f800000u) out.scale[i] = 0x7fu;
      const float m = e4m3_value(out.scale[i]);
      // (a block of zeros, or a NaN's, gets codes 0 by a zero in place of 1 / 0)
      d[i] = m * unit;
      dl[i] = fmaf(m, unit, -d[i]);
      inv2[i] = m > 0.f ? rcp(d[i]) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (exact) {
      float t[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 q = odd_quotients(y[i][e], y[i][e + 1], d[i], dl[i], inv2[i]);
        t[e] = q.x;
        t[e + 1] = q.y;
      }
      out.c[i] = out.alt[i] = codes8<KV>(t);
    } else {
      float lo[8], hi[8];
      const float k = inv2[i] * (kValueErr + kQuotErr);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        // (+ 0: a negative zero, from a zero head and a negative weight, is no doubt)
        const float2 t = __ffma2_rn(make_float2(y[i][e], y[i][e + 1]), make_float2(inv2[i], inv2[i]), make_float2(0.f, 0.f));
        const float2 off = make_float2(err[i][e], err[i][e + 1]);
        const float2 l = __ffma2_rn(off, make_float2(-k, -k), t), h = __ffma2_rn(off, make_float2(k, k), t);
        lo[e] = l.x;
        lo[e + 1] = l.y;
        hi[e] = h.x;
        hi[e + 1] = h.y;
      }
      out.c[i] = codes8<KV>(lo);
      out.alt[i] = codes8<KV>(hi);
    }
    if (KV == kFp4 && inv2[i] == 0.f) out.c[i] = out.alt[i] = make_uint2(0, 0);
    *doubt |= out.c[i].x != out.alt[i].x || out.c[i].y != out.alt[i].y;
  }
  return out;
}

// What a warp works on, and what it has loaded of it.
template <typename T, int D, int R>
struct Item {
  int64_t t;       // token
  int kind;        // 0, 1, 2: q, k, v
  int first;       // first head; group g takes first + g, first + g + GROUPS, ...
  int b, pos, rpos;
  uint4 raw[R][2];

  __device__ __forceinline__ int heads(const pkd_append_args& a) const {
    return kind == 0 ? a.num_qo_heads : a.pool.num_kv_heads;
  }
  __device__ __forceinline__ Place place(const pkd_append_args& a, int lane) const {
    return place_of<D>(lane, kind == 2 ? 0 : a.rotary_dim, a.interleaved);
  }
  __device__ __forceinline__ int64_t step(const pkd_append_args& a) const {
    return kind == 0 ? a.q_strides[1] : kind == 1 ? a.k_strides[1] : a.v_strides[1];
  }
  __device__ __forceinline__ const T* row0(const pkd_append_args& a) const {
    const int64_t st = kind == 0 ? a.q_strides[0] : kind == 1 ? a.k_strides[0] : a.v_strides[0];
    return static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + t * st;
  }
  __device__ __forceinline__ const void* weight(const pkd_append_args& a) const {
    return kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
  }
  __device__ __forceinline__ void weights(const pkd_append_args& a, int lane, float (&wv)[2][8]) const {
    if (!weight(a)) return;
    const Place pl = place(a, lane);
    load_weight8<T>(weight(a), a.weight_f32, pl.d[0], wv[0]);
    load_weight8<T>(weight(a), a.weight_f32, pl.d[1], wv[1]);
  }
  __device__ __forceinline__ void aim(const AppendParams& p, int c) {
    constexpr int GROUPS = 32 / (D / 16);
    kind = c < p.qc ? 0 : c < p.qc + p.kc ? 1 : 2;
    first = (c - (kind == 0 ? 0 : kind == 1 ? p.qc : p.qc + p.kc)) * R * GROUPS;
  }
  __device__ __forceinline__ void load(const AppendParams& p, uint32_t token, int lane) {
    constexpr int GROUPS = 32 / (D / 16);
    const pkd_append_args& a = p.a;
    t = p.token0 + token;
    b = __ldg(a.batch_indices + t);
    pos = __ldg(a.positions + t);
    rpos = a.rotary_dim && a.rope_positions ? __ldg(a.rope_positions + t) : pos;
    const Place pl = place(a, lane);
    const int n = heads(a);
    const T* src = row0(a);
    const int64_t st = step(a);
#pragma unroll
    for (int j = 0; j < R; ++j) {  // (a padding row's values are read and dropped; no head: zeros)
      const int h = first + lane / (D / 16) + j * GROUPS;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        raw[j][i] = h < n ? *reinterpret_cast<const uint4*>(src + h * st + pl.d[i]) : make_uint4(0, 0, 0, 0);
    }
  }
};

template <typename T, int KV, int D, int R>
__device__ __forceinline__ void append_item(const AppendParams& p, const Item<T, D, R>& it,
                                            float (&wv)[2][8], int lane) {
  constexpr int LANES = D / 16, GROUPS = 32 / LANES;
  const pkd_append_args& a = p.a;
  const int kind = it.kind, first = it.first, heads = it.heads(a), rotary = a.rotary_dim, rpos = it.rpos;
  const int64_t t = it.t;
  const int h0 = first + lane / LANES;
  const Place pl = it.place(a, lane);
  const uint4 (&raw)[R][2] = it.raw;
  const void* w = it.weight(a);
  if (!is16<KV>()) it.weights(a, lane, wv);
  // cosines and sines: of the lane's eight pairs (piece 0 with piece 1), or of the four of each piece
  const bool turnable = !rotary || (rpos >= 0 && rpos < a.cos_sin_rows);
  const float* cs_row = rotary && turnable ? a.cos_sin + (int64_t)rpos * rotary : nullptr;
  float cs[8], sn[8];
  if (pl.turned && turnable) {
    const int half = rotary / 2;
    const int at0 = pl.split ? pl.d[0] : pl.d[0] / 2, at1 = pl.split ? pl.d[0] + 4 : pl.d[1] / 2;
    const float4 u0 = __ldg(reinterpret_cast<const float4*>(cs_row + at0));
    const float4 u1 = __ldg(reinterpret_cast<const float4*>(cs_row + at1));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(cs_row + half + at0));
    const float4 s1 = __ldg(reinterpret_cast<const float4*>(cs_row + half + at1));
    cs[0] = u0.x; cs[1] = u0.y; cs[2] = u0.z; cs[3] = u0.w;
    cs[4] = u1.x; cs[5] = u1.y; cs[6] = u1.z; cs[7] = u1.w;
    sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
    sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
  }
  // (what hangs on the batch index comes after the loads that do not)
  if (it.b < 0) return;
  if (!turnable) {
    if (lane == 0 && a.status) atomicOr(a.status, PKD_STATUS_BAD_TOKEN);
    return;
  }
  Slot slot{0, 0, 0};
  if (kind != 0) {
    slot = find_slot(a.pool, p.page_log, it.b, it.pos);
    if (slot.status) {
      if (lane == 0 && a.status) atomicOr(a.status, slot.status);
      return;
    }
  }
  const float unit = kind == 2 ? a.pool.v_scale : a.pool.k_scale, inv = kind == 2 ? p.v_inv : p.k_inv;

#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (first + j * GROUPS >= heads) break;  // the warp's last heads are done
    const int h = h0 + j * GROUPS;
    const bool live = h < heads;
    float y[2][8], err[2][8];  // err: |terms| that a value is the sum of
    unpack8<T>(raw[j][0], y[0]);
    unpack8<T>(raw[j][1], y[1]);
    // ---- norm
    if (w) {
      float2 ss[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int e = 0; e < 8; e += 2)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 v = make_float2(y[i][e], y[i][e + 1]);
          ss[i] = __ffma2_rn(v, v, ss[i]);
        }
      float sum = (ss[0].x + ss[0].y) + (ss[1].x + ss[1].y);
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
      float m = fmaf(sum, 1.f / D, p.eps);
      // bf16 has 32-bit floats' range: rows whose squares would leave it are scaled by a power of 2
      if (std::is_same<T, __nv_bfloat16>::value && __any_sync(~0u, !(m > 0x1p-100f && m < 0x1p120f))) {
        const float z = m > 0x1p-100f && m < 0x1p120f ? 1.f : m < 1.f ? 0x1p80f : 0x1p-70f;
        m = scaled_mean<T, D>(raw[j][0], raw[j][1], z) + p.eps * z * z;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][e] *= z;
      }
      const float rn = rsqrtf(m);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 v = __fmul2_rn(__fmul2_rn(make_float2(y[i][e], y[i][e + 1]), make_float2(rn, rn)),
                                      make_float2(wv[i][e], wv[i][e + 1]));
          y[i][e] = v.x;
          y[i][e + 1] = v.y;
        }
    }
    // ---- rotation
    if (!is16<KV>()) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) err[i][e] = fabsf(y[i][e]);
    }
    if (pl.turned) {
      if (pl.split) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 u = make_float2(y[0][e], y[0][e + 1]), v = make_float2(y[1][e], y[1][e + 1]);
          const float2 cc = make_float2(cs[e], cs[e + 1]), s = make_float2(sn[e], sn[e + 1]);
          const float2 vs = __fmul2_rn(v, make_float2(-s.x, -s.y)), us = __fmul2_rn(u, s);
          const float2 nu = __ffma2_rn(u, cc, vs), nv = __ffma2_rn(v, cc, us);
          if (!is16<KV>()) {
            err[0][e] = fabsf(u.x * cc.x) + fabsf(vs.x);
            err[0][e + 1] = fabsf(u.y * cc.y) + fabsf(vs.y);
            err[1][e] = fabsf(v.x * cc.x) + fabsf(us.x);
            err[1][e + 1] = fabsf(v.y * cc.y) + fabsf(us.y);
          }
          y[0][e] = nu.x;
          y[0][e + 1] = nu.y;
          y[1][e] = nv.x;
          y[1][e + 1] = nv.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = y[i][2 * e], v = y[i][2 * e + 1], cc = cs[4 * i + e], s = sn[4 * i + e];
            const float vs = v * -s, us = u * s;
            if (!is16<KV>()) {
              err[i][2 * e] = fabsf(u * cc) + fabsf(vs);
              err[i][2 * e + 1] = fabsf(v * cc) + fabsf(us);
            }
            y[i][2 * e] = fmaf(u, cc, vs);
            y[i][2 * e + 1] = fmaf(v, cc, us);
          }
      }
    }
    // ---- out
    if (kind == 0) {
      T* dst = static_cast<T*>(a.q_out) + t * a.q_out_strides[0] + h * a.q_out_strides[1];
      if (live) {
        *reinterpret_cast<uint4*>(dst + pl.d[0]) = pack8<T>(y[0]);
        *reinterpret_cast<uint4*>(dst + pl.d[1]) = pack8<T>(y[1]);
      }
      continue;
    }
    char* dst = row_addr<is16<KV>() ? kSame16 : KV>(kind == 2 ? a.pool.v : a.pool.k, a.pool.strides, slot, h, 0);
    if constexpr (is16<KV>()) {
      if (live) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (KV == kOver16) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] = odd_quotient(y[i][e], unit);
            *reinterpret_cast<uint4*>(dst + 2 * pl.d[i]) = pack8<T>(y[i]);
          } else {
            *reinterpret_cast<uint4*>(dst + 2 * pl.d[i]) = kind == 2 ? raw[j][i] : pack8<T>(y[i]);
          }
        }
      }
    } else {
      const bool exact = kind == 2 || (!w && !pl.turned);
      bool doubt = false;
      auto exact_norm = [&] { return w ? exact_rnorm<T, D>(raw[j], a.eps) : 1.0; };
      auto exact_at = [&](double rn, int i, int e, float m) {
        return exact_quotient<T>(it.row0(a) + h * it.step(a), w, a.weight_f32, cs_row, rotary, a.interleaved, rn,
                                 pl.d[i] + e, m, unit);
      };
      Codes cd = quick_codes<KV>(pl, y, err, exact, kind == 2, unit, inv, live, exact_norm, exact_at, &doubt);
      if (__any_sync(~0u, doubt && live)) {
        const double rn = exact_norm();
        if (live) {
          constexpr int kBits = KV == kFp8 ? 8 : 4;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float m = KV == kFp4 ? e4m3_value(cd.scale[i]) : 1.f;
            uint64_t code = cd.c[i].x | (uint64_t)cd.c[i].y << 32;
            uint64_t diff = code ^ (cd.alt[i].x | (uint64_t)cd.alt[i].y << 32);
            while (diff) {  // (one value, as a rule)
              const int e = (__ffsll(diff) - 1) / kBits;
              const uint64_t field = ((uint64_t(1) << kBits) - 1) << (e * kBits);
              const float x = exact_at(rn, i, e, m);
              code = (code & ~field) | ((uint64_t)codes2<KV>(x, x) << (e * kBits) & field);
              diff &= ~field;
            }
            cd.c[i] = make_uint2((uint32_t)code, (uint32_t)(code >> 32));
          }
        }
      }
      if (live) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (KV == kFp8) {
            *reinterpret_cast<uint2*>(dst + pl.d[i]) = cd.c[i];
          } else {
            *reinterpret_cast<uint32_t*>(dst + pl.d[i] / 2) = cd.c[i].x;
            if ((pl.d[i] & 8) == 0)
              scale_addr(kind == 2 ? a.pool.v_scales : a.pool.k_scales, a.pool.scale_strides, slot, h, 0)[pl.d[i] / 16] =
                  (uint8_t)cd.scale[i];
          }
        }
      }
    }
  }
}

template <typename T, int KV, int D, int R>
__global__ void __launch_bounds__(kThreads, kCtas) append_kernel(const __grid_constant__ AppendParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // whole warps, the next item's rows under way while the current one is worked on
  constexpr bool KEEP = is16<KV>();
  const int lane = threadIdx.x & 31;
  uint32_t item = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (item >= p.warps) return;
  Item<T, D, R> it, next;
  uint32_t token = item / p.chunks;
  it.aim(p, (int)(item - token * p.chunks));
  it.load(p, token, lane);
  float wv[2][8];
  if (KEEP) it.weights(p.a, lane, wv);
  while (true) {
    const bool more = item + p.warps < p.items && item + p.warps > item;
    item += p.warps;
    next.kind = it.kind;
    next.first = it.first;
    if (more) {
      if (KEEP) {
        token += p.parallel;
      } else {
        token = item / p.chunks;
        next.aim(p, (int)(item - token * p.chunks));
      }
      next.load(p, token, lane);
    }
    append_item<T, KV, D, R>(p, it, wv, lane);
    if (!more) break;
    it = next;
  }
}

template <typename T, int KV, int D, int R>
cudaError_t launch_r(const pkd_append_args& a, int sms, cudaStream_t s) {
  constexpr int PER = R * 32 / (D / 16);  // heads of a warp
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
    // as many warps as fit at once, and no more than there are items
    uint32_t room = (uint32_t)sms * kCtas * (kThreads / 32);
    if (is16<KV>()) room = (room < p.chunks ? 1 : room / p.chunks) * p.chunks;
    p.warps = p.items < room ? p.items : room;
    p.parallel = p.warps / p.chunks;
    const unsigned grid = (p.warps + kThreads / 32 - 1) / (kThreads / 32);
    cudaError_t e = launch_pdl(append_kernel<T, KV, D, R>, p, grid, kThreads, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int KV, int D>
cudaError_t launch_d(const pkd_append_args& a, int sms, cudaStream_t s) {
  // Heads a group takes: one while the call leaves SMs idle, two once there is work for every SM
  // several times over, which keeps more bytes under way.  One token of 32 + 2 * 8 heads of 128, a
  // replayed graph: 4.8 us with one, 5.5 with two.  Calls in a stream, with one and with two: the 8,190
  // tokens above 82.0 and 63.5 us, into e4m3 106 and 96, into 4 bits 153 and 137; the chunk above 32.5
  // and 32.9, into 4 bits 43.8 and 41.0; 8,192 tokens of 16 + 2 * 16 heads of 64 into 16, 8 and 4 bits
  // 28.5 and 23.2, 41.8 and 39.7, 58.9 and 56.4.  (Two heads' instances for codes spill: 64 to 72
  // bytes a thread into e4m3, 264 to 324 into 4 bits; one head's 0 and 128 to 136.)
  const int64_t rows = a.num_tokens * (a.num_qo_heads + 2 * (int64_t)a.pool.num_kv_heads);
  if (rows * (D / 8) >= (int64_t)8192 * sms) return launch_r<T, KV, D, 2>(a, sms, s);
  return launch_r<T, KV, D, 1>(a, sms, s);
}

template <typename T, int KV>
cudaError_t launch_kv(const pkd_append_args& a, int sms, cudaStream_t s) {
  switch (a.pool.head_dim) {
    case 64: return launch_d<T, KV, 64>(a, sms, s);
    case 128: return launch_d<T, KV, 128>(a, sms, s);
    default: return launch_d<T, KV, 256>(a, sms, s);
  }
}

template <typename T>
cudaError_t launch_t(const pkd_append_args& a, int sms, cudaStream_t s) {
  switch (a.pool.dtype) {
    case PKD_DTYPE_E4M3: return launch_kv<T, kFp8>(a, sms, s);
    case PKD_DTYPE_E2M1: return launch_kv<T, kFp4>(a, sms, s);
    default:
      if (a.pool.k_scale != 1.f || a.pool.v_scale != 1.f) return launch_kv<T, kOver16>(a, sms, s);
      return launch_kv<T, kSame16>(a, sms, s);
  }
}

}  // namespace

cudaError_t launch_append(const pkd_append_args& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return a.in_dtype == PKD_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, sms, s) : launch_t<__half>(a, sms, s);
}

}  // namespace pkd
