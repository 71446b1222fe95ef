// decode_e2m1_kernels.cuh -- batch decode attention over a paged KV cache held in 4 bits.
//
// What it computes: decode_kernels.cuh's task (one chunk of a row's tokens, one kv head, up to 8
// qo heads) on a cache whose K and V hold e2m1 values, two a byte (the first in the low half),
// with one e4m3 scale per 16 consecutive dims: x[d] = e2m1[d] * scale[d / 16].  Such a product
// has at most 6 significant bits and lies in [2^-10, 2688], so it is an fp16 value: both MMAs
// (S^T = K Q^T and O^T += V^T P^T, mma.m16n8k16, fp32 accumulators) take K and V exactly.  What is
// rounded before the epilogue is P, to fp16: 11 bits, and an absolute 2^-32 of the row's largest weight
// (P is held 2^kHeadroom above it, so that what lies far below a dominant key still counts in the
// numerator as it does in the sum, which is taken in 32 bits); and of a bf16 q what lies more than 2^27
// below its head's largest value (load_q_e2m1).  A second product with what P's rounding leaves took
// 48.8 us for 46.5, 122 for 110 and 72 for 60 (the last with 8 heads of 256, cap and window); the error
// of fp16 outputs against 64 bits was 2.1e-4 instead of 3.0e-4, of bf16 outputs 1.7e-3 in both.
//
// Structure as in decode_kernels.cuh (producer warp, mbarrier ring, consumer warps, split partials
// merged by the last chunk's CTA), with these differences:
//   * four consumer warps take two slices of 16 tokens of a tile each and make one softmax step of
//     them; more and smaller CTAs per SM (up to four) hide each other's waits;
//   * the codes come by TMA, one box per page that holds both its K and its V rows (a 5-D map with
//     K and V as an axis): the TMA unit takes some 65 cycles a request whatever its size, and a
//     page's K rows alone are 1 KiB at page size 16.  The producer's lanes copy the scales
//     (D/16 bytes a token: too short for a tensor-map box in every layout) by cp.async on the
//     same full barrier, and keep the ids of 32 pages in registers, loaded 32 pages ahead.
//     Tokens that are not attended, or whose page id is bad, get zero scales: whatever bits their
//     codes hold, their V rows are zeros (an e2m1 code is always finite), so no row needs masking
//     before P V;
//   * K: lane tig of a row reads 16 bytes (32 dims, two scale blocks) at once and feeds them to
//     eight k steps; the dims of a k step are spread over the four lanes, and q's fragments are
//     loaded in the same order (a dot product does not depend on the order of its terms);
//   * V: ldmatrix.trans moves 16-bit units, four dims of a token, and a cvt turns one byte into two
//     dims of ONE token, where an MMA wants pairs of tokens.  Instead of permuting every pair of
//     registers, the product is taken twice with P next to zeros: slots {2t, 2t+1} of an A row hold
//     dims d and d+1 of token t; B = (p, 0) gives O[d] and B = (0, p) gives O[d+1].  That costs
//     eight more MMAs per 16 tokens (head_dim 128) and saves 32 permutes.
//   * tasks of up to 4 qo heads: the eight columns of P^T are those heads twice, next to (p, 0) and to
//     (0, p), so that one MMA makes both products.
// Bound: instructions next to HBM.  A cvt per pair of values (head_dim 128: 64 per 16 tokens and
// warp) and the scales' products go through pipes of 2 warp instructions a cycle.  32 qo and 8 kv
// heads of 128, 4 contexts of 131,072 (604 MB, HND, fp16): 110 us, 5.5 TB/s, ALU pipe 55 %,
// tensor pipe 28 %; with the copies alone 94 us, with the arithmetic alone 99.  64 contexts of
// 512 to 4,096 (171 MB, NHD, bf16): 46 us, 3.7 TB/s, of which 7 us go into NHD's scale copies (8 bytes a token, each
// in a sector of its own; HND: 39.7 us).
#pragma once

#include <cfloat>

#include "decode_kernels.cuh"

namespace pkd {

// log2 of the weight of a row's largest key right after its maximum was taken; with kLazyMax on top of
// it a weight stays below 2^15, inside fp16.
constexpr float kHeadroom = 7.f;

// D: head_dim.  HEADS: qo heads of a task, 4 or 8.  SL: 16-token slices a consumer warp takes of each
// tile.  NW consumer warps and one producer warp; a tile is NW * SL * 16 tokens.
template <int D_, int HEADS_, int NW_, int SL_, int NSTAGES_>
struct E2m1Geom {
  static constexpr int D = D_, HEADS = HEADS_, NW = NW_, SL = SL_, NSTAGES = NSTAGES_;
  static constexpr int TS = NW * SL * 16;
  static constexpr int SLICE = NW * 16;  // tokens between a warp's slices
  static constexpr int NCONS = NW * 32;
  static constexpr int THREADS = NCONS + 32;
  static constexpr int ROW = D / 2;   // code bytes of a token: the width of a box and its swizzle
  static constexpr int SB = D / 16;   // scale bytes of a token
  static constexpr int TILE_BYTES = TS * ROW;
  static constexpr int SF_TILE = TS * SB;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES + 2 * SF_TILE;
  static constexpr int PIPE_BYTES = NSTAGES * STAGE_BYTES;
  static constexpr int EPI_BYTES = NW * (kSlotHeads * D + 2 * kSlotHeads) * 4;
  static constexpr int SMEM_BYTES = PIPE_BYTES + 1024;
  // O^T accumulators: [32-dim chunk] of rows (d, d + 2), and with 8 heads another for (d + 1, d + 3)
  static constexpr int ACC = HEADS == 4 ? D / 32 : D / 16;
  static_assert(HEADS == 4 || HEADS == 8, "");
  static_assert(STAGE_BYTES % 1024 == 0, "stages keep the swizzle's alignment");
  static_assert(EPI_BYTES <= PIPE_BYTES, "the epilogue's image fits in the pipeline stages");
  static_assert(TS >= 32 && TS <= 256 && (TS & (TS - 1)) == 0, "whole boxes, at most 32 pages of 8 slots");
};

namespace dev {

// The eight e2m1 codes of a word as four half2 (byte 0 first), exactly.
__device__ __forceinline__ void e2m1x8_to_half2x4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* map, int c0, int c1, int c2,
                                            int c3, int c4, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar),
      "l"(policy)
      : "memory");
}

// BYTES (4, 8 or 16) bytes to shared memory, zeros if !valid (the source is then not read).
template <int BYTES>
__device__ __forceinline__ void cp_async_zfill(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
                 "r"(n)
                 : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// One of the barrier's expected arrivals, made once all of this thread's earlier cp.async landed.
__device__ __forceinline__ void cp_async_mbar_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace dev

// Byte offset of 16-byte chunk c of row r in rows of ROW bytes, as the TMA unit's swizzle of that
// width stores it: 32 bytes: address bit 4 ^= bit 7; 64: bits 4-5 ^= bits 7-8; 128: bits 4-6 ^=
// bits 7-9.
template <int ROW>
__device__ __forceinline__ uint32_t e2m1_off(int r, int c) {
  if constexpr (ROW == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  if constexpr (ROW == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
}

// A stage holds its boxes one after the other, each as `br` K rows and then br V rows (a box is a
// page, or a piece of a page of SLICE tokens, so that slices lie at a fixed distance).  Row of token
// j's K; its V is br rows further.
__device__ __forceinline__ int e2m1_row(int j, int br) { return j + (j & -br); }

// Token (within 16) of row j of S^T.  Rows of 64 and 32 bytes: in order.  Rows of 128 bytes: the
// two rows that one phase of a K load reads must differ in bit 2 for their swizzled chunks to fall
// into different halves, so 0, 4, 1, 5, ...; ldmatrix then reads V's rows in the same order.
template <int D>
__device__ __forceinline__ int e2m1_tok(int j) {
  if constexpr (D == 256) return (j & 8) | ((j & 1) << 2) | ((j >> 1) & 3);
  return j;
}

// The ids of a task's pages, 32 at a time over the lanes, the next 32 under way: page ids would
// otherwise be a load that every tile's copies wait for.  The pages of a tile never straddle two
// windows (a tile holds a power of two of them, at most 32).
struct PageWindow {
  const int32_t* ids;  // the chunk's first page id
  int n;               // pages of the chunk
  int w;               // cur holds pages 32w .. 32w + 31
  int cur, nxt;
  __device__ __forceinline__ int load(int at) const { return at < n ? __ldg(ids + at) : 0; }
  __device__ __forceinline__ PageWindow(const DecodeParams& p, const BlockCoords& b, int first, int lane)
      : ids(p.indices + b.it.page_base + b.it.chunk_tok0 / p.page_size),
        n((b.it.tok_end - b.it.chunk_tok0 + p.page_size - 1) / p.page_size), w(first >> 5) {
    cur = load(32 * w + lane);
    nxt = load(32 * w + 32 + lane);
  }
  // moves to the window of page `at`, the current one or the next
  __device__ __forceinline__ void move(int at, int lane) {
    if ((at >> 5) != w) {
      ++w;
      cur = nxt;
      nxt = load(32 * w + 32 + lane);
    }
  }
  // the id of page `at` of this window; whole warps
  __device__ __forceinline__ int id(int at) const { return __shfl_sync(~0u, cur, at & 31); }
};

// ------------------------------------------------------------------------------ producer
template <class G>
__device__ __forceinline__ void produce_e2m1(const DecodeE2m1Params& p, const BlockCoords& b,
                                             uint32_t smem, uint32_t full0, uint32_t empty0,
                                             volatile int* abort_flag, int lane) {
  using namespace dev;
  constexpr int TS = G::TS, NSTAGES = G::NSTAGES;
  const int ps = p.page_size, ps_log = __ffs(ps) - 1;
  const int br = ps < G::SLICE ? ps : G::SLICE;  // rows of a box: a page, or a piece of one
  const int boxes = TS / br;
  const uint32_t tx_per_box = 2u * br * G::ROW;
  const uint64_t pol = policy_evict_first();
  const uint8_t* ksf = p.k_sf + b.kvh * p.sf_stride[2];
  const int64_t to_v = p.v_sf - p.k_sf;
  // pages of up to 32 slots put a lane's tokens into one slot, tile after tile
  const int64_t lane_slot = (int64_t)(lane & (ps - 1)) * p.sf_stride[1];
  if (lane == 0) prefetch_tmap(&p.tmap_k);
  PageWindow win(p, b, b.j0 * TS / ps, lane);
  int issued = 0, s = 0;
  uint32_t phase = 1;
  bool ok = true, bad_page = false;
  for (int i = 0; i < b.ntiles; ++i) {
    const int tile0 = (b.j0 + i) * TS;  // from the chunk's first token
    const int t0 = b.it.chunk_tok0 + tile0;
    const int bt0 = t0 + lane * br;
    const bool need = lane < boxes && bt0 < b.it.tok_end && bt0 + br > b.it.tok_begin;
    win.move(tile0 >> ps_log, lane);
    const int pid = win.id((tile0 + lane * br) >> ps_log);  // (lanes past the boxes: any page)
    const bool whole = t0 >= b.it.tok_begin && t0 + TS <= b.it.tok_end;
    const uint8_t* src[TS / 32];
    bool valid[TS / 32];
#pragma unroll
    for (int k = 0; k < TS / 32; ++k) {
      const int j = lane + 32 * k;
      const uint32_t id = (uint32_t)win.id((tile0 + j) >> ps_log);
      valid[k] = id < p.num_pages && (whole || (t0 + j >= b.it.tok_begin && t0 + j < b.it.tok_end));
      src[k] = ksf + (valid[k] ? id : 0u) * p.sf_stride[0] +
               (ps <= 32 ? lane_slot : (int64_t)((tile0 + j) & (ps - 1)) * p.sf_stride[1]);
    }
    if (i >= NSTAGES && !__all_sync(~0u, mbar_wait(empty0 + 8 * s, phase, abort_flag, p.wait_ns))) {
      ok = false;
      break;
    }
    bad_page |= need && (uint32_t)pid >= p.num_pages;
    const unsigned m = __ballot_sync(0xffffffffu, need);
    if (lane == 0) mbar_arrive_expect_tx(full0 + 8 * s, __popc(m) * tx_per_box);
    __syncwarp();
    const uint32_t stage = smem + s * G::STAGE_BYTES;
    if (need) {
      const int slot0 = bt0 & (ps - 1);
      const int c1 = p.hnd ? slot0 : b.kvh;
      const int c2 = p.hnd ? b.kvh : slot0;
      const uint32_t dst = stage + lane * 2 * br * G::ROW;
      tma_load_5d(dst, &p.tmap_k, 0, c1, c2, 0, pid, full0 + 8 * s, pol);
      if (p.kv_maps == 2) tma_load_5d(dst + br * G::ROW, &p.tmap_v, 0, c1, c2, 0, pid, full0 + 8 * s, pol);
    }
    const uint32_t sf = stage + 2 * G::TILE_BYTES + lane * G::SB;
#pragma unroll
    for (int k = 0; k < TS / 32; ++k) {
      cp_async_zfill<G::SB>(sf + k * 32 * G::SB, src[k], valid[k]);
      cp_async_zfill<G::SB>(sf + G::SF_TILE + k * 32 * G::SB, src[k] + to_v, valid[k]);
    }
    cp_async_mbar_arrive(full0 + 8 * s);
    issued = i + 1;
    if (++s == NSTAGES) {
      s = 0;
      phase ^= 1;
    }
  }
  // A page id outside the pool: reported, and read as zeros (the tensor map's bounds, and the
  // zero scales above).
  if (__any_sync(~0u, bad_page) && lane == 0) atomicOr(p.status, kStatusBadPage);
  if (!ok) {
    *abort_flag = 1;
    if (lane == 0) atomicOr(p.status, kStatusTimeout);
  }
  // As in produce(): the warp stays until its copies in flight have landed, with the full limit.
  if (lane == 0) {
    volatile int never = 0;
    for (int u = issued - NSTAGES < 0 ? 0 : issued - NSTAGES; u < issued; ++u)
      mbar_wait(full0 + 8 * (u % NSTAGES), (u / NSTAGES) & 1, &never);
  }
}

// ------------------------------------------------------------------------------ consumer
// First of the four consecutive dims that lane tig's k slots {2tig, 2tig+1, 2tig+8, 2tig+9} hold
// in k step kk: four k steps of 16 dims a lane at head_dim 64, else eight of 32 dims a lane in
// each 128-dim column block.
template <int D>
__device__ __forceinline__ int e2m1_k_dim(int kk, int tig) {
  if constexpr (D == 64) return 16 * tig + 4 * kk;
  return 128 * (kk >> 3) + 32 * tig + 4 * (kk & 7);
}

// The B fragments of Q^T in fp16.  A bf16 head is scaled by a power of two (exact) that puts its
// largest finite value into [2^13, 2^14), so that whatever its range no value that matters
// overflows or loses bits; qmul holds the powers to multiply back for this lane's two C columns
// (qo heads 2tig and 2tig + 1).
// With HEADS 4, columns 4-7 repeat columns 0-3.
template <typename TQ, int D, int HEADS>
__device__ __forceinline__ void load_q_e2m1(const DecodeParams& p, const BlockCoords& b, int lane,
                                            uint32_t (&qb)[D / 16][2], float (&qmul)[2]) {
  using namespace dev;
  const int g = (lane >> 2) & (HEADS - 1), tig = lane & 3;
  const bool live = g < b.gcnt;
  const TQ* qrow = reinterpret_cast<const TQ*>(p.q) +
                   ((size_t)b.it.req * p.num_qo_heads + b.g0 + (live ? g : 0)) * D;
  qmul[0] = qmul[1] = 1.f;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint2 v = *reinterpret_cast<const uint2*>(qrow + e2m1_k_dim<D>(kk, tig));
    qb[kk][0] = live ? v.x : 0u;
    qb[kk][1] = live ? v.y : 0u;
  }
  if constexpr (!std::is_same<TQ, __half>::value) {
    float amax = 0.f;
    auto see = [&](float x) { if (fabsf(x) < __int_as_float(0x7f800000)) amax = fmaxf(amax, fabsf(x)); };
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 f = unpack2<TQ>(qb[kk][h]);
        see(f.x);
        see(f.y);
      }
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
    const int qexp = amax > 0.f ? max(ilogbf(amax) - 13, -100) : 0;
    const float down = __int_as_float((127 - qexp) << 23), up = __int_as_float((127 + qexp) << 23);
    qmul[0] = __shfl_sync(~0u, up, 8 * tig);
    qmul[1] = __shfl_sync(~0u, up, 8 * tig + 4);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 f = unpack2<TQ>(qb[kk][h]);
        qb[kk][h] = pack2<__half>(f.x * down, f.y * down);
      }
  }
}

// c = a * b, without an accumulator to clear.
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// cap * tanh(x) in base-2 units.  Up to |x| = 1 Lambert's continued fraction for tanh, cut after
// five terms (off by less than 6e-8 of its value there); beyond, 1 - 2 / (e^(2x) + 1), which loses
// bits for small x alone.
__device__ __forceinline__ float soft_cap(float x, float cap_log2, bool any_large) {
  const float y = x * x;
  const float n = fmaf(y, y + 105.f, 945.f), d = fmaf(y, fmaf(15.f, y, 420.f), 945.f);
  float t = x * __fdividef(n, d);
  if (any_large) t = fabsf(x) > 1.f ? tanh_via_exp2(x) : t;
  return cap_log2 * t;
}

// x * (the low or the high half of s, on both halves).
__device__ __forceinline__ uint32_t scaled(uint32_t x, uint32_t s, bool high) {
  const __half2 v = *reinterpret_cast<const __half2*>(&x), f = *reinterpret_cast<const __half2*>(&s);
  const __half2 z = __hmul2(v, high ? __high2half2(f) : __low2half2(f));
  return *reinterpret_cast<const uint32_t*>(&z);
}

template <typename TQ, class G>
__device__ __forceinline__ void consume_e2m1(const DecodeE2m1Params& p, const BlockCoords& b,
                                             uint32_t smem, uint32_t full0, uint32_t empty0,
                                             volatile int* abort_flag, int warp, int lane,
                                             float (&m2)[2], float (&lsum)[2],
                                             float (&acc)[G::ACC][4]) {
  using namespace dev;
  constexpr int D = G::D, TS = G::TS, SL = G::SL, HEADS = G::HEADS;
  uint32_t qb[D / 16][2];
  float qmul[2];
  load_q_e2m1<TQ, D, HEADS>(p, b, lane, qb, qmul);
  const float scale_qk[2] = {p.scale_qk * qmul[0], p.scale_qk * qmul[1]};
  const float cap_log2 = p.cap_log2;
  const int g_row = lane >> 2, tig = lane & 3;
  const int br = p.page_size < G::SLICE ? p.page_size : G::SLICE;
  // tokens (within a 16-token slice) of this lane's two S^T rows
  const int tok_a = e2m1_tok<D>(g_row), tok_b = tok_a + 8;
  // ALiBi slopes of this lane's two C columns (dead columns read the last live head's)
  const float slope0 = alibi_slope<D>(p, b.g0 + min((2 * tig) & (HEADS - 1), b.gcnt - 1));
  const float slope1 = alibi_slope<D>(p, b.g0 + min((2 * tig + 1) & (HEADS - 1), b.gcnt - 1));
  // Offsets inside a stage, of the warp's first slice.  K: at head_dim 64 the lane's 8 bytes are
  // half of chunk tig / 2, else its 16 bytes are chunk tig (of each 64 bytes).
  constexpr int NCB = D / 128 + (D == 64);
  const int ja = warp * 16 + tok_a;
  uint32_t koff_a[NCB], koff_b[NCB];
#pragma unroll
  for (int cb = 0; cb < NCB; ++cb) {
    const int chunk = D == 64 ? tig >> 1 : 4 * cb + tig, in = D == 64 ? (tig & 1) * 8 : 0;
    koff_a[cb] = e2m1_off<G::ROW>(e2m1_row(ja, br), chunk) + in;
    koff_b[cb] = e2m1_off<G::ROW>(e2m1_row(ja + 8, br), chunk) + in;
  }
  const uint32_t ksf = 2 * G::TILE_BYTES + ja * G::SB + (D == 64 ? tig : 2 * tig);
  // V: ldmatrix row of this lane (matrices: S^T rows 0-7 and 8-15 of chunk c, then of chunk c + 1)
  const int vr = e2m1_row(warp * 16 + (lane & 8) + e2m1_tok<D>(lane & 7), br) + br, vc = lane >> 4;
  uint32_t voff[D / 64];
#pragma unroll
  for (int x = 0; x < D / 64; ++x) voff[x] = e2m1_off<G::ROW>(vr, 2 * x + vc);
  // scales of S^T rows 2tig and 2tig + 1 (and 8 further)
  const uint32_t vsf = 2 * G::TILE_BYTES + G::SF_TILE + (warp * 16 + e2m1_tok<D>(2 * tig)) * G::SB;
  constexpr int kOdd = (D == 256 ? 4 : 1) * G::SB;  // token of row 2tig + 1 against that of 2tig
  // bytes 0, 2 (or 1, 3) of two scale words: blocks 2ch + (g_row >= 4) of chunks ch = 0 .. 3
  const uint32_t sf_sel = g_row >= 4 ? 0x7531u : 0x6420u;
  // HEADS 4: columns 0-3 of B take P in the even slots, columns 4-7 in the odd ones
  const uint32_t p_sel0 = g_row < 4 ? 0x4410u : 0x1044u, p_sel1 = g_row < 4 ? 0x4432u : 0x3244u;
  constexpr uint32_t kSlice = 2 * G::SLICE * G::ROW;  // stage offset of a warp's next slice

  int s = 0;
  uint32_t phase = 0;
  for (int i = 0; i < b.ntiles; ++i) {
    const int t_w = b.it.chunk_tok0 + (b.j0 + i) * TS + warp * 16;  // first token of slice 0
    if (!__all_sync(~0u, mbar_wait(full0 + 8 * s, phase, abort_flag, p.wait_ns))) {
      *abort_flag = 1;  // warp-uniform: the warp leaves the loop together
      atomicOr(p.status, kStatusTimeout);
      break;
    }
    // attended tokens [lo, hi), counted from t_w
    const int lo = b.it.tok_begin - t_w, hi = b.it.tok_end - t_w;
    const uint32_t st = stage_after_wait(smem + s * G::STAGE_BYTES);
    bool work = hi > 0 && lo < 16;
#pragma unroll
    for (int h = 1; h < SL; ++h) work |= hi > h * G::SLICE && lo < h * G::SLICE + 16;
    if (work) {
      // ---- S^T = K * Q^T : rows = 16 tokens, cols = qo heads
      float c[SL][4];
#pragma unroll
      for (int h = 0; h < SL; ++h) {
        auto k_word = [&](int kk, uint32_t wa, uint32_t wb, uint32_t sa, uint32_t sb, bool high_a, bool high_b) {
          uint32_t x[4], y[4];
          e2m1x8_to_half2x4(wa, x);
          e2m1x8_to_half2x4(wb, y);
          const uint32_t a0[4] = {scaled(x[0], sa, high_a), scaled(y[0], sb, high_b),
                                  scaled(x[1], sa, high_a), scaled(y[1], sb, high_b)};
          if (kk == 0) mma_first(c[h], a0, qb[kk][0], qb[kk][1]);
          else mma_16816<__half>(c[h], a0, qb[kk][0], qb[kk][1]);
          const uint32_t a1[4] = {scaled(x[2], sa, high_a), scaled(y[2], sb, high_b),
                                  scaled(x[3], sa, high_a), scaled(y[3], sb, high_b)};
          mma_16816<__half>(c[h], a1, qb[kk + 1][0], qb[kk + 1][1]);
        };
        const uint32_t sth = st + h * kSlice, sfh = st + ksf + h * G::SLICE * G::SB;
        if constexpr (D == 64) {
          const uint2 wa = lds_v2(sth + koff_a[0]), wb = lds_v2(sth + koff_b[0]);
          const uint32_t sf = e4m3x2_to_half2((uint16_t)(lds_u8(sfh) | lds_u8(sfh + 8 * G::SB) << 8));
          k_word(0, wa.x, wb.x, sf, sf, false, true);
          k_word(2, wa.y, wb.y, sf, sf, false, true);
        } else {
#pragma unroll
          for (int cb = 0; cb < NCB; ++cb) {
            const uint4 wa = lds_v4(sth + koff_a[cb]), wb = lds_v4(sth + koff_b[cb]);
            const uint32_t fa = e4m3x2_to_half2((uint16_t)lds_u16(sfh + cb * 8));
            const uint32_t fb = e4m3x2_to_half2((uint16_t)lds_u16(sfh + 8 * G::SB + cb * 8));
            k_word(8 * cb, wa.x, wb.x, fa, fb, false, false);
            k_word(8 * cb + 2, wa.y, wb.y, fa, fb, false, false);
            k_word(8 * cb + 4, wa.z, wb.z, fa, fb, true, true);
            k_word(8 * cb + 6, wa.w, wb.w, fa, fb, true, true);
          }
        }
      }
      // ---- online softmax over the slices' tokens, per qo-head column (see consume_tc).  sc[e]:
      // rows g_row (e & 2 clear) and g_row + 8 of slice e / 4, column e & 1
      float sc[4 * SL];
#pragma unroll
      for (int e = 0; e < 4 * SL; ++e) sc[e] = c[e >> 2][e & 3] * scale_qk[e & 1];
      if (p.alibi) {
#pragma unroll
        for (int e = 0; e < 4 * SL; ++e) {
          const int t = ((e & 2) ? tok_b : tok_a) + (e >> 2) * G::SLICE;
          sc[e] += ((e & 1) ? slope1 : slope0) * (float)(t_w + t - b.it.q_pos);
        }
      }
      if (cap_log2 > 0.f) {
        float largest = 0.f;
#pragma unroll
        for (int e = 0; e < 4 * SL; ++e) largest = fmaxf(largest, fabsf(sc[e]));
        const bool any_large = __any_sync(~0u, largest > 1.f);
#pragma unroll
        for (int e = 0; e < 4 * SL; ++e) sc[e] = soft_cap(sc[e], cap_log2, any_large);
      }
      if (lo > 0 || hi < (SL - 1) * G::SLICE + 16) {
#pragma unroll
        for (int e = 0; e < 4 * SL; ++e) {
          const int t = ((e & 2) ? tok_b : tok_a) + (e >> 2) * G::SLICE;
          if (t < lo || t >= hi) sc[e] = kNegInf;
        }
      }
      float top[2] = {fmaxf(sc[0], sc[2]), fmaxf(sc[1], sc[3])};
#pragma unroll
      for (int h = 1; h < SL; ++h) {
        top[0] = fmaxf(top[0], fmaxf(sc[4 * h], sc[4 * h + 2]));
        top[1] = fmaxf(top[1], fmaxf(sc[4 * h + 1], sc[4 * h + 3]));
      }
      if (__any_sync(~0u, top[0] > m2[0] + (kHeadroom + kLazyMax) || top[1] > m2[1] + (kHeadroom + kLazyMax))) {
        float alpha[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mx = top[j];
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
          const float mnew = fmaxf(m2[j], mx - kHeadroom);
          alpha[j] = fast_exp2(m2[j] - mnew);
          lsum[j] *= alpha[j];
          m2[j] = mnew;
        }
        // (HEADS 4: columns 4-7 of O^T belong to the heads of columns 0-3, whose m2 they repeat)
#pragma unroll
        for (int mb = 0; mb < G::ACC; ++mb) {
          acc[mb][0] *= alpha[0];
          acc[mb][1] *= alpha[1];
          acc[mb][2] *= alpha[0];
          acc[mb][3] *= alpha[1];
        }
      }
#pragma unroll
      for (int e = 0; e < 4 * SL; ++e) sc[e] = fast_exp2(sc[e] - m2[e & 1]);
      // (a step's weights first: every addition to a large sum rounds small ones, and the same way)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float step = sc[j] + sc[j + 2];
#pragma unroll
        for (int h = 1; h < SL; ++h) step += sc[4 * h + j] + sc[4 * h + j + 2];
        lsum[j] += step;
      }
#pragma unroll
      for (int h = 0; h < SL; ++h) {
        // ---- P^T as B operands next to zeros, in fp16 (p <= 2^15, see kHeadroom): set 0 takes S^T
        // rows 2t (and 2t + 8), set 1 rows 2t + 1 (and 2t + 9)
        const uint32_t p0 = movmatrix_trans(pack2<__half>(sc[4 * h], sc[4 * h + 1]));
        const uint32_t p1 = movmatrix_trans(pack2<__half>(sc[4 * h + 2], sc[4 * h + 3]));
        uint32_t be[2][2], bo[2][2];
        if constexpr (HEADS == 4) {
          be[0][0] = prmt(p0, 0, p_sel0);
          be[0][1] = prmt(p1, 0, p_sel0);
          be[1][0] = prmt(p0, 0, p_sel1);
          be[1][1] = prmt(p1, 0, p_sel1);
        } else {
          be[0][0] = p0 & 0xffffu;
          be[0][1] = p1 & 0xffffu;
          be[1][0] = p0 >> 16;
          be[1][1] = p1 >> 16;
          bo[0][0] = p0 << 16;
          bo[0][1] = p1 << 16;
          bo[1][0] = p0 & 0xffff0000u;
          bo[1][1] = p1 & 0xffff0000u;
        }
        // ---- O^T += V^T * P^T, chunks ch of 32 dims: see stash_e2m1 for what acc holds.
        // sf[t4][x]: scales of rows 2tig, 2tig + 1, 2tig + 8, 2tig + 9 for chunks 2x and 2x + 1
        uint32_t sf[4][D / 64];
#pragma unroll
        for (int t4 = 0; t4 < 4; ++t4) {
          const uint32_t at = st + vsf + (t4 & 1) * kOdd + ((t4 >> 1) * 8 + h * G::SLICE) * G::SB;
          if constexpr (D == 64) {
            const uint32_t w = lds_u32(at);
            sf[t4][0] = e4m3x2_to_half2((uint16_t)prmt(w, w, sf_sel));
          } else if constexpr (D == 128) {
            const uint2 w = lds_v2(at);
            e4m3x4_to_half2x2(prmt(w.x, w.y, sf_sel), sf[t4][0], sf[t4][1]);
          } else {
            const uint4 w = lds_v4(at);
            e4m3x4_to_half2x2(prmt(w.x, w.y, sf_sel), sf[t4][0], sf[t4][1]);
            e4m3x4_to_half2x2(prmt(w.z, w.w, sf_sel), sf[t4][2], sf[t4][3]);
          }
        }
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {  // two chunks at a time
          uint32_t r[4];
          ldsm_x4_trans(st + h * kSlice + voff[x], r);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int ch = 2 * x + y;
            uint32_t u[4], w[4];  // dims {0, 1}, {2, 3} of the even row's token, then of the odd one's
            e2m1x8_to_half2x4(r[2 * y], u);
            e2m1x8_to_half2x4(r[2 * y + 1], w);
#pragma unroll
            for (int set = 0; set < 2; ++set) {
              const uint32_t a[4] = {scaled(u[2 * set], sf[set][x], y), scaled(u[2 * set + 1], sf[set][x], y),
                                     scaled(w[2 * set], sf[set + 2][x], y), scaled(w[2 * set + 1], sf[set + 2][x], y)};
              if constexpr (HEADS == 4) {
                mma_16816<__half>(acc[ch], a, be[set][0], be[set][1]);
              } else {
                mma_16816<__half>(acc[2 * ch], a, be[set][0], be[set][1]);
                mma_16816<__half>(acc[2 * ch + 1], a, bo[set][0], bo[set][1]);
              }
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * s);
    if (++s == G::NSTAGES) {
      s = 0;
      phase ^= 1;
    }
  }
}

// A consumer warp's state into its slot of the epilogue image.  Lane (row r, tig) holds of chunk ch
//   8 heads: heads 2tig, 2tig + 1; dims 32ch + 4r + {0, 2} in acc[2ch], {1, 3} in acc[2ch + 1];
//   4 heads: heads 2(tig % 2), + 1; dims 32ch + 4r + {0, 2} (tig < 2) or {1, 3} in acc[ch].
template <class G>
__device__ __forceinline__ void stash_e2m1(const EpiView<G::D>& e, int warp, int lane,
                                           float (&m2)[2], float (&lsum)[2],
                                           float (&acc)[G::ACC][4]) {
  constexpr int D = G::D;
  const int gr = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float l = lsum[j];
    l += __shfl_xor_sync(~0u, l, 4);
    l += __shfl_xor_sync(~0u, l, 8);
    l += __shfl_xor_sync(~0u, l, 16);
    if (gr == 0 && 2 * tig < G::HEADS) {
      e.m[warp * kSlotHeads + tig * 2 + j] = m2[j];
      e.l[warp * kSlotHeads + tig * 2 + j] = l;
    }
  }
  float* a = e.acc + warp * kSlotHeads * D + 4 * gr;
#pragma unroll
  for (int ch = 0; ch < D / 32; ++ch)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (G::HEADS == 8) {
        *reinterpret_cast<float4*>(a + (tig * 2 + j) * D + 32 * ch) =
            make_float4(acc[2 * ch][j], acc[2 * ch + 1][j], acc[2 * ch][j + 2], acc[2 * ch + 1][j + 2]);
      } else {
        float* d = a + ((tig & 1) * 2 + j) * D + 32 * ch + (tig >> 1);
        d[0] = acc[ch][j];
        d[2] = acc[ch][j + 2];
      }
    }
}

// ------------------------------------------------------------------------------ kernel
template <typename TQ, class G, int CTAS>
__global__ void __launch_bounds__(G::THREADS, CTAS)
    decode_e2m1_kernel(const __grid_constant__ DecodeE2m1Params p) {
  using namespace dev;
  constexpr int D = G::D, NSTAGES = G::NSTAGES;
  __shared__ __align__(8) uint64_t bars[2 * NSTAGES];
  __shared__ int abort_flag_s;
  __shared__ int merge_last_s;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem_p =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_u32(smem_p);
  const uint32_t full0 = smem_u32(&bars[0]);
  const uint32_t empty0 = smem_u32(&bars[NSTAGES]);
  volatile int* abort_flag = &abort_flag_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Programmatic dependent launch, as in decode_paged_kernel: the task list came with the plan's
  // upload, everything else is touched only after the previous kernel has finished.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (p.task_count != nullptr && (int)blockIdx.x >= *p.task_count) return;
  const BlockCoords b = task_coords<G::TS, G::HEADS>(p);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int s = 0; s < NSTAGES; ++s) {
      mbar_init(full0 + 8 * s, 1 + 32);  // the codes' TMA transactions, and every lane's scale copies
      mbar_init(empty0 + 8 * s, G::NW);
    }
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0)
    abort_flag_s = (*reinterpret_cast<volatile uint32_t*>(p.status) & kStatusTimeout) ? 1 : 0;
  __syncthreads();
  if (abort_flag_s) return;  // an earlier launch timed out: touch nothing

  if (warp == G::NW) {
    produce_e2m1<G>(p, b, smem, full0, empty0, abort_flag, lane);
    return;
  }
  const EpiView<D> epi(smem_p, G::NW);
  // (a finite start: 2^(-inf - m2) is then 0 for a row without an attended key, not NaN)
  float m2[2] = {-FLT_MAX, -FLT_MAX}, lsum[2] = {0.f, 0.f};
  float acc[G::ACC][4];
#pragma unroll
  for (int mb = 0; mb < G::ACC; ++mb) acc[mb][0] = acc[mb][1] = acc[mb][2] = acc[mb][3] = 0.f;
  consume_e2m1<TQ, G>(p, b, smem, full0, empty0, abort_flag, warp, lane, m2, lsum, acc);
  // every consumer is done with the stages; one shared decision whether any wait gave up
  if (named_bar_or(1, G::NCONS, *abort_flag != 0)) return;
  stash_e2m1<G>(epi, warp, lane, m2, lsum, acc);
  named_bar_sync(1, G::NCONS);
  store_task<TQ, D, G::NW>(p, b, epi, threadIdx.x);
  if (b.it.out_slot >= 0) merge_unit<TQ, D, G::NCONS>(p, b, threadIdx.x, &merge_last_s);
}

template <typename TQ, class G, int CTAS>
DecodeKernel make_decode_e2m1(int q_dtype) {
  DecodeKernel k;
  k.kind = kTensorCore;
  k.q_dtype = q_dtype;
  k.kv_dtype = kE2M1;
  k.head_dim = G::D;
  k.heads_per_cta = G::HEADS;
  k.fn = reinterpret_cast<const void*>(&decode_e2m1_kernel<TQ, G, CTAS>);
  k.threads = G::THREADS;
  k.smem_bytes = G::SMEM_BYTES;
  k.tile_tokens = G::TS;
  k.rope = 0;
  k.nstages = G::NSTAGES;
  k.max_ctas = CTAS;
  k.box_rows = G::SLICE;
  return k;
}

}  // namespace pkd
