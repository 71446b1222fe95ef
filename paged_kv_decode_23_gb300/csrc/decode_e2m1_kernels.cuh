// decode_e2m1_kernels.cuh -- batch decode attention over a paged KV cache held in 4 bits.
//
// What it computes: decode_kernels.cuh's task (one chunk of a row's tokens, one kv head, up to 8
// qo heads) on a cache whose K and V hold e2m1 values, two a byte (the first in the low half),
// with one e4m3 scale per 16 consecutive dims: x[d] = e2m1[d] * scale[d / 16].  Such a product
// has at most 6 significant bits and lies in [2^-10, 2688], so it is an fp16 value: both MMAs
// (S^T = K Q^T and O^T += V^T P^T, mma.m16n8k16, fp32 accumulators) take exact operands and the
// only rounding before the epilogue is P's to fp16 (11 bits).
//
// Structure as in decode_kernels.cuh (producer warp, mbarrier ring, consumer warps of 16 tokens
// each, split partials merged by the last chunk's CTA), with these differences:
//   * the codes of a tile come by TMA, one box per (page, 64-byte column block, K|V), swizzled
//     so that both the K row reads and ldmatrix are free of bank conflicts;
//   * the scales (D/16 bytes a row: too short for a tensor-map box in every layout) come by
//     cp.async, one a token, on the same full barrier.  Tokens that are not attended, or whose
//     page id is bad, get zero scales: whatever bits their codes hold, their V rows are zeros
//     (an e2m1 code is always finite), so no row needs masking before P V;
//   * K: lane tig of a row reads 16 bytes (32 dims, two scale blocks) at once and feeds them to
//     eight k steps; the dims of a k step are spread over the four lanes, and q's fragments are
//     loaded in the same order (a dot product does not depend on the order of its terms);
//   * V: ldmatrix.trans moves 16-bit units, four dims of a token, so one register holds four
//     dims of two neighbouring tokens: exactly the token pairs of four V^T fragments.
// Bound: 144 bytes per token and kv head at head_dim 128 against 0.28 bytes per fp16 pair to
// widen: the widening (a cvt and a multiply per pair, one permute more for V) takes most of the
// issue slots that the bytes leave, see the figures at the registry.
#pragma once

#include "decode_kernels.cuh"

namespace pkd {

template <int D, int TS, int NSTAGES>
struct E2m1Geom {
  static constexpr int NW = TS / 16;
  static constexpr int NCONS = NW * 32;
  static constexpr int THREADS = NCONS + 32;
  static constexpr int ROW = D / 2;                  // code bytes of a token
  static constexpr int CB = ROW < 64 ? ROW : 64;     // bytes of a column block (TMA box width)
  static constexpr int NBLK = ROW / CB;
  static constexpr int SB = D / 16;                  // scale bytes of a token
  static constexpr int TILE_BYTES = TS * ROW;
  static constexpr int SF_TILE = TS * SB;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES + 2 * SF_TILE;
  static constexpr int PIPE_BYTES = NSTAGES * STAGE_BYTES;
  static constexpr int EPI_BYTES = NW * (kSlotHeads * D + 2 * kSlotHeads) * 4;
  static constexpr int SMEM_BYTES = PIPE_BYTES + 1024;
  static_assert(STAGE_BYTES % 1024 == 0, "stages keep the swizzle's alignment");
  static_assert(EPI_BYTES <= PIPE_BYTES, "the epilogue's image fits in the pipeline stages");
  static_assert(TS % 32 == 0 && NW <= 8, "a scale copy per lane and token; 16-token warp slices");
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

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t x, uint32_t y) {
  uint32_t z;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
  return z;
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
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

// One of the barrier's expected arrivals, made once all of this thread's earlier cp.async landed.
__device__ __forceinline__ void cp_async_mbar_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace dev

// Byte offset of 16-byte chunk c of row r inside a column block of CB bytes a row, as the TMA
// unit's 64-byte (32-byte) swizzle stores it: address bits 4-5 ^= bits 7-8 (bit 4 ^= bit 7).
template <int CB>
__device__ __forceinline__ uint32_t e2m1_off(int r, int c) {
  if constexpr (CB == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
}

// ------------------------------------------------------------------------------ producer
template <class G, int TS, int NSTAGES>
__device__ __forceinline__ void produce_e2m1(const DecodeE2m1Params& p, const BlockCoords& b,
                                             uint32_t smem, uint32_t full0, uint32_t empty0,
                                             volatile int* abort_flag, int lane) {
  using namespace dev;
  const int ps = p.page_size;
  const int br = ps < TS ? ps : TS;  // rows per box: a whole page, or a tile inside a page
  const int boxes = TS / br;
  const int br_log = __ffs(br) - 1;
  const uint32_t tx_per_box = 2u * G::NBLK * br * G::CB;
  const uint64_t pol = policy_evict_first();
  const uint8_t* ksf = p.k_sf + b.kvh * p.sf_stride[2];
  const uint8_t* vsf = p.v_sf + b.kvh * p.sf_stride[2];
  if (lane == 0) {
    prefetch_tmap(&p.tmap_k);
    prefetch_tmap(&p.tmap_v);
  }
  int issued = 0;
  bool ok = true, bad_page = false;
  for (int i = 0; i < b.ntiles; ++i) {
    const int s = i % NSTAGES;
    const int t0 = b.it.chunk_tok0 + (b.j0 + i) * TS;
    const int bt0 = t0 + lane * br;
    const bool need = lane < boxes && bt0 < b.it.tok_end && bt0 + br > b.it.tok_begin;
    int pid = 0;
    if (need) pid = __ldg(p.indices + b.it.page_base + bt0 / ps);
    if (i >= NSTAGES && !__all_sync(~0u, mbar_wait(empty0 + 8 * s, ((i / NSTAGES) - 1) & 1,
                                                   abort_flag, p.wait_ns))) {
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
      const uint32_t kdst = stage + lane * br * G::CB;
#pragma unroll
      for (int blk = 0; blk < G::NBLK; ++blk) {
        tma_load_4d(kdst + blk * TS * G::CB, &p.tmap_k, blk * G::CB, c1, c2, pid, full0 + 8 * s, pol);
        tma_load_4d(kdst + G::TILE_BYTES + blk * TS * G::CB, &p.tmap_v, blk * G::CB, c1, c2, pid,
                    full0 + 8 * s, pol);
      }
    }
    const uint32_t sf = stage + 2 * G::TILE_BYTES;
#pragma unroll
    for (int k = 0; k < TS / 32; ++k) {
      const int j = lane + 32 * k;
      const int t = t0 + j;
      const uint32_t tp = (uint32_t)__shfl_sync(~0u, pid, j >> br_log);
      const bool valid = t >= b.it.tok_begin && t < b.it.tok_end && tp < p.num_pages;
      const int64_t off =
          valid ? (int64_t)tp * p.sf_stride[0] + (int64_t)(t & (ps - 1)) * p.sf_stride[1] : 0;
      cp_async_zfill<G::SB>(sf + j * G::SB, ksf + off, valid);
      cp_async_zfill<G::SB>(sf + G::SF_TILE + j * G::SB, vsf + off, valid);
    }
    cp_async_mbar_arrive(full0 + 8 * s);
    issued = i + 1;
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
template <typename TQ, int D>
__device__ __forceinline__ void load_q_e2m1(const DecodeParams& p, const BlockCoords& b, int lane,
                                            uint32_t (&qb)[D / 16][2], float (&qmul)[2]) {
  using namespace dev;
  const int g = lane >> 2, tig = lane & 3;
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
    const float down = exp2f(static_cast<float>(-qexp)), up = exp2f(static_cast<float>(qexp));
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

template <typename TQ, int D, int TS, int NSTAGES>
__device__ __forceinline__ void consume_e2m1(const DecodeE2m1Params& p, const BlockCoords& b,
                                             uint32_t smem, uint32_t full0, uint32_t empty0,
                                             volatile int* abort_flag, int warp, int lane,
                                             float (&m2)[2], float (&lsum)[2],
                                             float (&acc)[D / 16][4]) {
  using namespace dev;
  using G = E2m1Geom<D, TS, NSTAGES>;
  uint32_t qb[D / 16][2];
  float qmul[2];
  load_q_e2m1<TQ, D>(p, b, lane, qb, qmul);
  const float scale_qk[2] = {p.scale_qk * qmul[0], p.scale_qk * qmul[1]};
  const float cap_log2 = p.cap_log2;
  const int g_row = lane >> 2, tig = lane & 3;
  const float slope0 = alibi_slope<D>(p, b.g0 + min(2 * tig, b.gcnt - 1));
  const float slope1 = alibi_slope<D>(p, b.g0 + min(2 * tig + 1, b.gcnt - 1));
  // Offsets inside a stage.  K: rows g_row and g_row + 8 of the warp's slice; at head_dim 64 the
  // lane's 8 bytes are half of chunk tig / 2, else its 16 bytes are chunk tig of a column block.
  const int ra = warp * 16 + g_row, rb = ra + 8;
  const uint32_t koff_a = D == 64 ? e2m1_off<G::CB>(ra, tig >> 1) + (tig & 1) * 8 : e2m1_off<G::CB>(ra, tig);
  const uint32_t koff_b = D == 64 ? e2m1_off<G::CB>(rb, tig >> 1) + (tig & 1) * 8 : e2m1_off<G::CB>(rb, tig);
  const uint32_t ksf_a = 2 * G::TILE_BYTES + ra * G::SB + (D == 64 ? tig : 2 * tig);
  const uint32_t ksf_b = ksf_a + 8 * G::SB;
  // V: ldmatrix row of this lane (matrices: tokens 0-7 and 8-15 of chunk c, then of chunk c + 1)
  const int vr = warp * 16 + (lane & 15), vc = lane >> 4;
  uint32_t voff[G::CB / 32];
#pragma unroll
  for (int c2 = 0; c2 < G::CB / 32; ++c2) voff[c2] = G::TILE_BYTES + e2m1_off<G::CB>(vr, 2 * c2 + vc);
  const uint32_t vsf0 = 2 * G::TILE_BYTES + G::SF_TILE + (warp * 16 + 2 * tig) * G::SB;
  // bytes of the two tokens' scale words: blocks 2ch + (g_row >= 4) of two chunks ch, ch + 1
  const uint32_t sf_sel = g_row >= 4 ? 0x7351u : 0x6240u;

  for (int i = 0; i < b.ntiles; ++i) {
    const int s = i % NSTAGES;
    const int t_w = b.it.chunk_tok0 + (b.j0 + i) * TS + warp * 16;  // first token of my slice
    if (!__all_sync(~0u, mbar_wait(full0 + 8 * s, (i / NSTAGES) & 1, abort_flag, p.wait_ns))) {
      *abort_flag = 1;  // warp-uniform: the warp leaves the loop together
      atomicOr(p.status, kStatusTimeout);
      break;
    }
    const int vlo = max(0, b.it.tok_begin - t_w);
    const int vhi = min(16, b.it.tok_end - t_w);
    const uint32_t st = stage_after_wait(smem + s * G::STAGE_BYTES);
    if (vhi > vlo) {
      // ---- S^T = K * Q^T : rows = 16 tokens, cols = 8 qo heads, two accumulators
      float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
      auto k_word = [&](int kk, uint32_t wa, uint32_t wb, uint32_t sa, uint32_t sb) {
        uint32_t x[4], y[4];
        e2m1x8_to_half2x4(wa, x);
        e2m1x8_to_half2x4(wb, y);
        uint32_t a0[4] = {hmul2_u32(x[0], sa), hmul2_u32(y[0], sb), hmul2_u32(x[1], sa), hmul2_u32(y[1], sb)};
        mma_16816<__half>(c, a0, qb[kk][0], qb[kk][1]);
        uint32_t a1[4] = {hmul2_u32(x[2], sa), hmul2_u32(y[2], sb), hmul2_u32(x[3], sa), hmul2_u32(y[3], sb)};
        mma_16816<__half>(c2, a1, qb[kk + 1][0], qb[kk + 1][1]);
      };
      if constexpr (D == 64) {
        const uint2 wa = lds_v2(st + koff_a), wb = lds_v2(st + koff_b);
        uint32_t lo, hi;
        uint32_t sf = 0;
        asm("ld.shared.u8 %0, [%1];" : "=r"(lo) : "r"(st + ksf_a));
        asm("ld.shared.u8 %0, [%1];" : "=r"(hi) : "r"(st + ksf_b));
        sf = e4m3x2_to_half2((uint16_t)(lo | (hi << 8)));
        const uint32_t sa = prmt(sf, sf, 0x1010), sb = prmt(sf, sf, 0x3232);
        k_word(0, wa.x, wb.x, sa, sb);
        k_word(2, wa.y, wb.y, sa, sb);
      } else {
#pragma unroll
        for (int cb = 0; cb < G::NBLK; ++cb) {
          const uint4 wa = lds_v4(st + koff_a + cb * TS * G::CB), wb = lds_v4(st + koff_b + cb * TS * G::CB);
          const uint32_t fa = e4m3x2_to_half2((uint16_t)lds_u16(st + ksf_a + cb * 8));
          const uint32_t fb = e4m3x2_to_half2((uint16_t)lds_u16(st + ksf_b + cb * 8));
          const uint32_t sa0 = prmt(fa, fa, 0x1010), sa1 = prmt(fa, fa, 0x3232);
          const uint32_t sb0 = prmt(fb, fb, 0x1010), sb1 = prmt(fb, fb, 0x3232);
          k_word(8 * cb, wa.x, wb.x, sa0, sb0);
          k_word(8 * cb + 2, wa.y, wb.y, sa0, sb0);
          k_word(8 * cb + 4, wa.z, wb.z, sa1, sb1);
          k_word(8 * cb + 6, wa.w, wb.w, sa1, sb1);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] += c2[e];
      // ---- online softmax over the 16 tokens, per qo-head column (see consume_tc)
      float sc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = e >= 2 ? g_row + 8 : g_row;
        const float bias = ((e & 1) ? slope1 : slope0) * (float)(t_w + t - b.it.q_pos);
        const float sv = score_log2(c[e], scale_qk[e & 1], bias, cap_log2);
        sc[e] = (t >= vlo && t < vhi) ? sv : kNegInf;
      }
      const bool grow = sc[0] > m2[0] + kLazyMax || sc[2] > m2[0] + kLazyMax ||
                        sc[1] > m2[1] + kLazyMax || sc[3] > m2[1] + kLazyMax;
      if (__any_sync(~0u, grow)) {
        float alpha[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mx = fmaxf(sc[j], sc[j + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
          const float mnew = fmaxf(m2[j], mx);
          const float ref = mnew == kNegInf ? 0.f : mnew;
          alpha[j] = fast_exp2(m2[j] - ref);
          sc[j] = fast_exp2(sc[j] - ref);
          sc[j + 2] = fast_exp2(sc[j + 2] - ref);
          lsum[j] = lsum[j] * alpha[j] + sc[j] + sc[j + 2];
          m2[j] = mnew;
        }
        if (__any_sync(~0u, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int mb = 0; mb < D / 16; ++mb) {
            acc[mb][0] *= alpha[0];
            acc[mb][1] *= alpha[1];
            acc[mb][2] *= alpha[0];
            acc[mb][3] *= alpha[1];
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float ref = m2[j] == kNegInf ? 0.f : m2[j];
          sc[j] = fast_exp2(sc[j] - ref);
          sc[j + 2] = fast_exp2(sc[j + 2] - ref);
          lsum[j] += sc[j] + sc[j + 2];
        }
      }
      // ---- P^T as the B operand, in fp16 (p <= 2^kLazyMax; 11 bits, see the header)
      const uint32_t b0 = movmatrix_trans(pack2<__half>(sc[0], sc[1]));
      const uint32_t b1 = movmatrix_trans(pack2<__half>(sc[2], sc[3]));
      // ---- O^T += V^T * P^T.  Chunk ch (32 dims): rows r and r + 8 of acc[2ch + m] hold dims
      // 32ch + 4r + 2m and 32ch + 4r + 2m + 1.
      uint32_t s01[D / 32], s89[D / 32];  // {scale of token 2tig (+8), of token 2tig + 1 (+9)}
      {
        const uint32_t a = st + vsf0;
        uint32_t w[4][D / 64];  // tokens 2tig, 2tig + 1, 2tig + 8, 2tig + 9
#pragma unroll
        for (int t4 = 0; t4 < 4; ++t4) {
          const uint32_t at = a + ((t4 & 1) + 8 * (t4 >> 1)) * G::SB;
          if constexpr (D == 64) w[t4][0] = lds_u32(at);
          else if constexpr (D == 128) { const uint2 v = lds_v2(at); w[t4][0] = v.x; w[t4][1] = v.y; }
          else { const uint4 v = lds_v4(at); w[t4][0] = v.x; w[t4][1] = v.y; w[t4][2] = v.z; w[t4][3] = v.w; }
        }
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          e4m3x4_to_half2x2(prmt(w[0][x], w[1][x], sf_sel), s01[2 * x], s01[2 * x + 1]);
          e4m3x4_to_half2x2(prmt(w[2][x], w[3][x], sf_sel), s89[2 * x], s89[2 * x + 1]);
        }
      }
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {  // two chunks at a time
        uint32_t r[4];
        ldsm_x4_trans(st + voff[x % (G::CB / 32)] + (x / (G::CB / 32)) * TS * G::CB, r);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int ch = 2 * x + y;
          uint32_t u[4], w[4];  // dims {0, 1} and {2, 3} of the even token, then of the odd one
          e2m1x8_to_half2x4(r[2 * y], u);
          e2m1x8_to_half2x4(r[2 * y + 1], w);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint32_t a[4] = {hmul2_u32(prmt(u[m], u[m + 2], 0x5410), s01[ch]),
                             hmul2_u32(prmt(u[m], u[m + 2], 0x7632), s01[ch]),
                             hmul2_u32(prmt(w[m], w[m + 2], 0x5410), s89[ch]),
                             hmul2_u32(prmt(w[m], w[m + 2], 0x7632), s89[ch])};
            mma_16816<__half>(acc[2 * ch + m], a, b0, b1);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * s);
  }
}

// A consumer warp's state into its slot of the epilogue image.
template <int D>
__device__ __forceinline__ void stash_e2m1(const EpiView<D>& e, int warp, int lane, float (&m2)[2],
                                           float (&lsum)[2], float (&acc)[D / 16][4]) {
  const int gr = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float l = lsum[j];
    l += __shfl_xor_sync(~0u, l, 4);
    l += __shfl_xor_sync(~0u, l, 8);
    l += __shfl_xor_sync(~0u, l, 16);
    if (gr == 0) {
      e.m[warp * kSlotHeads + tig * 2 + j] = m2[j];
      e.l[warp * kSlotHeads + tig * 2 + j] = l;
    }
  }
  float* a = e.acc + warp * kSlotHeads * D + 4 * gr;
#pragma unroll
  for (int ch = 0; ch < D / 32; ++ch)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<float4*>(a + (tig * 2 + j) * D + 32 * ch) =
          make_float4(acc[2 * ch][j], acc[2 * ch][j + 2], acc[2 * ch + 1][j], acc[2 * ch + 1][j + 2]);
}

// ------------------------------------------------------------------------------ kernel
template <typename TQ, int D, int TS, int NSTAGES>
__global__ void __launch_bounds__(E2m1Geom<D, TS, NSTAGES>::THREADS, 2)
    decode_e2m1_kernel(const __grid_constant__ DecodeE2m1Params p) {
  using namespace dev;
  using G = E2m1Geom<D, TS, NSTAGES>;
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
  const BlockCoords b = task_coords<TS, 8>(p);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int s = 0; s < NSTAGES; ++s) {
      mbar_init(full0 + 8 * s, 1 + 32);  // the TMA transactions, and every lane's scale copies
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
    produce_e2m1<G, TS, NSTAGES>(p, b, smem, full0, empty0, abort_flag, lane);
    return;
  }
  const EpiView<D> epi(smem_p, G::NW);
  float m2[2] = {kNegInf, kNegInf}, lsum[2] = {0.f, 0.f};
  float acc[D / 16][4];
#pragma unroll
  for (int mb = 0; mb < D / 16; ++mb) acc[mb][0] = acc[mb][1] = acc[mb][2] = acc[mb][3] = 0.f;
  consume_e2m1<TQ, D, TS, NSTAGES>(p, b, smem, full0, empty0, abort_flag, warp, lane, m2, lsum, acc);
  // every consumer is done with the stages; one shared decision whether any wait gave up
  if (named_bar_or(1, G::NCONS, *abort_flag != 0)) return;
  stash_e2m1<D>(epi, warp, lane, m2, lsum, acc);
  named_bar_sync(1, G::NCONS);
  store_task<TQ, D, G::NW>(p, b, epi, threadIdx.x);
  if (b.it.out_slot >= 0) merge_unit<TQ, D, G::NCONS>(p, b, threadIdx.x, &merge_last_s);
}

template <typename TQ, int D, int TS, int NSTAGES>
DecodeKernel make_decode_e2m1(int q_dtype) {
  using G = E2m1Geom<D, TS, NSTAGES>;
  DecodeKernel k;
  k.kind = kTensorCore;
  k.q_dtype = q_dtype;
  k.kv_dtype = kE2M1;
  k.head_dim = D;
  k.heads_per_cta = 8;
  k.fn = reinterpret_cast<const void*>(&decode_e2m1_kernel<TQ, D, TS, NSTAGES>);
  k.threads = G::THREADS;
  k.smem_bytes = G::SMEM_BYTES;
  k.tile_tokens = TS;
  k.rope = 0;
  k.nstages = NSTAGES;
  return k;
}

}  // namespace pkd
