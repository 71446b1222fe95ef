// cache_evict.cu -- cut each sequence of a paged cache back to a budget of tokens, in place: its first
// tokens (sinks), its newest and the heaviest of the others stay, by sums of attention weights per key
// and kv head.
//
// For n > B tokens, S sinks and R newest, m = B - S - R of the candidates [S, n - R) are chosen: the
// largest weights, equal ones by slot.  Every kv head chooses for itself.  Slots then hold:
//   [0, S)      the sinks, where they were;
//   [S, B - R)  the chosen, those among them that lie there already where they were; the i-th slot
//               left free takes the i-th chosen of [B - R, n - R) (as many as there are free slots);
//   [B - R, B)  the newest, in order.
// So no row moves that need not, and what moves is read and written once.  A row that moves into
// [S, B - R) overwrites nothing that is read; the newest are shifted down after those rows are read,
// tile by tile in ascending order (their sources lie above every earlier tile's destinations).
#include "cache_rows.cuh"

namespace pkd {

namespace {

using rows::find_slot;
using rows::Slot;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;  // of an 11-bit digit

// Order of weights as unsigned numbers: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct EvictParams {
  pkd_evict_args a;
  int page_log;
  int pieces;  // 16-byte pieces of a K (or V) row
  int words;   // 4-byte words of its scales
};

// One (sequence, kv head): where its rows lie.
struct Lane {
  const EvictParams& p;
  const int32_t* ids;  // the sequence's page ids
  int head;
  __device__ __forceinline__ int64_t page(int t) const { return __ldg(ids + (t >> p.page_log)); }
  __device__ __forceinline__ int slot(int t) const { return t & ((1 << p.page_log) - 1); }
  __device__ __forceinline__ float* weight(int t) const {
    const int64_t* st = p.a.weight_strides;
    return p.a.key_weights + page(t) * st[0] + head * st[1] + slot(t) * st[2];
  }
  // 16-byte piece q of token t's K row (q < pieces) or V row
  __device__ __forceinline__ uint4* piece(int t, int q, int elt) const {
    const pkd_paged_pool& c = p.a.pool;
    const int64_t at = (page(t) * c.strides[0] + slot(t) * c.strides[1] + head * c.strides[2]) * elt;
    const bool v = q >= p.pieces;
    return reinterpret_cast<uint4*>(static_cast<char*>(v ? c.v : c.k) + at) + (v ? q - p.pieces : q);
  }
  // word q of token t's K scales (q < words), V scales (q < 2 words) or its weight (q = 2 words)
  __device__ __forceinline__ uint32_t* word(int t, int q) const {
    if (q == 2 * p.words) return reinterpret_cast<uint32_t*>(weight(t));
    const pkd_paged_pool& c = p.a.pool;
    const int64_t at = page(t) * c.scale_strides[0] + slot(t) * c.scale_strides[1] + head * c.scale_strides[2];
    const bool v = q >= p.words;
    return reinterpret_cast<uint32_t*>(static_cast<char*>(v ? c.v_scales : c.k_scales) + at) + (v ? q - p.words : q);
  }
};

// Exclusive prefix of `mine` over the block's threads, and the sum; `part` holds kWarps + 1 ints.
__device__ __forceinline__ int block_prefix(int mine, int* part, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // (part may still be read from the call before)
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  return before + x - mine;
}

template <int ELT>
__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int hist[kBins];
  __shared__ int part[kWarps];
  __shared__ int found[2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const pkd_evict_args& a = p.a;
  const int hkv = a.pool.num_kv_heads;
  const int seq = blockIdx.x / hkv, tid = threadIdx.x;
  const int B = a.budget, S = a.num_sink_tokens, R = a.num_recent, m = B - S - R;
  const int n = __ldg(a.kv_lens + seq);
  int32_t* kept = a.kept ? a.kept + (int64_t)blockIdx.x * B : nullptr;
  const int64_t first = __ldg(a.pool.indptr + seq), end = __ldg(a.pool.indptr + seq + 1);
  const int64_t pages = ((int64_t)n + (1 << p.page_log) - 1) >> p.page_log;
  uint32_t bad = n < 0 || (n > 0 && (first < 0 || first + pages > end || first + pages > a.pool.num_indices))
                     ? PKD_STATUS_BAD_TOKEN : 0u;
  const Lane at{p, a.pool.indices + first, (int)(blockIdx.x % hkv)};
  if (!bad && n > B) {
    bool off = false;
    for (int64_t i = tid; i < pages; i += kThreads) {
      const int64_t id = __ldg(at.ids + i);
      off |= id < 0 || id >= a.pool.num_pages;
    }
    if (__syncthreads_or(off)) bad = PKD_STATUS_BAD_PAGE;
  }
  if (bad && a.status && tid == 0) atomicOr(a.status, bad);
  if (bad || n <= B) {
    if (kept)
      for (int j = tid; j < B; j += kThreads) kept[j] = bad || j >= n ? -1 : j;
    return;
  }

  // ---- the m-th largest key T among the candidates, and how many of those equal to it are chosen
  uint32_t T = 0xffffffffu;
  int equal = 0;
  if (m > 0) {
    uint32_t prefix = 0;
    int want = m;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int t = S + tid; t < n - R; t += kThreads) {
        const uint32_t k = order_key(*at.weight(t));
        if (pass == 0 || k >> (shift + bits) == prefix) atomicAdd(&hist[(k >> shift) & ((1 << bits) - 1)], 1);
      }
      __syncthreads();
      // threads take kBins / kThreads bins each, from the highest down
      constexpr int E = kBins / kThreads;
      int mine = 0, total;
      const int top = kBins - 1 - tid * E;
#pragma unroll
      for (int i = 0; i < E; ++i) mine += hist[top - i];
      int above = block_prefix(mine, part, total);
      if (above < want && want <= above + mine) {
        int i = 0;
        while (above + hist[top - i] < want) above += hist[top - i++];
        found[0] = top - i;
        found[1] = above;
      }
      __syncthreads();
      prefix = prefix << bits | (uint32_t)found[0];
      want -= found[1];
      __syncthreads();
    }
    T = prefix;
    equal = want;
  }

  // ---- free slots of [S, B - R) and the chosen above them, in order
  int2* moves = reinterpret_cast<int2*>(a.moves) + (int64_t)blockIdx.x * m;
  int n_equal = 0, n_free = 0, n_moves = 0;
  for (int t0 = S; m > 0 && t0 < n - R; t0 += kThreads) {
    const int t = t0 + tid;
    const uint32_t k = t < n - R ? order_key(*at.weight(t)) : 0u;
    const bool eq = t < n - R && k == T;
    int total;
    const int rank = n_equal + block_prefix(eq, part, total);
    n_equal += total;
    const bool chosen = t < n - R && (k > T || (eq && rank < equal));
    const bool stays = t < B - R, is_free = t < n - R && stays && !chosen, is_move = chosen && !stays;
    // (both counts in one prefix: 16 bits hold a tile's)
    const int before = block_prefix(is_free | is_move << 16, part, total);
    if (is_free) moves[n_free + (before & 0xffff)].y = t;
    if (is_move) moves[n_moves + (before >> 16)].x = t;
    if (kept && stays && t < n - R && chosen) kept[t] = t;
    n_free += total & 0xffff;
    n_moves += total >> 16;
  }
  if (kept) {
    for (int j = tid; j < S; j += kThreads) kept[j] = j;
    for (int j = B - R + tid; j < B; j += kThreads) kept[j] = j + n - B;
  }
  __syncthreads();

  // ---- the chosen into the free slots
  const int P = 2 * p.pieces, W = 2 * p.words + 1;
  for (int i = tid; i < n_moves; i += kThreads) {
    const int2 mv = moves[i];
    if (kept) kept[mv.y] = mv.x;
  }
  for (int64_t i = tid; i < (int64_t)n_moves * P; i += kThreads) {
    const int2 mv = moves[i / P];
    const int q = (int)(i % P);
    *at.piece(mv.y, q, ELT) = *at.piece(mv.x, q, ELT);
  }
  for (int64_t i = tid; i < (int64_t)n_moves * W; i += kThreads) {
    const int2 mv = moves[i / W];
    const int q = (int)(i % W);
    *at.word(mv.y, q) = *at.word(mv.x, q);
  }
  __syncthreads();

  // ---- the newest into [B - R, B)
  const int d = n - B;
  for (int64_t i0 = 0; i0 < (int64_t)R * P; i0 += kThreads) {
    const int64_t i = i0 + tid;
    const int j = B - R + (int)(i / P), q = (int)(i % P);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (i < (int64_t)R * P) v = *at.piece(j + d, q, ELT);
    __syncthreads();
    if (i < (int64_t)R * P) *at.piece(j, q, ELT) = v;
  }
  for (int64_t i0 = 0; i0 < (int64_t)R * W; i0 += kThreads) {
    const int64_t i = i0 + tid;
    const int j = B - R + (int)(i / W), q = (int)(i % W);
    uint32_t v = 0;
    if (i < (int64_t)R * W) v = *at.word(j + d, q);
    __syncthreads();
    if (i < (int64_t)R * W) *at.word(j, q) = v;
  }
  __syncthreads();
  for (int t = B + tid; t < n; t += kThreads) *at.weight(t) = 0.f;
}

}  // namespace

cudaError_t launch_evict(const pkd_evict_args& a, cudaStream_t s) {
  EvictParams p;
  p.a = a;
  p.page_log = 31 - __builtin_clz((unsigned)a.pool.page_size);
  const int elt = a.pool.dtype == PKD_DTYPE_F16 || a.pool.dtype == PKD_DTYPE_BF16 ? 2 : 1;
  const bool codes = a.pool.dtype == PKD_DTYPE_E2M1;
  p.pieces = a.pool.head_dim * elt / (codes ? 2 : 1) / 16;
  p.words = codes ? a.pool.head_dim / 64 : 0;
  const unsigned grid = (unsigned)a.pool.batch * (unsigned)a.pool.num_kv_heads;
  return launch_pdl(elt == 2 ? evict_kernel<2> : evict_kernel<1>, p, grid, kThreads, s);
}

}  // namespace pkd
