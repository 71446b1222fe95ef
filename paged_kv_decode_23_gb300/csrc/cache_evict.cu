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
// So no row moves that need not, and what moves is read and written once.
//
// A cluster of CTAs takes one (sequence, kv head): each holds the keys of a run of candidates in shared
// memory, finds the m-th largest with the others (three digits of 11, 11 and 10 bits: histograms, summed
// over the cluster), counts what it chooses, and lists its free slots and moves behind those of the CTAs
// before it; then all move rows.  A row that moves into [S, B - R) overwrites nothing that is read; the
// newest are shifted down once those rows are read, in tiles that are read whole before they are written
// (a tile's sources lie above every earlier tile's destinations), each CTA a part of the rows' columns.
//
// Bound: the moves are a copy's traffic, what comes before them is waiting (three dependent loads, then
// exchanges between the CTAs of a cluster, some 2 us each) and, where a CTA holds thousands of keys, instructions.
// 64 sequences of 2,049 to 2,064 tokens to 2,048, 8 heads of 128, 16 bits: 25 us (80 MB, 12 us at a copy's
// rate; 17 us with the rows in L2), 9 of them selection; 4 of 60,000 to 131,072 to 8,192: 83 us (270 MB, 40), some
// 27 of them selection and 45 the moves.  Places worked out once a row and passed by shuffles, and strides in 32
// bits, took 9 M of 17.8 M warp instructions away (38 -> 25 us in the first); loops over keys that are known to
// lie in shared memory 9 us in the second.
#include <cooperative_groups.h>

#include <algorithm>

#include "cache_rows.cuh"

namespace pkd {

namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 2048;  // of an 11-bit digit
constexpr int kMaxRanks = 8;
// Where at most so many keys share the digits found so far, they are compared with each other instead of
// going through the next digits (without that 512 units of 2,064 tokens take 1.5 to 3 us more).
constexpr int kFew = 256;
constexpr int kMostKeys = 16 << 10;  // that a CTA holds
constexpr int kMostTokens = 1 << 30;  // (positions and steps past them stay in 32 bits)

// Order of weights as unsigned numbers: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The weight of a key, but for 0 (of either sign) and NaN.
__device__ __forceinline__ float weight_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

struct EvictParams {
  const int32_t *indptr, *indices, *kv_lens;
  int64_t num_indices;
  uint32_t num_pages;
  int32_t num_kv_heads, budget, sinks, recent;
  int32_t *kept, *moves;
  int64_t places;  // of moves: where the list of free slots begins
  uint32_t* status;
  // K and V rows: strides of page and slot in 16-byte units, of a head in bytes; scales in 4-byte units
  // and bytes, weights in elements
  char *k, *v, *k_scales, *v_scales;
  float* weights;
  uint32_t page16, slot16, scale_page4, scale_slot4, weight_page, weight_slot;
  int64_t head, scale_head, weight_head;
  int quads;       // 1: the weights of four slots (from a multiple of 4) are one aligned float4
  int page_log;
  int pieces_log;  // 16-byte pieces of a row, K and V together: 1 << pieces_log
  int words;       // 4-byte words of a row's scales, K (or V) alone
  int cap;         // keys that a CTA's shared memory holds; the others are read again
  int ahead;       // of the newest, rows that are fetched into L2 while the others are chosen
};

// One (sequence, kv head): where its rows lie.
struct Rows {
  const EvictParams& p;
  const int32_t* ids;  // the sequence's page ids
  char *k, *v;         // its head's rows of page 0, slot 0
  int64_t scale_head;
  float* w;
  __device__ __forceinline__ Rows(const EvictParams& p, const int32_t* ids, int head)
      : p(p), ids(ids), k(p.k + head * p.head), v(p.v + head * p.head), scale_head(head * p.scale_head),
        w(p.weights + head * p.weight_head) {}
  __device__ __forceinline__ uint32_t page(int t) const { return (uint32_t)__ldg(ids + (t >> p.page_log)); }
  __device__ __forceinline__ uint32_t slot(int t) const { return t & ((1 << p.page_log) - 1); }
  __device__ __forceinline__ float* weight_in(uint32_t page, int t) const {
    return w + ((uint64_t)page * p.weight_page + (uint64_t)slot(t) * p.weight_slot);
  }
  __device__ __forceinline__ float* weight(int t) const { return weight_in(page(t), t); }
  // 16-byte units from the pool's base to token t's row, of K and V alike; 16-byte piece q of the row at
  // such an offset: the K row's, then the V row's
  __device__ __forceinline__ uint64_t offset(int t) const {
    return (uint64_t)page(t) * p.page16 + (uint64_t)slot(t) * p.slot16;
  }
  __device__ __forceinline__ uint4* piece_at(uint64_t offset, int q) const {
    const int half = 1 << (p.pieces_log - 1);
    return reinterpret_cast<uint4*>(q & half ? v : k) + (offset + (q & (half - 1)));
  }
  // word q of token t's K scales (q < words) or V scales
  __device__ __forceinline__ uint32_t* word(int t, int q) const {
    const uint64_t at = (uint64_t)page(t) * p.scale_page4 + (uint64_t)slot(t) * p.scale_slot4;
    const bool v = q >= p.words;
    return reinterpret_cast<uint32_t*>((v ? p.v_scales : p.k_scales) + scale_head) + (at + (v ? q - p.words : q));
  }
};

// Exclusive prefix of `mine` over the block's threads, and the sum; `part` holds a number per warp.  A
// barrier lies between two calls.
template <int THREADS>
__device__ __forceinline__ int block_prefix(int mine, int* part, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  return before + x - mine;
}

// CLUSTER: several CTAs a (sequence, kv head), else one.  LOADS: groups of four keys a thread has under way.
template <int THREADS, int CTAS, bool CLUSTER, int LOADS>
__global__ void __launch_bounds__(THREADS, CTAS) evict_kernel(const __grid_constant__ EvictParams p) {
  constexpr int WARPS = THREADS / 32, E = kBins / THREADS;  // bins a thread sums
  static_assert(E % 4 == 0, "");
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int hist[2][kBins];
  __shared__ uint32_t few[kFew];  // keys among which the last digits are found without histograms
  __shared__ int part[2][WARPS];
  __shared__ int found[3];
  // to the cluster: counts of equal and of larger keys below B - R and not, tokens below; bad pages; keys in `few`
  __shared__ int said[7];
  __shared__ int theirs[5][kMaxRanks];  // what the CTAs of the cluster said
  asm volatile("griddepcontrol.wait;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
  auto sync = [&] {
    if constexpr (CLUSTER) cluster.sync();
    else __syncthreads();
  };
  auto of_rank = [&](auto* x, int r) { return CLUSTER ? cluster.map_shared_rank(x, r) : x; };
  const int hkv = p.num_kv_heads, unit = blockIdx.x / ranks, seq = unit / hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int all = ranks * THREADS, me = rank * THREADS + tid;
  const int B = p.budget, S = p.sinks, R = p.recent, m = B - S - R;
  const int n = __ldg(p.kv_lens + seq);
  int32_t* kept = p.kept ? p.kept + (int64_t)unit * B : nullptr;
  const int64_t first = __ldg(p.indptr + seq), end = __ldg(p.indptr + seq + 1);
  const int64_t pages = ((int64_t)n + (1 << p.page_log) - 1) >> p.page_log;
  const bool no_token = n < 0 || n > kMostTokens ||
                        (n > 0 && (first < 0 || first + pages > end || first + pages > p.num_indices));
  if (no_token || n <= B) {  // (the whole cluster)
    if (no_token && p.status && rank == 0 && tid == 0) atomicOr(p.status, PKD_STATUS_BAD_TOKEN);
    if (kept)
      for (int j = me; j < B; j += all) kept[j] = no_token || j >= n ? -1 : j;
    return;
  }
  const Rows at(p, p.indices + first, unit % hkv);

  // ---- the keys of this CTA's run of tokens [lo, lo + v1); those from v0 on are candidates
  const int start = S & ~3, per = ((n - R - start + ranks - 1) / ranks + 31) & ~31;
  const int lo = (int)min((int64_t)start + (int64_t)rank * per, (int64_t)(n - R));
  const int v0 = max(S - lo, 0), v1 = min(per, n - R - lo);
  bool off = false;
  auto known = [&](uint32_t id) {
    off |= id >= p.num_pages;
    return id < p.num_pages;
  };
  for (int i = tid; i < kBins / 4; i += THREADS) reinterpret_cast<int4*>(hist[0])[i] = make_int4(0, 0, 0, 0);
  if (tid < 7) said[tid] = 0;
  __syncthreads();
  for (int i = 4 * tid; i < v1; i += 4 * LOADS * THREADS) {
    uint32_t id[LOADS];
    float4 x[LOADS];
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int j = i + 4 * u * THREADS;
      id[u] = j < v1 ? at.page(lo + j) : 0u;
    }
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int j = i + 4 * u * THREADS;
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < v1 && known(id[u])) {
        const float* src = at.weight_in(id[u], lo + j);
        if (p.quads) {
          x[u] = *reinterpret_cast<const float4*>(src);
        } else {
          x[u].x = src[0];
          x[u].y = src[p.weight_slot];
          x[u].z = src[2 * (uint64_t)p.weight_slot];
          x[u].w = src[3 * (uint64_t)p.weight_slot];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int j = i + 4 * u * THREADS;
      if (j >= v1) break;
      const uint4 k = make_uint4(order_key(x[u].x), order_key(x[u].y), order_key(x[u].z), order_key(x[u].w));
      if (j < p.cap) *reinterpret_cast<uint4*>(keys + j) = k;
      if (j >= v0) atomicAdd(&hist[0][k.x >> 21], 1);
      if (j + 1 >= v0 && j + 1 < v1) atomicAdd(&hist[0][k.y >> 21], 1);
      if (j + 2 >= v0 && j + 2 < v1) atomicAdd(&hist[0][k.z >> 21], 1);
      if (j + 3 >= v0 && j + 3 < v1) atomicAdd(&hist[0][k.w >> 21], 1);
    }
  }
  // the newest's rows will be read whatever is chosen (before the keys' loads this was no gain)
  {
    const int line_log = max(p.pieces_log - 3, 1);  // 128-byte lines of a row: K's, then V's (shorter rows: one each)
    for (int x = me; x < p.ahead << line_log; x += all) {
      const int t = n - 1 - (x >> line_log);
      if (known(at.page(t)))
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            at.piece_at(at.offset(t), (x & ((1 << line_log) - 1)) << (p.pieces_log - line_log))));
    }
  }
  // (the pages of the sinks and of the newest)
  if (rank == 0)
    for (int64_t i = tid; i << p.page_log < S; i += THREADS) known((uint32_t)__ldg(at.ids + i));
  if (rank == ranks - 1)
    for (int64_t i = ((n - R) >> p.page_log) + tid; i < pages; i += THREADS) known((uint32_t)__ldg(at.ids + i));
  bool bad = __syncthreads_or(off);
  if constexpr (CLUSTER) {
    if (tid == 0) said[5] = bad;
    sync();
    bad = __syncthreads_or(tid < ranks ? *of_rank(&said[5], tid) : 0);
  }
  if (bad) {
    if (p.status && rank == 0 && tid == 0) atomicOr(p.status, PKD_STATUS_BAD_PAGE);
    if (kept)
      for (int j = me; j < B; j += all) kept[j] = -1;
    sync();  // (no CTA leaves while another may still read its flag)
    return;
  }
  // where most slots take their tokens from; the moves below change what they change
  if (kept)
    for (int j = me; j < B; j += all) kept[j] = j < B - R ? j : j + n - B;
  int2* moves = reinterpret_cast<int2*>(p.moves) + (int64_t)unit * m;
  int32_t* places = p.moves + p.places + (int64_t)unit * m;
  int n_moves = 0;
  auto choose = [&](auto key) {
    // ---- the m-th largest key T among the candidates, and how many of those equal to it are chosen
    uint32_t T = 0xffffffffu;
    int equal = 0;  // (m = 0: nothing is chosen)
    if (m > 0) {
      T = 0;
      equal = m;
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        int* h = hist[pass & 1];
        if (pass > 0) {
          for (int i = tid; i < kBins / 4; i += THREADS) reinterpret_cast<int4*>(h)[i] = make_int4(0, 0, 0, 0);
          __syncthreads();
#pragma unroll 4
          for (int i = v0 + tid; i < v1; i += THREADS) {
            const uint32_t k = key(i);
            if (k >> (shift + bits) == T) atomicAdd(&h[(k >> shift) & ((1 << bits) - 1)], 1);
          }
          sync();
        }
        // threads take E bins each, from the highest down, summed over the cluster
        const int top = kBins - 1 - tid * E;
        int sum[E], mine = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) sum[i] = 0;
#pragma unroll
        for (int r = 0; r < (CLUSTER ? kMaxRanks : 1); ++r)
          if (r < ranks) {
            const int4* hr = reinterpret_cast<const int4*>(of_rank(h, r)) + (top >> 2);
#pragma unroll
            for (int i = 0; i < E; i += 4) {
              const int4 v = hr[-(i >> 2)];
              sum[i] += v.w; sum[i + 1] += v.z; sum[i + 2] += v.y; sum[i + 3] += v.x;
            }
          }
#pragma unroll
        for (int i = 0; i < E; ++i) mine += sum[i];
        int all_keys;
        int above = block_prefix<THREADS>(mine, part[0], all_keys);
        if (above < equal && equal <= above + mine) {
#pragma unroll
          for (int i = 0; i < E; ++i) {
            if (above < equal && equal <= above + sum[i]) {
              found[0] = top - i;
              found[1] = above;
              found[2] = sum[i];
            }
            above += sum[i];
          }
        }
        __syncthreads();
        T = T << bits | (uint32_t)found[0];
        equal -= found[1];
        const int left = found[2];
        __syncthreads();  // (found is written again)
        if (pass < 2 && left <= kFew) {
          // few keys begin with T: each is compared with all of them
          for (int i = v0 + tid; i < v1; i += THREADS) {
            const uint32_t k = key(i);
            if (k >> shift == T) {
              const int x = atomicAdd(&said[6], 1);
              if (x < kFew) few[x] = k;
            }
          }
          sync();
          if constexpr (CLUSTER) {  // those of all CTAs, into the histogram that is not in use
            uint32_t* list = reinterpret_cast<uint32_t*>(hist[~pass & 1]);
            if (tid < ranks) theirs[0][tid] = *of_rank(&said[6], tid);
            __syncthreads();
            for (int i = tid; i < left; i += THREADS) {
              int r = 0, j = i;
              while (r + 1 < ranks && j >= theirs[0][r]) j -= theirs[0][r++];
              list[i] = of_rank(few, r)[j & (kFew - 1)];
            }
            __syncthreads();
          }
          const uint32_t* list = CLUSTER ? reinterpret_cast<const uint32_t*>(hist[~pass & 1]) : few;
          for (int i = tid; i < left; i += THREADS) {
            const uint32_t k = list[i];
            int greater = 0, same = 0;
            for (int j = 0; j < left; ++j) {
              greater += list[j] > k;
              same += list[j] == k;
            }
            if (greater < equal && equal <= greater + same) {  // (of equal keys, all say the same)
              found[0] = (int)k;
              found[1] = greater;
            }
          }
          __syncthreads();
          T = (uint32_t)found[0];
          equal -= found[1];
          break;
        }
      }
    }

    // ---- counts of each thread's run; the chosen among equal keys are the first of them.  (Runs of an
    // odd length keep the threads of a warp in different banks.)
    const int run = ((v1 - v0 + THREADS - 1) / THREADS) | 1;
    const int i0 = min(v0 + tid * run, v1), i1 = min(i0 + run, v1);
    const int edge = min(max(B - R - lo, i0), i1);  // [i0, edge) lies in [S, B - R)
    int gt_low = 0, gt_high = 0, eq_low = 0, eq_high = 0;
#pragma unroll 4
    for (int i = i0; i < edge; ++i) {
      const uint32_t k = key(i);
      gt_low += k > T;
      eq_low += k == T;
    }
#pragma unroll 4
    for (int i = edge; i < i1; ++i) {
      const uint32_t k = key(i);
      gt_high += k > T;
      eq_high += k == T;
    }
    // Equal keys before this thread's, and with them what it leaves free and moves; then both before it.
    // A CTA's tokens below B - R come before its others, so its sums of five counts say how many of its
    // equal keys are chosen on either side: one exchange between the CTAs.
    int total;
    int eq_base = block_prefix<THREADS>(eq_low + eq_high, part[1], total);
    int free_base = 0, move_base = 0;
    if constexpr (CLUSTER) {
      const int five[5] = {eq_low, eq_high, gt_low, gt_high, edge - i0};
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        const int x = __reduce_add_sync(~0u, five[i]);
        if (lane == 0 && x) atomicAdd(&said[i], x);
      }
      sync();
      for (int i = tid; i < 5 * ranks; i += THREADS) theirs[i % 5][i / 5] = of_rank(said, i / 5)[i % 5];
      __syncthreads();
      int eq_before = 0;
      n_moves = 0;
      for (int r = 0; r < ranks; ++r) {
        const int of[5] = {theirs[0][r], theirs[1][r], theirs[2][r], theirs[3][r], theirs[4][r]};
        const int lows = of[0], highs = of[1];
        const int take_low = max(0, min(lows, equal - eq_before));
        const int take_high = max(0, min(highs, equal - eq_before - lows));
        if (r < rank) {
          eq_base += lows + highs;
          free_base += of[4] - of[2] - take_low;
          move_base += of[3] + take_high;
        }
        n_moves += of[3] + take_high;
        eq_before += lows + highs;
      }
    }
    eq_low = max(0, min(eq_low, equal - eq_base));
    eq_high = max(0, min(eq_high, equal - eq_base - eq_low));
    free_base += block_prefix<THREADS>(edge - i0 - gt_low - eq_low, part[0], total);
    move_base += block_prefix<THREADS>(gt_high + eq_high, part[1], total);
    if constexpr (!CLUSTER) n_moves = total;

    // ---- the lists: the i-th free slot of [S, B - R) takes the i-th chosen above it, its weight with it
    {
      int left = equal - eq_base;  // equal keys still to choose
#pragma unroll 4
      for (int i = i0; i < edge; ++i) {
        const uint32_t k = key(i);
        if (k <= T && !(k == T && left-- > 0) && free_base < m) places[free_base++] = lo + i;
      }
#pragma unroll 4
      for (int i = edge; i < i1; ++i) {
        const uint32_t k = key(i);
        if (k >= T && (k > T || left-- > 0) && move_base < m) {
          const bool plain = k != 0xffffffffu && k != 0x80000000u;
          moves[move_base++] = make_int2(lo + i, __float_as_int(plain ? weight_of(k) : *at.weight(lo + i)));
        }
      }
    }
  };
  // (A run that shared memory does not hold goes through the same steps, its last keys read again.  Were they
  // to change meanwhile, what is chosen would mean nothing; that lists and rows stay in their bounds all the
  // same is what the tests of free_base, move_base and of the places below are for.)
  if (v1 <= p.cap) choose([&](int i) { return keys[i]; });
  else choose([&](int i) { return i < p.cap ? keys[i] : order_key(*at.weight(lo + i)); });
  sync();
  n_moves = min(n_moves, m);

  // ---- candidates' slots that no token is left in
  const int W = 2 * p.words;
  for (int t = (B & ~3) + 4 * me; t < n - R; t += 4 * all) {
    float* w = at.weight(t);
    if (p.quads && t >= B && t + 4 <= n - R) {
      *reinterpret_cast<float4*>(w) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      for (int i = 0; i < 4; ++i)
        if (t + i >= B && t + i < n - R) w[i * (uint64_t)p.weight_slot] = 0.f;
    }
  }

  // ---- the chosen into the free slots: a warp takes up to 32 rows at a time, a lane finds one's places and
  // moves its scales and weight, and the lanes move the pieces of all together
  const int P = 1 << p.pieces_log;
  const int per_warp = min(32, (n_moves + ranks * WARPS - 1) / (ranks * WARPS));
  for (int r0 = (rank * WARPS + warp) * per_warp; r0 < n_moves; r0 += ranks * WARPS * per_warp) {
    const int rows = min(per_warp, n_moves - r0);
    uint64_t from = 0, to = 0;
    if (lane < rows) {
      int2 mv = __ldcg(moves + r0 + lane);
      int place = __ldcg(places + r0 + lane);
      if (mv.x < B - R || mv.x >= n - R) mv.x = B - R;
      if (place < S || place >= B - R) place = S;
      from = at.offset(mv.x);
      to = at.offset(place);
      if (kept) kept[place] = mv.x;
      *at.weight(place) = __int_as_float(mv.y);
      for (int q = 0; q < W; ++q) *at.word(place, q) = *at.word(mv.x, q);
    }
    const int n_pieces = rows << p.pieces_log;
    constexpr int U = 4;                           // pieces under way a thread
    for (int x0 = 0; x0 < n_pieces; x0 += 32 * U) {  // (whole warps)
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int y = x0 + 32 * u + lane;
        const uint64_t src = __shfl_sync(~0u, from, y >> p.pieces_log);
        if (y < n_pieces) v[u] = *at.piece_at(src, y & (P - 1));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int y = x0 + 32 * u + lane;
        const uint64_t dst = __shfl_sync(~0u, to, y >> p.pieces_log);
        if (y < n_pieces) *at.piece_at(dst, y & (P - 1)) = v[u];
      }
    }
  }
  sync();

  // ---- the newest into [B - R, B): a CTA takes 1 << part_log pieces of every row, a tile of rows at a time
  const int d = n - B;
  int part_log = p.pieces_log;
  while (CLUSTER && part_log > 1 && P >> part_log < ranks) --part_log;
  if (rank < P >> part_log) {
    constexpr int U = 4;
    const int q0 = rank << part_log, q_mask = (1 << part_log) - 1;
    const int per_tile = min(32, (32 * U) >> part_log);  // rows of a warp
    for (int r0 = 0; r0 < R; r0 += WARPS * per_tile) {
      const int j0 = r0 + warp * per_tile, n_pieces = max(0, min(per_tile, R - j0)) << part_log;
      uint64_t from = 0, to = 0;
      if (lane < n_pieces >> part_log) {
        to = at.offset(B - R + j0 + lane);
        from = at.offset(B - R + j0 + lane + d);
      }
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int y = 32 * u + lane;
        const uint64_t src = __shfl_sync(~0u, from, y >> part_log);
        if (y < n_pieces) v[u] = *at.piece_at(src, q0 + (y & q_mask));
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int y = 32 * u + lane;
        const uint64_t dst = __shfl_sync(~0u, to, y >> part_log);
        if (y < n_pieces) *at.piece_at(dst, q0 + (y & q_mask)) = v[u];
      }
    }
  }
  // their scales and weights: the last CTA, which then clears what they leave
  if (rank == ranks - 1) {
    for (int q = 0; q <= W; ++q)
      for (int r0 = 0; r0 < R; r0 += THREADS) {
        const int j = B - R + r0 + tid;
        uint32_t x = 0;
        if (j < B) x = q < W ? *at.word(j + d, q) : __float_as_uint(*at.weight(j + d));
        __syncthreads();
        if (j < B) {
          if (q < W) *at.word(j, q) = x;
          else *at.weight(j) = __uint_as_float(x);
        }
      }
    __syncthreads();
    for (int t = max(B, n - R) + tid; t < n; t += THREADS) *at.weight(t) = 0.f;
  }
}

template <int THREADS, int CTAS, bool CLUSTER, int LOADS>
cudaError_t launch(const EvictParams& p, int units, int ranks, cudaStream_t s) {
  const int smem = p.cap * 4;
  const void* fn = reinterpret_cast<const void*>(&evict_kernel<THREADS, CTAS, CLUSTER, LOADS>);
  if (smem > 16 << 10) {  // with what the kernel has besides, more than a launch may take unasked
    // (always the same limit: calls on other threads, and captured ones, must not find it lowered)
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMostKeys);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * ranks));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 2 : 1;
  void* args[] = {const_cast<EvictParams*>(&p)};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_evict(const pkd_evict_args& a, cudaStream_t s) {
  const pkd_paged_pool& c = a.pool;
  const bool wide = c.dtype == PKD_DTYPE_F16 || c.dtype == PKD_DTYPE_BF16, codes = c.dtype == PKD_DTYPE_E2M1;
  const int64_t elt = wide ? 2 : 1;
  EvictParams p = {};
  p.indptr = c.indptr;
  p.indices = c.indices;
  p.kv_lens = a.kv_lens;
  p.num_indices = c.num_indices;
  p.num_pages = (uint32_t)std::min<int64_t>(c.num_pages, INT64_C(1) << 31);
  p.num_kv_heads = c.num_kv_heads;
  p.budget = a.budget;
  p.sinks = a.num_sink_tokens;
  p.recent = a.num_recent;
  p.kept = a.kept;
  p.moves = a.moves;
  p.status = a.status;
  p.k = static_cast<char*>(c.k);
  p.v = static_cast<char*>(c.v);
  p.k_scales = static_cast<char*>(c.k_scales);
  p.v_scales = static_cast<char*>(c.v_scales);
  p.weights = a.key_weights;
  // (the stride of an axis of one entry is never used)
  auto units_of = [](int64_t stride, int64_t unit, int64_t n) { return n > 1 ? (uint32_t)(stride / unit) : 0u; };
  p.page16 = units_of(c.strides[0] * elt, 16, c.num_pages);
  p.slot16 = units_of(c.strides[1] * elt, 16, c.page_size);
  p.head = c.num_kv_heads > 1 ? c.strides[2] * elt : 0;
  if (codes) {
    p.scale_page4 = units_of(c.scale_strides[0], 4, c.num_pages);
    p.scale_slot4 = units_of(c.scale_strides[1], 4, c.page_size);
    p.scale_head = c.num_kv_heads > 1 ? c.scale_strides[2] : 0;
  }
  p.weight_page = units_of(a.weight_strides[0], 1, c.num_pages);
  p.weight_head = c.num_kv_heads > 1 ? a.weight_strides[1] : 0;
  p.weight_slot = units_of(a.weight_strides[2], 1, c.page_size);
  p.quads = p.weight_slot == 1 && p.weight_page % 4 == 0 && p.weight_head % 4 == 0 &&
            reinterpret_cast<uintptr_t>(a.key_weights) % 16 == 0;
  p.page_log = 31 - __builtin_clz((unsigned)c.page_size);
  const int row = codes ? c.head_dim / 2 : c.head_dim * (int)elt;
  p.pieces_log = 31 - __builtin_clz((unsigned)(row / 8));
  p.words = codes ? c.head_dim / 64 : 0;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // The lengths are on the device; the pages that a sequence owns on average stand for them.  CTAs a
  // (sequence, kv head): as many as the GPU holds of 512 threads, two an SM, but none for fewer than some
  // 1,100 tokens, where the exchanges take longer than what they save (us for 1, 2, 4, 8 CTAs, 8 heads of 128):
  // 1 sequence of 2,064 tokens 10.4, 12.4, 12.4, 14.5; 8 of 4,096 28.7, 22.5, 23.3, 46.4; 1 of 16,000 55, 37,
  // 24.6, 22.6; 4 of 60,000 to 131,072 744, 392, 188, 94; 33 of 500 to 9,000 (2 heads of 256) 46, 38, 30, 52.
  const int units = c.batch * c.num_kv_heads;
  p.places = 2 * (int64_t)units * (a.budget - a.num_sink_tokens - a.num_recent);
  const int64_t tokens = c.num_indices * c.page_size / c.batch;
  int ranks = 1;
  while (ranks < kMaxRanks && (int64_t)units * ranks * 2 <= 2 * sms && tokens / (ranks * 2) >= 1100) ranks *= 2;
  // One CTA each: of 512 threads while all of those are resident at once, else of 256, four an SM, but for long
  // sequences (us with 512 and 256 threads: 256 units of 4,096 tokens 65.8, 71.7; 512 of 2,064 28.6, 25.0; of
  // 5,000 161, 159; of 9,000 184, 217; of 16,000 225, 311; 1,024 of 1,040 55, 44).
  const bool small = units > 2 * sms && tokens <= 6000;
  // room for the average and a half of it, up to what leaves the SM its CTAs: 32 KiB and 64 KiB (512 units of
  // 2,064 tokens, 256 threads each: 26.6 us with 32 KiB, 29.6 with 64).  Sequences longer than that read the rest
  // of their keys again in every pass
  const int most = small ? kMostKeys / 2 : kMostKeys;
  p.cap = 1024;
  while (p.cap < most && p.cap < tokens / ranks + tokens / ranks / 2) p.cap *= 2;
  // 64 sequences of 2,064 tokens with 128 newest, not in L2: 26.0 us for 28.4; up to what L2 holds beside
  // the rest, no gain elsewhere.
  const int64_t room = (int64_t(48) << 20) / ((int64_t)units * row * 2);
  p.ahead = (int)std::min<int64_t>(a.num_recent, room);
  if (ranks > 1) return launch<512, 2, true, 4>(p, units, ranks, s);
  return small ? launch<256, 4, false, 2>(p, units, 1, s) : launch<512, 2, false, 2>(p, units, 1, s);
}

}  // namespace pkd
