// key_weights.cu -- the second half of a decode that sums its keys' weights: the decode kernel has left
// every attended score s (base 2) and each row's softmax statistics, the maximum M and 1 / L with
// L = sum 2^(s - M); here each key's weight, 2^(s - M) / L summed over the query rows and the qo heads
// of its kv head, is added to its slot of the weights' pool.
//
// Why two kernels: a key's weight needs the whole row's L, which a split row has only once its last
// chunk is merged.  Keeping the scores costs 4 bytes written and read per key and qo head (through L2,
// mostly) where reading K again would cost a kv head's row of 2 * head_dim bytes.
// Sums run in the order of rows and heads, in 32 bits, in one thread per slot; what that thread adds to
// the pool is one reduction, so that a slot shared by several requests takes all their additions.
//
// Bound: loads under way (13 to 16 long-scoreboard stalls an issue, DRAM 26 to 45 %).  32 qo and 8 kv heads:
// 64 rows of 512 to 4,096 keys 11.7 us by itself, some 8 behind its decode, for 19 MB of scores and 9 MB of
// weights; 4 of 131,072 keys 23 us, 67 and 34 MB.  One key a thread and 4-byte loads took 16.5 and 45 us.  Fetching a
// thread's next tile ahead gained nothing.
#include "pkd_device.cuh"
#include "pkd_internal.h"

namespace pkd {

namespace {

constexpr int kThreads = kKeyTileTokens / 4;

// Adds x to the four slots at w (16-byte aligned).
__device__ __forceinline__ void add4(float* w, const float (&x)[4]) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(w), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3])
               : "memory");
}

__device__ __forceinline__ float4 ld_first(const float* p, uint64_t policy) {
  float4 v;
  asm volatile("ld.global.L2::cache_hint.v4.f32 {%0, %1, %2, %3}, [%4], %5;"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p), "l"(policy));
  return v;
}

// A thread takes four consecutive keys, so that scores are read 16 bytes at a time (a row's scores are
// laid out so that key t lies at a multiple of 16 bytes where t is one of 4, see KeyRow).
__global__ void __launch_bounds__(kThreads) key_weights_kernel(const __grid_constant__ KeyWeightParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (a decode launch that gave up left scores out)
  if (*reinterpret_cast<const volatile uint32_t*>(p.status) & dev::kStatusTimeout) return;
  const uint64_t pol = dev::policy_evict_first();
  const int hkv = p.num_kv_heads, group = p.num_qo_heads / hkv;
  const uint32_t units = (uint32_t)(p.tile_count ? *p.tile_count : p.num_tiles) * (uint32_t)hkv;
  for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int kvh = (int)(u % (uint32_t)hkv);
    const KeyTile tile = p.tiles[u / (uint32_t)hkv];
    const int t = (tile.t0 & ~3) + 4 * threadIdx.x;
    if (t >= tile.t1) continue;
    const uint32_t page = (uint32_t)__ldg(p.indices + tile.page_base + (t >> p.page_log));
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < p.q_len; ++j) {
      const int row = tile.req * p.q_len + j;
      const KeyRow kr = p.rows[row];
      bool in[4], any = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        in[i] = t + i < kr.sink || (t + i >= kr.win && t + i < kr.n);
        any |= in[i];
      }
      if (!any) continue;
      // (four keys of which some are sinks and some the window's: the two parts lie apart)
      const bool both = t < kr.sink && t + 3 >= kr.win;
      const float* s = p.scores + kr.base + (int64_t)kvh * group * kr.stride + t;
      const float* at = s + (t < kr.sink ? 0 : kr.shift);
      const float2* st = p.stats + (int64_t)row * p.num_qo_heads + kvh * group;
#pragma unroll 4
      for (int g = 0; g < group; ++g) {
        const float2 ml = st[g];
        float4 x = ld_first(at + (int64_t)g * kr.stride, pol);
        if (both) {
          const float4 y = *reinterpret_cast<const float4*>(s + (int64_t)g * kr.stride + kr.shift);
          x.y = t + 1 < kr.sink ? x.y : y.y;
          x.z = t + 2 < kr.sink ? x.z : y.z;
          x.w = t + 3 < kr.sink ? x.w : y.w;
        }
        sum[0] += in[0] ? dev::fast_exp2(x.x - ml.x) * ml.y : 0.f;
        sum[1] += in[1] ? dev::fast_exp2(x.y - ml.x) * ml.y : 0.f;
        sum[2] += in[2] ? dev::fast_exp2(x.z - ml.x) * ml.y : 0.f;
        sum[3] += in[3] ? dev::fast_exp2(x.w - ml.x) * ml.y : 0.f;
      }
    }
    if (page >= p.num_pages) continue;  // (the decode launch has reported the id)
    float* w = p.weights + page * p.strides[0] + kvh * p.strides[1] + (t & ((1 << p.page_log) - 1)) * p.strides[2];
    if (p.quads && t >= tile.t0 && t + 4 <= tile.t1) {
      add4(w, sum);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t + i >= tile.t0 && t + i < tile.t1) atomicAdd(w + i * p.strides[2], sum[i]);
    }
  }
}

}  // namespace

const void* key_weights_fn(int* threads) {
  *threads = kThreads;
  return reinterpret_cast<const void*>(&key_weights_kernel);
}

}  // namespace pkd
