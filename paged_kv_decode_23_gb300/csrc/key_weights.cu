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
#include "pkd_device.cuh"
#include "pkd_internal.h"

namespace pkd {

namespace {

__global__ void __launch_bounds__(kKeyTileTokens) key_weights_kernel(const __grid_constant__ KeyWeightParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (a decode launch that gave up left scores out)
  if (*reinterpret_cast<const volatile uint32_t*>(p.status) & dev::kStatusTimeout) return;
  const int hkv = p.num_kv_heads, group = p.num_qo_heads / hkv;
  const int64_t units = (int64_t)(p.tile_count ? *p.tile_count : p.num_tiles) * hkv;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int kvh = (int)(u % hkv);
    const KeyTile tile = p.tiles[u / hkv];
    const int t = tile.t0 + threadIdx.x;
    if (t >= tile.t1) continue;
    float sum = 0.f;
    for (int j = 0; j < p.q_len; ++j) {
      const int row = tile.req * p.q_len + j;
      const KeyRow kr = p.rows[row];
      const bool sink = t < kr.sink;
      if (t >= kr.n || (!sink && t < kr.win)) continue;
      const float* s = p.scores + kr.base + (int64_t)kvh * group * kr.stride + t + (sink ? 0 : kr.shift);
      const float2* st = p.stats + (int64_t)row * p.num_qo_heads + kvh * group;
#pragma unroll 4
      for (int g = 0; g < group; ++g) {
        const float2 ml = st[g];
        sum += dev::fast_exp2(s[(int64_t)g * kr.stride] - ml.x) * ml.y;
      }
    }
    const uint32_t page = (uint32_t)p.indices[tile.page_base + t / p.page_size];
    if (page < p.num_pages)  // (the decode launch has reported other ids)
      atomicAdd(p.weights + page * p.strides[0] + kvh * p.strides[1] + (t & (p.page_size - 1)) * p.strides[2], sum);
  }
}

}  // namespace

const void* key_weights_fn() { return reinterpret_cast<const void*>(&key_weights_kernel); }

}  // namespace pkd
