// Stable counting sort of small keys inside one thread block, shared by the
// router and the adapters' preparation: entry e of n with key(e) in [0, G)
// goes to base[key] + (its rank among the block's entries of that key, in
// increasing e). Each warp owns a contiguous run of entries; inside 32 entries
// the ranks come from __match_any_sync, across runs from the warps' counters.
#pragma once

#include <cstdint>

#include "pgg_ptx.cuh"

namespace pgg {

__device__ __forceinline__ uint32_t lanes_below(int lane) { return (1u << lane) - 1u; }

// cnt [warps][G] in shared memory: this warp's entries of each key. `run` is the
// warps' entries each (a multiple of 32).
template <typename Key>
__device__ __forceinline__ void sort_count(uint32_t* cnt, int G, int n, int run, Key key) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int i = threadIdx.x; i < warps * G; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  uint32_t* mine = cnt + warp * G;
  const int end = (warp + 1) * run < n ? (warp + 1) * run : n;
  for (int e0 = warp * run; e0 < end; e0 += 32) {
    const int e = e0 + lane;
    const int k = e < end ? key(e) : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, k);
    if (k >= 0 && (same & lanes_below(lane)) == 0) mine[k] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
}

// Turns the warps' counts into the first place of each (warp, key), from
// base(key); then calls place(e, where) for every entry.
template <typename Key, typename Base, typename Place>
__device__ __forceinline__ void sort_place(uint32_t* cnt, int G, int n, int run, Key key, Base base,
                                           Place place) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int g = threadIdx.x; g < G; g += blockDim.x) {
    uint32_t at = base(g);
    for (int w = 0; w < warps; ++w) {
      const uint32_t c = cnt[w * G + g];
      cnt[w * G + g] = at;
      at += c;
    }
  }
  __syncthreads();
  uint32_t* mine = cnt + warp * G;
  const int end = (warp + 1) * run < n ? (warp + 1) * run : n;
  for (int e0 = warp * run; e0 < end; e0 += 32) {
    const int e = e0 + lane;
    const int k = e < end ? key(e) : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, k);
    const uint32_t below = same & lanes_below(lane);
    if (k >= 0) place(e, mine[k] + __popc(below));
    __syncwarp();
    if (k >= 0 && below == 0) mine[k] += __popc(same);
    __syncwarp();
  }
}

// Exclusive scan of one value per thread over the block (at most 1024 threads);
// s_warp holds 33 words. Ends with a barrier.
__device__ __forceinline__ uint32_t block_scan_u32(uint32_t v, uint32_t* s_warp, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = lane < warps ? s_warp[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, w, d);
      if (lane >= d) w += y;
    }
    if (lane < warps) s_warp[lane] = w;
    if (lane == warps - 1) s_warp[32] = w;
  }
  __syncthreads();
  const uint32_t before = warp > 0 ? s_warp[warp - 1] : 0;
  *total = s_warp[32];
  __syncthreads();
  return before + x - v;
}

}  // namespace pgg
