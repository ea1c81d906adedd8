// Sums over the threads of a block.
#pragma once

#include <cstdint>

namespace pgg {

// Sums of K values (1, 3, 4 or 8) over the block, the same bits in every thread. Two buffers in
// turn, so that one barrier a call is enough. Several values are added together: after two exchanges
// a lane goes on with one of four, so that it takes 6 shuffles, not 20, before the barrier and 7
// after (of eight: three exchanges, 9 and 10).
template <int K>
struct BlockSum {
  float part[2][32][K == 1 ? 1 : K <= 4 ? 4 : 8];
};

template <int K, int M>
__device__ __forceinline__ void block_sum(BlockSum<M>* s, int* turn, float (&v)[K]) {
  static_assert(K <= M && (K == 1 || K == 3 || K == 4 || K == 8), "room, and how many at a time");
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if constexpr (K == 1) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v[0] += __shfl_xor_sync(kAll, v[0], d);
    if (warps == 1) return;
    if (lane == 0) s->part[*turn][warp][0] = v[0];
    __syncthreads();
    v[0] = lane < warps ? s->part[*turn][lane][0] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v[0] += __shfl_xor_sync(kAll, v[0], d);
  } else if constexpr (K == 8) {
    // lane bits 0, 1, 2 pick the upper or lower half of what is left: value 4 b0 + 2 b1 + b2
    const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
    float h[4], q[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = (b0 ? v[i + 4] : v[i]) + __shfl_xor_sync(kAll, b0 ? v[i] : v[i + 4], 1);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      q[i] = (b1 ? h[i + 2] : h[i]) + __shfl_xor_sync(kAll, b1 ? h[i] : h[i + 2], 2);
    float x = (b2 ? q[1] : q[0]) + __shfl_xor_sync(kAll, b2 ? q[0] : q[1], 4);
#pragma unroll
    for (int d = 8; d < 32; d *= 2) x += __shfl_xor_sync(kAll, x, d);
    if (warps > 1) {
      if (lane < 8) s->part[*turn][warp][lane] = x;
      __syncthreads();
      x = 0.0f;
      for (int w = lane >> 3; w < warps; w += 4) x += s->part[*turn][w][lane & 7];
#pragma unroll
      for (int d = 8; d < 32; d *= 2) x += __shfl_xor_sync(kAll, x, d);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = __shfl_sync(kAll, x, (i >> 2 & 1) | (i & 2) | (i & 1) << 2);
  } else {
    // lane bit 0 picks values {0, 1} or {2, 3}, bit 1 one of the two
    const float v2 = v[2], v3 = K > 3 ? v[K - 1] : 0.0f;
    const bool b0 = lane & 1, b1 = lane & 2;
    float x = (b0 ? v2 : v[0]) + __shfl_xor_sync(kAll, b0 ? v[0] : v2, 1);
    float y = (b0 ? v3 : v[1]) + __shfl_xor_sync(kAll, b0 ? v[1] : v3, 1);
    x = (b1 ? y : x) + __shfl_xor_sync(kAll, b1 ? x : y, 2);
#pragma unroll
    for (int d = 4; d < 32; d *= 2) x += __shfl_xor_sync(kAll, x, d);
    if (warps > 1) {
      if (lane < 4) s->part[*turn][warp][lane] = x;
      __syncthreads();
      x = 0.0f;
      for (int w = lane >> 2; w < warps; w += 8) x += s->part[*turn][w][lane & 3];
#pragma unroll
      for (int d = 4; d < 32; d *= 2) x += __shfl_xor_sync(kAll, x, d);
    }
    // lane 0: value 0, lane 2: value 1, lane 1: value 2, lane 3: value 3
    v[0] = __shfl_sync(kAll, x, 0);
    v[1] = __shfl_sync(kAll, x, 2);
    v[2] = __shfl_sync(kAll, x, 1);
    if constexpr (K > 3) v[K - 1] = __shfl_sync(kAll, x, 3);
  }
  *turn ^= 1;
}

}  // namespace pgg
