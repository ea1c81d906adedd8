// What the tensor-core kernels of the 4-bit products share: how rows of x are laid out and fetched.
#pragma once

#include <cstdint>

#include "pgg_block.h"
#include "pgg_ptx.cuh"
#include "pgg_vec.cuh"

namespace pgg {

// The largest |x| of a row over its 128 threads, and (rest, 0 for each thread whose values are finite)
// whether it holds an infinity or NaN; the largest is then 1.
__device__ __forceinline__ float row_max(float v, float rest, float* s, bool* infinite) {
  const bool bad = __any_sync(0xFFFFFFFFu, rest != 0.0f);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = bad ? -1.0f : v;
  __syncthreads();
  *infinite = fminf(fminf(s[0], s[1]), fminf(s[2], s[3])) < 0.0f;
  return *infinite ? 1.0f : fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
}

constexpr int kListed = 512;  // positions of infinities that a block keeps

// The results of a row of x that holds infinities or NaN, by the definition: each element that is not
// finite times its weight, and beside these sums the rest counts nothing. (The products take code and
// zero, or the weight's two parts, one by one: inf code - inf zero and inf 0 are NaN where the weight
// times inf is not.) 128 threads, a column (gated: two) each in turn; the order of the terms does not
// show in the sum. x: the row; row, pos: its places in the outputs; g: its expert.
template <int DT>
__device__ __noinline__ void write_infinite_row(const W4Args& a, const uint16_t* x, int64_t g,
                                                int64_t row, int64_t pos) {
  __shared__ int s_at[kListed], s_count;
  const bool gated = a.product == PGG_W4_GATED;
  if (threadIdx.x == 0) s_count = 0;
  __syncthreads();
  bool nan = false;
  for (int64_t k = threadIdx.x; k < a.K; k += 128) {
    const float v = vec::load1<DT>(x, k);
    if (fabsf(v) < INFINITY) continue;
    nan = nan || v != v;
    const int at = atomicAdd(&s_count, 1);
    if (at < kListed) s_at[at] = static_cast<int>(k);
  }
  nan = __syncthreads_or(nan) != 0;
  const bool listed = s_count <= kListed;
  const int n = listed ? s_count : static_cast<int>(a.K);
  const int64_t columns = gated ? 2 * a.N : a.N;
  auto sum_of = [&](int64_t c) {
    const int64_t col = g * columns + c;
    float sum = nan ? NAN : 0.0f;
    for (int i = 0; i < n && sum == sum; ++i) {
      const int k = listed ? s_at[i] : i;
      const float v = vec::load1<DT>(x, k);
      if (fabsf(v) < INFINITY) continue;
      const int64_t q = col * a.groups + k / a.group;
      const int code = (a.codes[col * a.row_bytes + (k >> 1)] >> (4 * (k & 1))) & 15;
      const float scale =
          a.scale_f32 ? static_cast<const float*>(a.scales)[q] : vec::load1<DT>(a.scales, q);
      sum += scale * static_cast<float>(code - (a.zeros ? a.zeros[q] : 8)) * v;
    }
    return sum;
  };
  const int64_t out = (a.product == PGG_W4_COMBINED ? pos : row) * a.N;
  for (int64_t c = threadIdx.x; c < a.N; c += 128) {
    float v = sum_of(c);
    if (gated)
      v = (a.probs ? a.probs[pos] : 1.0f) * (v / (1.0f + expf(-v)) * sum_of(a.N + c));
    if (a.out_f32)
      static_cast<float*>(a.out)[out + c] = v;
    else
      vec::store1<DT>(a.out, out + c, v);
  }
  __syncthreads();  // (s_at and s_count are the next such row's)
}

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          ptx::smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(ptx::smem_addr(bar))
      : "memory");
}

}  // namespace pgg
