// The router of a mixture of experts: top-k choice from the logits, routing
// weights, and the expanded order (expandedRowIdx, groupList) that the grouped
// products read; and the gradient of the weights for the logits.
//
//     score    = softmax(logits) over all experts, or sigmoid(logits)
//     key[e]   = logit[e] + bias[e], or score[e] + bias[e]   (bias takes part in the choice only)
//     chosen   = the k largest keys, the lowest index first among equals
//     prob[j]  = scale * score[chosen_j]  (/ sum over the chosen when renormalised)
//     rows     = the pairs (token, j) sorted by (expert, token * k + j)
//
// A warp takes four tokens (or two, or one): the logits sit in registers, G / 8
// a lane; see choose_and_write in pgg_route_choose.cuh (65536 tokens, 256 experts,
// k 8, bf16: 25 to 27 us, by score + bias 48). A
// NaN key sorts below everything (the choice stays a valid one); scores follow IEEE
// arithmetic, so a softmax over a NaN or +inf logit gives NaN weights, whether that
// one is chosen or not. A masked expert (-inf) has weight 0; a token whose experts
// are all masked takes the lowest indices with weights 0. Everything is computed in
// 32 bits.
//
// Few tokens: one block does everything in one launch. Many: (1) choice, ranks
// and the block's count of every expert, (2) prefix sums of the counts over the
// blocks, (3) placement. The order is a stable counting sort, so the result
// depends on no atomic's order. What bounds the large case is instruction
// issue in the choice, not the 2 or 4 bytes read per logit.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pgg_ops.h"
#include "pgg_ptx.cuh"
#include "pgg_route_choose.cuh"
#include "pgg_sort.cuh"

namespace pgg {
namespace {

// (2) One warp per expert: exclusive prefix sums over the blocks, and the total.
__global__ void __launch_bounds__(32 * kWarps) count_scan_kernel(uint32_t* counts, int G,
                                                                 int blocks, int64_t* groups) {
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int g = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (g >= G) return;
  uint32_t* row = counts + static_cast<int64_t>(g) * blocks;
  uint32_t v[kMaxBlocks / 32];  // all loads at once: their latency is what this launch costs
#pragma unroll
  for (int i = 0; i < kMaxBlocks / 32; ++i) {
    const int b = 32 * i + lane;
    v[i] = b < blocks ? row[b] : 0u;
  }
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < kMaxBlocks / 32; ++i) {
    if (32 * i >= blocks) break;
    uint32_t x = v[i];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x += y;
    }
    if (32 * i + lane < blocks) row[32 * i + lane] = sum + x - v[i];
    sum += __shfl_sync(0xFFFFFFFFu, x, 31);
  }
  if (lane == 0) groups[g] = sum;
}

// (3) Placement of the block's pairs: the expert's first row, the pairs of the blocks before, the
// rank in the block.
__global__ void __launch_bounds__(32 * kWarps) route_place_kernel(const RouteArgs a) {
  extern __shared__ uint32_t s_base[];  // [G]
  __shared__ uint32_t s_scan[33];
  ptx::griddep_wait();
  uint32_t before = 0;
  for (int g0 = 0; g0 < a.G; g0 += blockDim.x) {
    const int g = g0 + threadIdx.x;
    const uint32_t c = g < a.G ? static_cast<uint32_t>(a.groups[g]) : 0u;
    const uint32_t here =
        g < a.G ? a.counts[static_cast<int64_t>(g) * a.blocks + blockIdx.x] : 0u;
    uint32_t total;
    const uint32_t at = block_scan_u32(c, s_scan, &total);
    if (g < a.G) s_base[g] = before + at + here;
    before += total;
  }
  __syncthreads();
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block * a.k;
  const int64_t p1 = p0 + static_cast<int64_t>(a.tokens_per_block) * a.k;
#pragma unroll 4
  for (int64_t p = p0 + threadIdx.x; p < (p1 < a.T * a.k ? p1 : a.T * a.k); p += blockDim.x)
    write_place(a, p, s_base[a.experts[p]] + a.rank[p]);
}

template <int DT>
__device__ __forceinline__ void store_grad(void* p, int64_t i, float v) {
  if constexpr (DT == PGG_F32) static_cast<float*>(p)[i] = v;
  if constexpr (DT == PGG_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  if constexpr (DT == PGG_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// A warp's zeros over a row of `bytes` (a multiple of 2), in the widest words that its address allows.
__device__ __forceinline__ void zero_row(char* p, int bytes, int lane) {
  const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) | bytes;
  if (low % 16 == 0) {
    for (int i = 16 * lane; i < bytes; i += 512)
      *reinterpret_cast<uint4*>(p + i) = make_uint4(0, 0, 0, 0);
  } else if (low % 4 == 0) {
    for (int i = 4 * lane; i < bytes; i += 128) *reinterpret_cast<uint32_t*>(p + i) = 0;
  } else {
    for (int i = 2 * lane; i < bytes; i += 64) *reinterpret_cast<uint16_t*>(p + i) = 0;
  }
}

// ------------------------------------------------------------------ gradient
//
//   softmax:                d_logit = s (ds - sum_e ds_e s_e), ds = scale * d_prob at the chosen
//   softmax, renormalised:  d_logit_j = scale * p_j (d_prob_j - sum_i d_prob_i p_i), chosen only
//   sigmoid:                d_logit_j = ds_j s_j (1 - s_j), ds = scale * d_prob
//   sigmoid, renormalised:  the same with ds_j = scale * (d_prob_j - sum_i d_prob_i p_i) / sum s
//
// One warp per token. Only the plain softmax reads the row and fills it with values; the others
// write zeros in wide words and then the chosen (31712 tokens, 384 experts, bf16: 16 us; through a
// row in shared memory 39). A row with a chosen index outside the experts, or one chosen twice,
// has no gradient: it is filled with NaN.
template <int DT, int V>
__global__ void __launch_bounds__(32 * kWarps) route_grad_kernel(const RouteGradArgs a) {
  extern __shared__ float s_row[];  // [warps][G]: ds of the chosen, 0 elsewhere
  constexpr int kSize = DT == PGG_F32 ? 4 : 2;
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* ds = s_row + warp * a.G;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t row = t * a.G;
    const bool on = lane < a.k;
    const int64_t e64 = on ? a.experts[t * a.k + lane] : 0;
    const float dp = on ? a.d_probs[t * a.k + lane] * a.scale : 0.0f;
    float l[V];
    if (!a.sigmoid && !a.renormalize) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        l[i] = lane + 32 * i < a.G ? load_logit<DT>(a.logits, row + lane + 32 * i) : -INFINITY;
    }
    const bool sparse = a.sigmoid || a.renormalize;
    if (!sparse)
      for (int i = lane; i < a.G; i += 32) ds[i] = 0.0f;
    const bool in = e64 >= 0 && e64 < a.G;
    const int e = in ? static_cast<int>(e64) : 0;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, on ? e : -1 - lane);
    const bool bad = __any_sync(0xFFFFFFFFu, on && (!in || __popc(same) > 1));
    const float lj = sparse && on ? load_logit<DT>(a.logits, row + e) : -INFINITY;
    if (sparse) {
      __syncwarp();  // (d_logits may be logits: all of the warp have read theirs)
      zero_row(static_cast<char*>(a.d_logits) + row * kSize, a.G * kSize, lane);
    }
    __syncwarp();
    if (bad) {
      for (int i = lane; i < a.G; i += 32) ds[i] = NAN;
    } else if (sparse) {
      float p, w;  // normalised weight, and d(weight before normalising) / d(logit) over the sum
      if (a.sigmoid) {
        const float s = on ? sigmoid(lj) : 0.0f;
        if (a.renormalize) {
          const float z = warp_sum(s);
          p = z == 0.0f ? 0.0f : s / z;
          w = p * sigmoid(-lj);  // 1 - s without its cancellation
        } else {
          p = 0.0f;
          w = s * sigmoid(-lj);
        }
      } else {
        const float m = warp_max(lj);
        p = on ? soft_exp(lj, m) : 0.0f;
        const float z = warp_sum(p);
        p = m == -INFINITY && z == 0.0f ? 0.0f : p / z;
        w = p;
      }
      const float dot = a.renormalize ? warp_sum(on ? dp * p : 0.0f) : 0.0f;
      // (the zeros of the other lanes came before: __syncwarp orders them)
      if (on) store_grad<DT>(a.d_logits, row + e, w * (dp - dot));
      continue;
    } else {
      float m = -INFINITY, z = 0.0f, dot = 0.0f;
      if (on) ds[e] = dp;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
      m = warp_max(m);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        l[i] = lane + 32 * i < a.G ? soft_exp(l[i], m) : 0.0f;
        z += l[i];
      }
      z = warp_sum(z);
      const float inv = m == -INFINITY && z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        l[i] *= inv;
        if (lane + 32 * i < a.G) dot += ds[lane + 32 * i] * l[i];
      }
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < a.G) ds[lane + 32 * i] = l[i] * (ds[lane + 32 * i] - dot);
    }
    __syncwarp();
    for (int i = lane; i < a.G; i += 32) {
      store_grad<DT>(a.d_logits, row + i, ds[i]);
    }
    __syncwarp();
  }
}

int log2_slots(int G) {
  int v = 1, i = 0;
  while (v * 32 < G) v *= 2, ++i;
  return i;
}

template <int DT>
cudaError_t launch_route_d(const RouteArgs& a, cudaStream_t stream) {
  // four or two tokens a warp where a quarter's or half's lanes are enough for the choices and the
  // logits
  if (a.k <= 8 && a.G <= 256) {
    if (a.G <= 32) return launch_route_t<DT, 4, 8, false>(a, stream);
    if (a.G <= 64) return launch_route_t<DT, 8, 8, false>(a, stream);
    if (a.G <= 128) return launch_route_t<DT, 16, 8, false>(a, stream);
    return launch_route_t<DT, 32, 8, false>(a, stream);
  }
  if (a.k <= 16 && a.G <= 512) {
    if (a.G <= 32) return launch_route_t<DT, 2, 16, false>(a, stream);
    if (a.G <= 64) return launch_route_t<DT, 4, 16, false>(a, stream);
    if (a.G <= 128) return launch_route_t<DT, 8, 16, false>(a, stream);
    if (a.G <= 256) return launch_route_t<DT, 16, 16, false>(a, stream);
    return launch_route_t<DT, 32, 16, false>(a, stream);
  }
  return launch_route_t<DT, 32, 32, false>(a, stream);
}

}  // namespace

cudaError_t launch_count_scan(uint32_t* counts, int G, int blocks, int64_t* groups,
                              cudaStream_t stream) {
  return launch_pdl(count_scan_kernel, dim3((G + kWarps - 1) / kWarps), dim3(32 * kWarps), 0,
                    stream, 1, counts, G, blocks, groups);
}

// Blocks of the choice and placement launches: one when all the pairs fit one
// block, else at most kMaxBlocks.
void route_blocks(int64_t T, int64_t G, int64_t k, int* blocks, int* tokens_per_block) {
  if (T * k <= kSmallEntries && T <= 256) {
    *blocks = 1;
    *tokens_per_block = static_cast<int>(T);
    return;
  }
  int64_t per = (T + kMaxBlocks - 1) / kMaxBlocks;
  per = (per + 3) / 4 * 4;  // whole steps of a warp
  *tokens_per_block = static_cast<int>(per);
  *blocks = static_cast<int>((T + per - 1) / per);
}

// The third launch, of any type.
cudaError_t launch_route_place(const RouteArgs& a, cudaStream_t stream) {
  return launch_pdl(route_place_kernel, dim3(a.blocks), dim3(32 * kWarps),
                    static_cast<size_t>(a.G) * 4, stream, 1, a);
}

cudaError_t launch_route(int dtype, const RouteArgs& a, cudaStream_t stream) {
  if (a.bias_on_score) return launch_route_scores(dtype, a, stream);
  if (dtype == PGG_F32) return launch_route_d<PGG_F32>(a, stream);
  if (dtype == PGG_F16) return launch_route_d<PGG_F16>(a, stream);
  if (dtype == PGG_BF16) return launch_route_d<PGG_BF16>(a, stream);
  return cudaErrorInvalidValue;
}

namespace {

template <int DT>
cudaError_t launch_route_grad_t(const RouteGradArgs& a, int num_sms, cudaStream_t stream) {
  using K = void (*)(const RouteGradArgs);
  static const K kern[6] = {route_grad_kernel<DT, 1>, route_grad_kernel<DT, 2>,
                            route_grad_kernel<DT, 4>, route_grad_kernel<DT, 8>,
                            route_grad_kernel<DT, 16>, route_grad_kernel<DT, 32>};
  int64_t blocks = (a.T + kWarps - 1) / kWarps;
  const int64_t cap = static_cast<int64_t>(num_sms) * 8;
  if (blocks > cap) blocks = cap;
  return launch_pdl(kern[log2_slots(a.G)], dim3(static_cast<unsigned>(blocks)), dim3(32 * kWarps),
                    static_cast<size_t>(kWarps) * a.G * 4, stream, 1, a);
}

}  // namespace

cudaError_t launch_route_grad(int dtype, const RouteGradArgs& a, int num_sms,
                              cudaStream_t stream) {
  if (dtype == PGG_F32) return launch_route_grad_t<PGG_F32>(a, num_sms, stream);
  if (dtype == PGG_F16) return launch_route_grad_t<PGG_F16>(a, num_sms, stream);
  if (dtype == PGG_BF16) return launch_route_grad_t<PGG_BF16>(a, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pgg
