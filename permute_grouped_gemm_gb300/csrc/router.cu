// The router of a mixture of experts: top-k choice from the logits, routing
// weights, and the expanded order (expandedRowIdx, groupList) that the grouped
// products read; and the gradient of the weights for the logits.
//
//     key[e]   = logit[e] + bias[e]          (bias takes part in the choice only)
//     chosen   = the k largest keys, the lowest index first among equals
//     score    = softmax(logits) over all experts, or sigmoid(logits)
//     prob[j]  = scale * score[chosen_j]  (/ sum over the chosen when renormalised)
//     rows     = the pairs (token, j) sorted by (expert, token * k + j)
//
// A warp takes one token: its logits sit in registers (G / 32 a lane) as
// sortable integers, and each of the k rounds is a lane-local maximum, one
// warp-wide integer maximum of the keys and one minimum of the index. A NaN key
// sorts below everything (the choice stays a valid one); scores follow IEEE
// arithmetic, so a NaN or +inf logit gives NaN weights. A masked expert
// (-inf) has weight 0; a token whose experts are all masked takes the lowest
// indices with weights 0. Everything is computed in 32 bits.
//
// Few tokens: one block does everything in one launch. Many: (1) choice and
// the block's count of every expert, (2) prefix sums of the counts over the
// blocks, (3) placement. The order is a stable counting sort, so the result
// depends on no atomic's order. What bounds the large case is instruction
// issue in the k rounds of the choice, not the 2 or 4 bytes read per logit.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pgg_ops.h"
#include "pgg_ptx.cuh"
#include "pgg_sort.cuh"

namespace pgg {
namespace {

constexpr int kWarps = 8;           // of the choice, placement and gradient blocks
constexpr int kSmallEntries = 2048; // one block does it all up to this many (token, j) pairs
constexpr int kSmallThreads = 1024;

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (DT == PGG_F32) return static_cast<const float*>(p)[i];
  if constexpr (DT == PGG_F16) return __half2float(static_cast<const __half*>(p)[i]);
  if constexpr (DT == PGG_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Order-preserving map of a float to an integer: NaN -> 0, -inf -> 1 or more,
// -0 and +0 to the same.
__device__ __forceinline__ uint32_t sort_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  return v;
}

// exp(l - m) of a softmax whose maximum is m; -inf gives 0 even when nothing else is there
__device__ __forceinline__ float soft_exp(float l, float m) {
  return l == -INFINITY ? 0.0f : expf(l - m);
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Chooses token t's experts with one warp: lane j < k returns expert and weight j.
template <int DT, int V>
__device__ __forceinline__ void choose(const RouteArgs& a, int64_t t, int lane, int* expert,
                                       float* prob) {
  float l[V];
  uint32_t key[V];
  float m = -INFINITY;
  const int64_t row = t * a.G;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < a.G ? load_logit<DT>(a.logits, row + e) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    m = fmaxf(m, l[i]);
    // keys are shifted up by one (NaN 1), so that 0 marks what is taken or not there
    key[i] = e < a.G ? sort_key(a.bias ? l[i] + a.bias[e] : l[i]) : 0u;
    if (e < a.G && key[i] == 0u) key[i] = 1u;
  }
  // what was chosen: lane j keeps round j's expert and logit
  int my_e = 0;
  float my_l = -INFINITY;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0;
    int slot = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        slot = i;
      }
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    const uint32_t idx = __reduce_min_sync(
        0xFFFFFFFFu, best == top ? static_cast<uint32_t>(lane + 32 * slot) : 0xFFFFFFFFu);
    const int owner = static_cast<int>(idx & 31u), oslot = static_cast<int>(idx >> 5);
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i == oslot) {
        v = l[i];
        if (lane == owner) key[i] = 0u;
      }
    v = __shfl_sync(0xFFFFFFFFu, v, owner);
    if (lane == j) {
      my_e = static_cast<int>(idx);
      my_l = v;
    }
  }
  float p;
  if (a.sigmoid) {
    p = lane < a.k ? sigmoid(my_l) : 0.0f;
    if (a.renormalize) {
      const float z = warp_sum(p);
      p = z == 0.0f ? 0.0f : p / z;
    }
  } else if (a.renormalize) {
    // softmax over the chosen alone: the others' part cancels
    const float mc = warp_max(lane < a.k ? my_l : -INFINITY);
    p = lane < a.k ? soft_exp(my_l, mc) : 0.0f;
    const float z = warp_sum(p);
    p = mc == -INFINITY && z == 0.0f ? 0.0f : p / z;
  } else {
    m = warp_max(m);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < a.G) z += soft_exp(l[i], m);
    z = warp_sum(z);
    p = m == -INFINITY && z == 0.0f ? 0.0f : soft_exp(my_l, m) / z;
  }
  *expert = my_e;
  *prob = p * a.scale;
}

template <int DT, int V>
__device__ __forceinline__ void choose_and_write(const RouteArgs& a, int64_t t, int lane,
                                                 int* s_expert) {
  int e;
  float p;
  choose<DT, V>(a, t, lane, &e, &p);
  if (lane < a.k) {
    a.experts[t * a.k + lane] = e;
    a.probs[t * a.k + lane] = p;
    s_expert[lane] = e;
  }
}

__device__ __forceinline__ void write_place(const RouteArgs& a, int64_t p, int64_t row) {
  if (a.row_idx_type == 0)
    a.idx[row] = p;
  else
    a.idx[p] = row;
}

// Everything in one block.
template <int DT, int V>
__global__ void __launch_bounds__(kSmallThreads) route_small_kernel(const RouteArgs a) {
  extern __shared__ uint32_t s_cnt[];  // [warps][G], then the entries' experts
  __shared__ uint32_t s_scan[33];
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int* s_expert = reinterpret_cast<int*>(s_cnt + warps * a.G);
  const int T = static_cast<int>(a.T), n = T * a.k;
  for (int t = warp; t < T; t += warps) choose_and_write<DT, V>(a, t, lane, s_expert + t * a.k);
  __syncthreads();
  const int run = ((n + warps - 1) / warps + 31) / 32 * 32;
  auto key = [&](int e) { return s_expert[e]; };
  sort_count(s_cnt, a.G, n, run, key);
  const int g = threadIdx.x;
  if (g == 0) a.hdr->status = 0;
  uint32_t c = 0;
  if (g < a.G) {
    for (int w = 0; w < warps; ++w) c += s_cnt[w * a.G + g];
    a.groups[g] = c;
  }
  uint32_t total;
  const uint32_t at = block_scan_u32(c, s_scan, &total);
  // blockDim >= G: thread g is the one that asks for key g's base
  sort_place(
      s_cnt, a.G, n, run, key, [&](int) { return at; },
      [&](int e, uint32_t where) { write_place(a, e, where); });
}

// (1) Choice, and the block's count of every expert.
template <int DT, int V>
__global__ void __launch_bounds__(32 * kWarps) route_choose_kernel(const RouteArgs a) {
  extern __shared__ uint32_t s_cnt[];  // [G]
  __shared__ int s_expert[kWarps][kMaxRouteTopK];
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int g = threadIdx.x; g < a.G; g += blockDim.x) s_cnt[g] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->status = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block;
  const int64_t t1 = t0 + a.tokens_per_block < a.T ? t0 + a.tokens_per_block : a.T;
  for (int64_t t = t0 + warp; t < t1; t += kWarps) {
    choose_and_write<DT, V>(a, t, lane, s_expert[warp]);
    __syncwarp();
    // (integer counts: the order of these additions changes nothing)
    if (lane < a.k) atomicAdd(&s_cnt[s_expert[warp][lane]], 1u);
    __syncwarp();
  }
  __syncthreads();
  for (int g = threadIdx.x; g < a.G; g += blockDim.x)
    a.counts[static_cast<int64_t>(g) * a.blocks + blockIdx.x] = s_cnt[g];
}

// (2) One warp per expert: exclusive prefix sums over the blocks, and the total.
__global__ void __launch_bounds__(32 * kWarps) count_scan_kernel(uint32_t* counts, int G,
                                                                 int blocks, int64_t* groups) {
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int g = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (g >= G) return;
  uint32_t* row = counts + static_cast<int64_t>(g) * blocks;
  uint32_t sum = 0;
  for (int b0 = 0; b0 < blocks; b0 += 32) {
    const int b = b0 + lane;
    const uint32_t v = b < blocks ? row[b] : 0u;
    uint32_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x += y;
    }
    if (b < blocks) row[b] = sum + x - v;
    sum += __shfl_sync(0xFFFFFFFFu, x, 31);
  }
  if (lane == 0) groups[g] = sum;
}

// (3) Placement of the block's entries.
__global__ void __launch_bounds__(32 * kWarps) route_place_kernel(const RouteArgs a) {
  extern __shared__ uint32_t s_cnt[];  // [warps][G], then [G] bases
  __shared__ uint32_t s_scan[33];
  ptx::griddep_wait();
  uint32_t* s_base = s_cnt + kWarps * a.G;
  uint32_t before = 0;
  for (int g0 = 0; g0 < a.G; g0 += blockDim.x) {
    const int g = g0 + threadIdx.x;
    const uint32_t c = g < a.G ? static_cast<uint32_t>(a.groups[g]) : 0u;
    uint32_t total;
    const uint32_t at = block_scan_u32(c, s_scan, &total);
    if (g < a.G)
      s_base[g] = before + at + a.counts[static_cast<int64_t>(g) * a.blocks + blockIdx.x];
    before += total;
  }
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block * a.k;
  const int64_t left = a.T * a.k - p0;
  const int most = a.tokens_per_block * a.k;
  const int n = left < most ? static_cast<int>(left) : most;
  const int run = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
  auto key = [&](int e) { return static_cast<int>(a.experts[p0 + e]); };
  sort_count(s_cnt, a.G, n, run, key);
  sort_place(
      s_cnt, a.G, n, run, key, [&](int g) { return s_base[g]; },
      [&](int e, uint32_t where) { write_place(a, p0 + e, where); });
}

// ------------------------------------------------------------------ gradient
//
//   softmax:                d_logit = s (ds - sum_e ds_e s_e), ds = scale * d_prob at the chosen
//   softmax, renormalised:  d_logit_j = scale * p_j (d_prob_j - sum_i d_prob_i p_i), chosen only
//   sigmoid:                d_logit_j = ds_j s_j (1 - s_j), ds = scale * d_prob
//   sigmoid, renormalised:  the same with ds_j = scale * (d_prob_j - sum_i d_prob_i p_i) / sum s
//
// One warp per token. The row is written whole; only the plain softmax reads
// it whole. A row with a chosen index outside the experts, or one chosen
// twice, has no gradient: it is filled with NaN.
template <int DT, int V>
__global__ void __launch_bounds__(32 * kWarps) route_grad_kernel(const RouteGradArgs a) {
  extern __shared__ float s_row[];  // [warps][G]: ds of the chosen, 0 elsewhere
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* ds = s_row + warp * a.G;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t row = t * a.G;
    for (int e = lane; e < a.G; e += 32) ds[e] = 0.0f;
    const bool on = lane < a.k;
    const int64_t e64 = on ? a.experts[t * a.k + lane] : 0;
    const bool in = e64 >= 0 && e64 < a.G;
    const int e = in ? static_cast<int>(e64) : 0;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, on ? e : -1 - lane);
    const bool bad = __any_sync(0xFFFFFFFFu, on && (!in || __popc(same) > 1));
    const float dp = on ? a.d_probs[t * a.k + lane] * a.scale : 0.0f;
    __syncwarp();
    if (bad) {
      for (int i = lane; i < a.G; i += 32) ds[i] = NAN;
    } else if (a.sigmoid || a.renormalize) {
      const float l = on ? load_logit<DT>(a.logits, row + e) : -INFINITY;
      float p, w;  // normalised weight, and d(weight before normalising) / d(logit) over the sum
      if (a.sigmoid) {
        const float s = on ? sigmoid(l) : 0.0f;
        if (a.renormalize) {
          const float z = warp_sum(s);
          p = z == 0.0f ? 0.0f : s / z;
          w = p * sigmoid(-l);  // 1 - s without its cancellation
        } else {
          p = 0.0f;
          w = s * sigmoid(-l);
        }
      } else {
        const float m = warp_max(l);
        p = on ? soft_exp(l, m) : 0.0f;
        const float z = warp_sum(p);
        p = m == -INFINITY && z == 0.0f ? 0.0f : p / z;
        w = p;
      }
      const float dot = a.renormalize ? warp_sum(on ? dp * p : 0.0f) : 0.0f;
      if (on) ds[e] = w * (dp - dot);
    } else {
      float l[V], m = -INFINITY, z = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        l[i] = lane + 32 * i < a.G ? load_logit<DT>(a.logits, row + lane + 32 * i) : -INFINITY;
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
      if constexpr (DT == PGG_F32) static_cast<float*>(a.d_logits)[row + i] = ds[i];
      if constexpr (DT == PGG_F16)
        static_cast<__half*>(a.d_logits)[row + i] = __float2half_rn(ds[i]);
      if constexpr (DT == PGG_BF16)
        static_cast<__nv_bfloat16*>(a.d_logits)[row + i] = __float2bfloat16_rn(ds[i]);
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
cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t stream) {
  using K = void (*)(const RouteArgs);
  static const K small[6] = {route_small_kernel<DT, 1>, route_small_kernel<DT, 2>,
                             route_small_kernel<DT, 4>, route_small_kernel<DT, 8>,
                             route_small_kernel<DT, 16>, route_small_kernel<DT, 32>};
  static const K many[6] = {route_choose_kernel<DT, 1>, route_choose_kernel<DT, 2>,
                            route_choose_kernel<DT, 4>, route_choose_kernel<DT, 8>,
                            route_choose_kernel<DT, 16>, route_choose_kernel<DT, 32>};
  const int v = log2_slots(a.G);
  if (a.blocks == 1) {
    // threads for the tokens and for the experts' scan, no more: fewer counters to clear
    int threads = static_cast<int>(a.T < 32 ? a.T : 32) * 32;
    const int for_scan = (a.G + 31) / 32 * 32;
    if (threads < for_scan) threads = for_scan;
    const size_t smem = (static_cast<size_t>(threads / 32) * a.G + a.T * a.k) * 4;
    cudaError_t err = cudaFuncSetAttribute(small[v], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    return launch_pdl(small[v], dim3(1), dim3(threads), smem, stream, 1, a);
  }
  cudaError_t err = launch_pdl(many[v], dim3(a.blocks), dim3(32 * kWarps),
                               static_cast<size_t>(a.G) * 4, stream, 1, a);
  if (err != cudaSuccess) return err;
  err = launch_count_scan(a.counts, a.G, a.blocks, a.groups, stream);
  if (err != cudaSuccess) return err;
  return launch_pdl(route_place_kernel, dim3(a.blocks), dim3(32 * kWarps),
                    static_cast<size_t>(kWarps + 1) * a.G * 4, stream, 1, a);
}

}  // namespace

cudaError_t launch_count_scan(uint32_t* counts, int G, int blocks, int64_t* groups,
                              cudaStream_t stream) {
  return launch_pdl(count_scan_kernel, dim3((G + kWarps - 1) / kWarps), dim3(32 * kWarps), 0,
                    stream, 1, counts, G, blocks, groups);
}

// Blocks of the choice and placement launches: one when all the pairs fit one
// block, else at most 1024 with a multiple of the block's warps of tokens each.
void route_blocks(int64_t T, int64_t G, int64_t k, int* blocks, int* tokens_per_block) {
  if (T * k <= kSmallEntries && T <= 256) {
    *blocks = 1;
    *tokens_per_block = static_cast<int>(T);
    return;
  }
  int64_t per = (T + 1023) / 1024;
  per = (per + kWarps - 1) / kWarps * kWarps;
  *tokens_per_block = static_cast<int>(per);
  *blocks = static_cast<int>((T + per - 1) / per);
}

cudaError_t launch_route(int dtype, const RouteArgs& a, cudaStream_t stream) {
  if (dtype == PGG_F32) return launch_route_t<PGG_F32>(a, stream);
  if (dtype == PGG_F16) return launch_route_t<PGG_F16>(a, stream);
  if (dtype == PGG_BF16) return launch_route_t<PGG_BF16>(a, stream);
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
