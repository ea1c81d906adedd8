// The router's choice of experts: device code and launches of route_small_kernel and
// route_choose_kernel, compiled in router.cu (choice by the logits) and in router_scores.cu (by
// score + bias). See router.cu for the operator.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pgg_ops.h"
#include "pgg_ops_launch.h"
#include "pgg_ptx.cuh"
#include "pgg_sort.cuh"

namespace pgg {
namespace {

constexpr int kWarps = 8;           // of the choice, placement and gradient blocks
constexpr int kSmallEntries = 2048; // one block does it all up to this many (token, j) pairs
constexpr int kSmallThreads = 512;
constexpr int kMaxBlocks = 608;     // of the choice and placement launches: four a multiprocessor

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (DT == PGG_F32) return static_cast<const float*>(p)[i];
  if constexpr (DT == PGG_F16) return __half2float(static_cast<const __half*>(p)[i]);
  if constexpr (DT == PGG_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Order-preserving map of a float (not -0) to an integer: NaN -> 1, -inf far above it.
__device__ __forceinline__ uint32_t sort_key(float f) {
  const int32_t u = __float_as_int(f);
  const uint32_t k = static_cast<uint32_t>(u ^ ((u >> 31) | static_cast<int32_t>(0x80000000)));
  return f != f ? 1u : k;
}

// Sum and maximum over groups of LPT lanes.
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = LPT / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = LPT / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  return v;
}

template <int LPT>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t v) {
  if constexpr (LPT == 32) {
    return __reduce_max_sync(0xFFFFFFFFu, v);
  } else {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) {
      const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
      v = o > v ? o : v;
    }
    return v;
  }
}

// The group's values (no NaN) in decreasing order, one a lane (a bitonic network).
template <int LPT>
__device__ __forceinline__ float sort_lanes(float v, int sl) {
#pragma unroll
  for (int size = 2; size <= LPT; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const float o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
      const bool larger = ((sl & d) == 0) == ((sl & size) == 0);
      v = larger ? fmaxf(v, o) : fminf(v, o);
    }
  return v;
}

// The same of two values a lane: 2 LPT in all, the 2 sl-th and the next in v0 and v1.
template <int LPT>
__device__ __forceinline__ void sort_lanes_two(float& v0, float& v1, int sl) {
#pragma unroll
  for (int size = 2; size <= 2 * LPT; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const bool down = (2 * sl & size) == 0;
      if (d == 1) {
        const float hi = fmaxf(v0, v1), lo = fminf(v0, v1);
        v0 = down ? hi : lo;
        v1 = down ? lo : hi;
      } else {
        const float o0 = __shfl_xor_sync(0xFFFFFFFFu, v0, d / 2);
        const float o1 = __shfl_xor_sync(0xFFFFFFFFu, v1, d / 2);
        const bool larger = ((2 * sl & d) == 0) == down;
        v0 = larger ? fmaxf(v0, o0) : fminf(v0, o0);
        v1 = larger ? fmaxf(v1, o1) : fminf(v1, o1);
      }
    }
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

// Maximum that is NaN when one of the two is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// What the bias is added to when it belongs to the scores: the score in fp32, -inf for a masked
// expert (or none). m and z: the softmax's maximum and sum. A candidate's key is worked out again
// from its logit, so each step is one rounding that the compiler may not merge with the sum.
__device__ __forceinline__ float score_of(float l, bool is_sigmoid, float m, float z) {
  const float s = is_sigmoid ? __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l)))
                             : __fdiv_rn(expf(__fsub_rn(l, m)), z);
  return l == -INFINITY ? -INFINITY : s;
}

// Where value i of lane sl of a token's LPT lanes sits in its row: VL neighbouring values a load,
// LPT VL a group of lanes.
template <int VL, int LPT>
__device__ __forceinline__ int expert_at(int i, int sl) {
  return (i / VL) * (LPT * VL) + sl * VL + i % VL;
}

// A row's logits, V a lane; -inf past the end. VL > 1: 4 VL or 2 VL bytes a load (G is a multiple
// of VL and the rows are aligned to it).
template <int DT, int V, int VL, int LPT>
__device__ __forceinline__ void load_row(const void* logits, int64_t row, int G, int sl,
                                         float (&l)[V]) {
  constexpr int kBytes = VL * (DT == PGG_F32 ? 4 : 2);
  if constexpr (VL == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      l[i] = expert_at<1, LPT>(i, sl) < G ? load_logit<DT>(logits, row + expert_at<1, LPT>(i, sl))
                                       : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += VL) {
      const int e = expert_at<VL, LPT>(i, sl);
      constexpr uint32_t kNone = DT == PGG_F32 ? 0xFF800000u : DT == PGG_BF16 ? 0xFF80FF80u
                                                                              : 0xFC00FC00u;
      uint32_t w[4] = {kNone, kNone, kNone, kNone};  // -inf
      if (e < G) {
        const char* p = static_cast<const char*>(logits) + (row + e) * (kBytes / VL);
        if constexpr (kBytes == 16) {
          const uint4 q = *reinterpret_cast<const uint4*>(p);
          w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else if constexpr (kBytes == 8) {
          const uint2 q = *reinterpret_cast<const uint2*>(p);
          w[0] = q.x, w[1] = q.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
#pragma unroll
      for (int c = 0; c < VL; ++c) {
        float f;
        if constexpr (DT == PGG_F32)
          f = __uint_as_float(w[c]);
        else if constexpr (DT == PGG_BF16)
          f = __uint_as_float(c % 2 ? w[c / 2] & 0xFFFF0000u : w[c / 2] << 16);
        else
          f = __half2float(__ushort_as_half(
              static_cast<unsigned short>(c % 2 ? w[c / 2] >> 16 : w[c / 2] & 0xFFFFu)));
        l[i + c] = f;
      }
    }
  }
}

// The bias in shared memory, in the order in which the lanes read it (value i of lane sl at
// i / 4 * 4 LPT + 4 sl + i % 4); 0 past the end.
template <int V, int VL, int LPT>
__device__ __forceinline__ void stage_bias(const RouteArgs& a, float* s_bias) {
  for (int j = threadIdx.x; j < V * LPT; j += blockDim.x) {
    const int c = V < 4 ? V : 4;
    const int i = j / (c * LPT) * c + j % c, sl = j / c % LPT;
    const int e = expert_at<VL, LPT>(i, sl);
    s_bias[j] = a.bias && e < a.G ? a.bias[e] : 0.0f;
  }
}

template <int V, int LPT>
__device__ __forceinline__ void add_bias(const float* s_bias, int sl, float (&l)[V]) {
  if constexpr (V < 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] += s_bias[V * sl + i];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 b = *reinterpret_cast<const float4*>(s_bias + i * LPT + 4 * sl);
      l[i] += b.x, l[i + 1] += b.y, l[i + 2] += b.z, l[i + 3] += b.w;
    }
  }
}

// A warp's scratch memory of the choice: the candidates of up to four tokens. (34 words apart, so
// that the tokens' broadcast reads of 16 bytes meet in different banks.)
constexpr int kCand = 32;
template <int LPT>
struct alignas(16) ChoiceScratch {
  uint64_t word[32 / LPT][kCand + 2];  // key above, the index's complement below: larger is first
  int expert[32 / LPT][kCand];
};

// The choice of 32 / LPT tokens from t0 on with one warp, LPT lanes each, written to probs,
// experts and s_expert [k] (a token at or past T writes nothing).
//
// The k-th largest of the lanes' maxima (of two halves each with 8 lanes) is at most the k-th
// largest key, so the chosen are among the keys that reach it: rarely more than k plus a few.
// Their indices are collected in shared memory, and the lanes, one a candidate, find each one's
// rank by counting those before it. Up to
// there the keys are floats (the maximum of two passes over a NaN, and no NaN reaches a
// threshold); only the few candidates become integers. Where too few lanes hold a key above -inf,
// or equal keys leave more than 32 candidates, the k rounds of a group-wide maximum are done
// instead. With two or four tokens a warp everything but the logits themselves is shared by them.
// Returns this lane's choice (its token's sl-th), -1 without one.
template <int DT, int V, int VL, int LPT, bool ON_SCORE>
__device__ __forceinline__ int choose_and_write(const RouteArgs& a, int64_t t0, int64_t t1,
                                                 int lane, const float* s_bias,
                                                 ChoiceScratch<LPT>* scratch, int* s_expert) {
  const int sl = lane % LPT, sub = lane / LPT;
  const int64_t t = t0 + sub < t1 ? t0 + sub : t1 - 1;  // (the last one again, not written)
  const bool there = t0 + sub < t1;
  uint64_t* const word = scratch->word[sub];
  int* const cand = scratch->expert[sub];
  s_expert += a.k * sub;
  float l[V];
  const int64_t row = t * a.G;
  load_row<DT, V, VL, LPT>(a.logits, row, a.G, sl, l);
  float m = -INFINITY, z = 0.0f;
  if (!a.sigmoid && (!a.renormalize || ON_SCORE)) {  // softmax over all
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
    m = group_max<LPT>(m);
#pragma unroll
    for (int i = 0; i < V; ++i) z += soft_exp(l[i], m);  // (0 past the end)
    z = group_sum<LPT>(z);
  }
  // a softmax over all with a NaN or +inf in it is NaN, which the sum over the chosen alone would
  // not show when that one is not chosen
  bool no_softmax = false;
  if (!a.sigmoid && a.renormalize) {
    float w = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) w = max_or_nan(w, l[i]);
    const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, !(w < INFINITY));
    no_softmax = ((lanes >> (LPT * sub)) & (0xFFFFFFFFu >> (32 - LPT))) != 0;
  }
  if constexpr (ON_SCORE) {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = score_of(l[i], a.sigmoid, m, z);
  }
  if (a.bias) add_bias<V, LPT>(s_bias, sl, l);
  float floor_key;
  if constexpr (LPT == 8) {
    float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) b0 = fmaxf(b0, l[i]), b1 = fmaxf(b1, l[V / 2 + i]);
    sort_lanes_two<LPT>(b0, b1, sl);
    floor_key = __shfl_sync(0xFFFFFFFFu, a.k & 1 ? b0 : b1, (a.k - 1) >> 1, LPT);
  } else {
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) best = fmaxf(best, l[i]);
    floor_key = __shfl_sync(0xFFFFFFFFu, sort_lanes<LPT>(best, sl), a.k - 1, LPT);
  }
  uint32_t mask = 0;  // this lane's candidates
#pragma unroll
  for (int i = 0; i < V; ++i) mask |= l[i] >= floor_key ? 1u << i : 0u;
  if (floor_key == -INFINITY) mask = 0;
  int upto = __popc(mask);
  int at = -upto;
#pragma unroll
  for (int d = 1; d < LPT; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, upto, d, LPT);
    if (sl >= d) upto += y;
  }
  at += upto;
  const int n = __shfl_sync(0xFFFFFFFFu, upto, LPT - 1, LPT);
  const bool few = n > 0 && n <= kCand;
  if (few) {
    for (; mask; mask &= mask - 1) cand[at++] = expert_at<VL, LPT>(__ffs(mask) - 1, sl);
  }
  __syncwarp();
  if (!__all_sync(0xFFFFFFFFu, few)) {
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      key[i] = expert_at<VL, LPT>(i, sl) < a.G ? sort_key(l[i] + 0.0f) : 0u;  // 0: not there
    for (int j = 0; j < a.k; ++j) {
      uint32_t top = 0, where = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) top = key[i] > top ? key[i] : top;
      top = group_max_u32<LPT>(top);
#pragma unroll
      for (int i = 0; i < V; ++i) {  // the lowest index: the largest complement
        const uint32_t x = ~static_cast<uint32_t>(expert_at<VL, LPT>(i, sl));
        if (key[i] == top && x > where) where = x;
      }
      where = ~group_max_u32<LPT>(where);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (static_cast<uint32_t>(expert_at<VL, LPT>(i, sl)) == where) key[i] = 0;
      if (!few && sl == 0) s_expert[j] = static_cast<int>(where);
    }
  }
  const int most = few ? n : 0;
  for (int c = sl; c < most + (most & 1); c += LPT) {  // (an even number: one of 0 is never before)
    uint64_t w = 0;
    if (c < most) {
      const int e = cand[c];
      const float b = a.bias ? a.bias[e] : 0.0f;  // (the sums of +0 are never -0)
      float f = load_logit<DT>(a.logits, row + e);
      if constexpr (ON_SCORE) f = score_of(f, a.sigmoid, m, z);
      w = static_cast<uint64_t>(sort_key(f + b + 0.0f)) << 32 |
          static_cast<uint32_t>(~e);
    }
    word[c] = w;
  }
  __syncwarp();
  constexpr int kPass = LPT < 16 ? 16 : LPT, kOwn = kPass / LPT;
  for (int c0 = 0; c0 < kCand; c0 += kPass) {
    if (!__any_sync(0xFFFFFFFFu, c0 < most)) break;
    uint64_t own[kOwn];
    int before[kOwn];
#pragma unroll
    for (int q = 0; q < kOwn; ++q) {
      const int c = c0 + q * LPT + sl;
      own[q] = c < most ? word[c] : 0;
      before[q] = c < most ? 0 : a.k;
    }
#pragma unroll 2
    for (int j = 0; j < most; j += 2) {
      const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(word + j);
#pragma unroll
      for (int q = 0; q < kOwn; ++q) before[q] += (w.x > own[q] ? 1 : 0) + (w.y > own[q] ? 1 : 0);
    }
#pragma unroll
    for (int q = 0; q < kOwn; ++q)
      if (before[q] < a.k) s_expert[before[q]] = static_cast<int>(~static_cast<uint32_t>(own[q]));
  }
  __syncwarp();
  const bool on = sl < a.k;
  const int e = on ? s_expert[sl] : 0;
  const float my_l = on ? load_logit<DT>(a.logits, row + e) : -INFINITY;
  float p;
  if (a.sigmoid) {
    p = on ? sigmoid(my_l) : 0.0f;
    if (a.renormalize) {
      z = group_sum<LPT>(p);
      p = z == 0.0f ? 0.0f : p / z;
    }
  } else if (a.renormalize) {
    // softmax over the chosen alone: the others' part cancels
    m = group_max<LPT>(my_l);
    p = on ? soft_exp(my_l, m) : 0.0f;
    z = group_sum<LPT>(p);
    p = m == -INFINITY && z == 0.0f ? 0.0f : p / z;
    if (no_softmax) p = NAN;
  } else {
    p = m == -INFINITY && z == 0.0f ? 0.0f : soft_exp(my_l, m) / z;
  }
  if (on && there) {
    a.experts[t * a.k + sl] = e;
    a.probs[t * a.k + sl] = p * a.scale;
  }
  return on && there ? e : -1;
}

__device__ __forceinline__ void write_place(const RouteArgs& a, int64_t p, int64_t row) {
  if (a.row_idx_type == 0)
    a.idx[row] = p;
  else
    a.idx[p] = row;
}

// Everything in one block.
template <int DT, int V, int VL, int LPT, bool ON_SCORE>
__global__ void __launch_bounds__(kSmallThreads) route_small_kernel(const RouteArgs a) {
  extern __shared__ uint32_t s_cnt[];  // [warps][G], the entries' experts, [G] bases
  __shared__ uint32_t s_scan[33];
  __shared__ ChoiceScratch<LPT> s_cand[kSmallThreads / 32];
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int* s_expert = reinterpret_cast<int*>(s_cnt + warps * a.G);
  const int T = static_cast<int>(a.T), n = T * a.k;
  __shared__ alignas(16) float s_bias[V * LPT];
  if (a.bias) {
    stage_bias<V, VL, LPT>(a, s_bias);
    __syncthreads();
  }
  constexpr int kTok = 32 / LPT;  // tokens of a warp at a time
  for (int t = kTok * warp; t < T; t += kTok * warps)
    choose_and_write<DT, V, VL, LPT, ON_SCORE>(a, t, T, lane, s_bias, &s_cand[warp],
                                               s_expert + t * a.k);
  __syncthreads();
  const int run = ((n + warps - 1) / warps + 31) / 32 * 32;
  auto key = [&](int e) { return s_expert[e]; };
  sort_count(s_cnt, a.G, n, run, key);
  if (threadIdx.x == 0) a.hdr->status = 0;
  uint32_t* s_base = reinterpret_cast<uint32_t*>(s_expert + n);
  uint32_t before = 0;
  for (int g0 = 0; g0 < a.G; g0 += blockDim.x) {
    const int g = g0 + threadIdx.x;
    uint32_t c = 0, total;
    if (g < a.G) {
      for (int w = 0; w < warps; ++w) c += s_cnt[w * a.G + g];
      a.groups[g] = c;
    }
    const uint32_t at = block_scan_u32(c, s_scan, &total);
    if (g < a.G) s_base[g] = before + at;
    before += total;
  }
  sort_place(
      s_cnt, a.G, n, run, key, [&](int g) { return s_base[g]; },
      [&](int e, uint32_t where) { write_place(a, e, where); });
}

// (1) Choice, every pair's rank among the block's pairs of its expert, and the block's count of
// every expert. A warp takes its tokens one after another and a token's choices are distinct, so a
// counter per warp and expert gives the ranks in order, without atomics; the warps' counts are then
// added up in their order.
template <int DT, int V, int VL, int LPT, bool ON_SCORE>
__global__ void __launch_bounds__(32 * kWarps, LPT < 32 ? 4 : 2) route_choose_kernel(const RouteArgs a) {
  extern __shared__ uint32_t s_cnt[];  // [warps][G]
  __shared__ ChoiceScratch<LPT> s_cand[kWarps];
  __shared__ int s_expert[kWarps][kMaxRouteTopK];  // (four tokens of at most 8, two of 16, one)
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ alignas(16) float s_bias[V * LPT];
  for (int i = threadIdx.x; i < kWarps * a.G; i += blockDim.x) s_cnt[i] = 0;
  if (a.bias) stage_bias<V, VL, LPT>(a, s_bias);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->status = 0;
  __syncthreads();
  constexpr int kTok = 32 / LPT;  // tokens of a warp at a time
  const int64_t b0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block;
  const int64_t b1 = b0 + a.tokens_per_block < a.T ? b0 + a.tokens_per_block : a.T;
  // whole steps of a warp, shared out evenly
  const int steps = (a.tokens_per_block + kTok - 1) / kTok;
  const int64_t w0 = b0 + steps * warp / kWarps * kTok, w1 = b0 + steps * (warp + 1) / kWarps * kTok;
  const int64_t t0 = w0 < b1 ? w0 : b1, t1 = w1 < b1 ? w1 : b1;
  uint32_t* mine = s_cnt + warp * a.G;
  for (int64_t t = t0; t < t1; t += kTok) {
    const int e = choose_and_write<DT, V, VL, LPT, ON_SCORE>(a, t, t1, lane, s_bias,
                                                             &s_cand[warp], s_expert[warp]);
    uint32_t r = 0;
#pragma unroll
    for (int s = 0; s < kTok; ++s) {
      if (e >= 0 && lane / LPT == s) r = mine[e]++;
      __syncwarp();
    }
    if (e >= 0) a.rank[(t + lane / LPT) * a.k + lane % LPT] = r;
  }
  __syncthreads();
  for (int g = threadIdx.x; g < a.G; g += blockDim.x) {
    uint32_t at = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t c = s_cnt[w * a.G + g];
      s_cnt[w * a.G + g] = at;
      at += c;
    }
    a.counts[static_cast<int64_t>(g) * a.blocks + blockIdx.x] = at;
  }
  __syncthreads();
  if (warp > 0)
#pragma unroll 4
    for (int64_t p = t0 * a.k + lane; p < t1 * a.k; p += 32)
      a.rank[p] += mine[a.experts[p]];
}

// Widest load of a row's logits: VL values, when the rows are a multiple of it and aligned to it.
template <int DT, int V>
constexpr int load_width() {
  return V < (DT == PGG_F32 ? 4 : 8) ? V : (DT == PGG_F32 ? 4 : 8);
}

template <int DT, int V, int VL, int LPT, bool ON_SCORE>
cudaError_t launch_route_v(const RouteArgs& a, cudaStream_t stream) {
  if (a.blocks == 1) {
    // threads for the tokens, no more: fewer counters to clear
    const int64_t warps = (a.T * LPT + 31) / 32;
    const int threads = static_cast<int>(warps < kSmallThreads / 32 ? warps : kSmallThreads / 32) * 32;
    // (the last step of a warp may leave choices for tokens past the last)
    const size_t smem =
        (static_cast<size_t>(threads / 32 + 1) * a.G + (a.T + 32 / LPT - 1) * a.k) * 4;
    auto kern = route_small_kernel<DT, V, VL, LPT, ON_SCORE>;
    // (G is at most V LPT, the pairs are at most kSmallEntries, a token's at most LPT)
    constexpr int kMost = ((kSmallThreads / 32 + 1) * V * LPT + kSmallEntries + 32) * 4;
    static SmemLimit limit;
    const cudaError_t err = allow_smem(&limit, kern, kMost);
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, dim3(1), dim3(threads), smem, stream, 1, a);
  }
  cudaError_t err = launch_pdl(route_choose_kernel<DT, V, VL, LPT, ON_SCORE>, dim3(a.blocks),
                               dim3(32 * kWarps), static_cast<size_t>(kWarps) * a.G * 4, stream, 1,
                               a);
  if (err != cudaSuccess) return err;
  err = launch_count_scan(a.counts, a.G, a.blocks, a.groups, stream);
  if (err != cudaSuccess) return err;
  return launch_route_place(a, stream);
}

template <int DT, int V, int LPT, bool ON_SCORE>
cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t stream) {
  constexpr int kVL = load_width<DT, V>();
  constexpr uintptr_t kAlign = kVL * (DT == PGG_F32 ? 4 : 2);
  if (kVL > 1 && a.G % kVL == 0 && reinterpret_cast<uintptr_t>(a.logits) % kAlign == 0)
    return launch_route_v<DT, V, kVL, LPT, ON_SCORE>(a, stream);
  return launch_route_v<DT, V, 1, LPT, ON_SCORE>(a, stream);
}

}  // namespace
}  // namespace pgg
