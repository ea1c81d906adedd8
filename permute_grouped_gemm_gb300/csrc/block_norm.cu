// The norms before and after a block with its gate and residual scale, in one
// pass over the rows, and their gradient:
//
//     n = N_post(y),  r = residual_scale x + gate n,  h = N_pre(r)
//     N(v) = v^ (offset + w) + b,  v^ = (v - mean) rstd  (rms: mean 0, no b)
//
//     g   = d_r + N_pre'(d_h),  d_x = residual_scale g
//     d_gate = g n, summed as the gate was broadcast;  d_n = g gate
//     d_y = N_post'(d_n)
//     N'(d) = rstd (u - v^ mean(u v^) - mean(u)),  u = d (offset + w)  (rms: no mean(u))
//     d_w = sum over rows of d v^,  d_b = sum over rows of d
//
// A block of threads takes a row at a time and holds it in registers, so each
// tensor is read once; sums are fp32 (variances of the centred values), and the
// pre norm takes r before it is rounded. Memory bounds it. In the gradient a
// thread keeps its columns' parts of the parameters' gradients in registers over
// all rows of its block; the blocks' sums are added in their order by a second
// launch: bitwise repeatable. Rows too long for registers are read again for each
// pass over them.

#include <cstdint>

#include "pgg_block.h"
#include "pgg_ptx.cuh"
#include "pgg_vec.cuh"

namespace pgg {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int64_t kGradBlocks = 304;  // most blocks of the gradient: two an SM

// Sums of K values over the block, the same bits in every thread. Two buffers in turn, so that one
// barrier a call is enough.
template <int K>
struct BlockSum {
  float part[2][32][K];
};

template <int K, int M>
__device__ __forceinline__ void block_sum(BlockSum<M>* s, int* turn, float (&v)[K]) {
  static_assert(K <= M, "room");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
  if (warps == 1) return;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < K; ++i) s->part[*turn][warp][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < K; ++i) {
    v[i] = lane < warps ? s->part[*turn][lane][i] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
  }
  *turn ^= 1;
}

// ------------------------------------------------------------------ rows in registers

// Mean and 1 / deviation of up to two rows of values held by the block.
template <int V, int NV, int M>
__device__ __forceinline__ void stats(BlockSum<M>* s, int* turn, int kind, const float (&v)[NV][V],
                                      int64_t H, float eps, float* mean, float* rstd) {
  const int64_t n = H / V;
  float sum[1] = {0.0f};
  *mean = 0.0f;
  if (kind == PGG_NORM_LAYER) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int c = 0; c < V; ++c) sum[0] += v[j][c];  // (0 outside the row)
    block_sum(s, turn, sum);
    *mean = sum[0] / static_cast<float>(H);
    sum[0] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = j * static_cast<int64_t>(blockDim.x) + threadIdx.x < n;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const float d = v[j][c] - *mean;
      if (in) sum[0] = fmaf(d, d, sum[0]);
    }
  }
  block_sum(s, turn, sum);
  *rstd = 1.0f / sqrtf(sum[0] / static_cast<float>(H) + eps);
}

// The weight's factor and the bias of V columns.
template <int DT, int V>
__device__ __forceinline__ void affine(const void* w, const void* b, bool f32, float offset,
                                       int64_t i, float (&f)[V], float (&add)[V]) {
  if (w) {
    vec::load_or_f32<DT, V>(w, f32, i, f);
#pragma unroll
    for (int c = 0; c < V; ++c) f[c] += offset;
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) f[c] = 1.0f;
  }
  if (b) {
    vec::load_or_f32<DT, V>(b, f32, i, add);
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) add[c] = 0.0f;
  }
}

// The gate of V columns of a row.
template <int DT, int V>
__device__ __forceinline__ void gate_at(const NormArgs& a, int64_t t, int64_t i, float (&g)[V]) {
  if (a.gate_kind == PGG_GATE_CHANNEL) {
    vec::load_or_f32<DT, V>(a.gate, a.p_f32, i, g);
  } else if (a.gate_kind == PGG_GATE_FULL) {
    vec::load_or_f32<DT, V>(a.gate, a.p_f32, t * a.H + i, g);
  } else {
    float one[1] = {1.0f};
    if (a.gate_kind == PGG_GATE_TOKEN) vec::load_or_f32<DT, 1>(a.gate, a.p_f32, t, one);
#pragma unroll
    for (int c = 0; c < V; ++c) g[c] = one[0];
  }
}

template <int DT, int V, int NV>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const NormArgs a) {
  __shared__ BlockSum<1> s;
  int turn = 0;
  ptx::griddep_wait();
  const int64_t n = a.H / V;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    float r[NV][V], y[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t q = j * static_cast<int64_t>(blockDim.x) + threadIdx.x;
#pragma unroll
      for (int c = 0; c < V; ++c) r[j][c] = y[j][c] = 0.0f;
      if (q < n) {
        vec::load<DT, V>(a.x, t * a.H + q * V, r[j]);
        if (a.y) vec::load_or_f32<DT, V>(a.y, a.y_f32, t * a.H + q * V, y[j]);
      }
    }
    float mean = 0.0f, rstd = 1.0f;
    if (a.post != PGG_NORM_NONE) stats(&s, &turn, a.post, y, a.H, a.eps, &mean, &rstd);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t q = j * static_cast<int64_t>(blockDim.x) + threadIdx.x;
      if (q >= n) continue;
      if (a.y) {
        float f[V], b[V], g[V];
        affine<DT, V>(a.w_post, a.b_post, a.p_f32, a.weight_offset, q * V, f, b);
        gate_at<DT, V>(a, t, q * V, g);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const float u = fmaf((y[j][c] - mean) * rstd, f[c], b[c]);
          r[j][c] = fmaf(g[c], u, a.residual_scale * r[j][c]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < V; ++c) r[j][c] *= a.residual_scale;
      }
      if (a.r) vec::store<DT, V>(a.r, t * a.H + q * V, r[j]);
    }
    if (a.pre == PGG_NORM_NONE) continue;
    stats(&s, &turn, a.pre, r, a.H, a.eps, &mean, &rstd);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t q = j * static_cast<int64_t>(blockDim.x) + threadIdx.x;
      if (q >= n) continue;
      float f[V], b[V];
      affine<DT, V>(a.w_pre, a.b_pre, a.p_f32, a.weight_offset, q * V, f, b);
#pragma unroll
      for (int c = 0; c < V; ++c) r[j][c] = fmaf((r[j][c] - mean) * rstd, f[c], b[c]);
      vec::store<DT, V>(a.h, t * a.H + q * V, r[j]);
    }
  }
}

// Columns' sums that a block keeps: gate (channel), w_post, b_post, w_pre, b_pre.
enum { kColGate, kColWPost, kColBPost, kColWPre, kColBPre, kCols };

// (BIAS: some norm has a mean, so there may be sums for a bias)
template <int DT, int V, int NV, bool BIAS>
__global__ void __launch_bounds__(kMaxThreads) block_norm_grad_kernel(const NormArgs a) {
  __shared__ BlockSum<3> s;
  int turn = 0;
  ptx::griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->status = 0;
  const int64_t n = a.H / V;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  float col[BIAS ? kCols : 3][NV][V] = {};  // without BIAS: gate, w_post, w_pre
  constexpr int kWPre = BIAS ? kColWPre : 2;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    // g: the gradient of r;  dh, then what it gives;  r and y, then normalised
    float g[NV][V], dh[NV][V], r[NV][V], y[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t q = j * static_cast<int64_t>(blockDim.x) + threadIdx.x;
#pragma unroll
      for (int c = 0; c < V; ++c) g[j][c] = dh[j][c] = r[j][c] = y[j][c] = 0.0f;
      if (q < n) {
        const int64_t i = t * a.H + q * V;
        if (a.d_r) vec::load<DT, V>(a.d_r, i, g[j]);
        if (a.y) vec::load_or_f32<DT, V>(a.y, a.y_f32, i, y[j]);
        if (a.pre != PGG_NORM_NONE) {
          vec::load_or_f32<DT, V>(a.d_h, a.dh_f32, i, dh[j]);
          vec::load<DT, V>(a.x, i, r[j]);
        }
      }
    }
    float mean, rstd;
    if (a.pre != PGG_NORM_NONE) {
      stats(&s, &turn, a.pre, r, a.H, a.eps, &mean, &rstd);
      float sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int64_t q = j * static_cast<int64_t>(blockDim.x) + threadIdx.x;
        if (q >= n) continue;
        float f[V], b[V];
        affine<DT, V>(a.w_pre, nullptr, a.p_f32, a.weight_offset, q * V, f, b);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          r[j][c] = (r[j][c] - mean) * rstd;
          col[kWPre][j][c] = fmaf(dh[j][c], r[j][c], col[kWPre][j][c]);
          if constexpr (BIAS) col[kColBPre][j][c] += dh[j][c];
          dh[j][c] *= f[c];
          sum[0] = fmaf(dh[j][c], r[j][c], sum[0]);
          sum[1] += dh[j][c];
        }
      }
      block_sum(&s, &turn, sum);
      const float along = sum[0] * inv_h;
      const float centre = a.pre == PGG_NORM_LAYER ? sum[1] * inv_h : 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int c = 0; c < V; ++c)
          g[j][c] = fmaf(rstd, dh[j][c] - fmaf(r[j][c], along, centre), g[j][c]);
    }
    // (r is done with: it holds d_x)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t q = j * static_cast<int64_t>(blockDim.x) + threadIdx.x;
      if (q >= n) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) r[j][c] = a.residual_scale * g[j][c];
      vec::store<DT, V>(a.r, t * a.H + q * V, r[j]);
    }
    if (!a.y) continue;
    mean = 0.0f;
    rstd = 1.0f;
    if (a.post != PGG_NORM_NONE) stats(&s, &turn, a.post, y, a.H, a.eps, &mean, &rstd);
    float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t q = j * static_cast<int64_t>(blockDim.x) + threadIdx.x;
      if (q >= n) continue;
      float f[V], b[V], gate[V], whole[V];
      affine<DT, V>(a.w_post, a.b_post, a.p_f32, a.weight_offset, q * V, f, b);
      gate_at<DT, V>(a, t, q * V, gate);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        y[j][c] = (y[j][c] - mean) * rstd;
        whole[c] = g[j][c] * fmaf(y[j][c], f[c], b[c]);
        col[kColGate][j][c] += whole[c];
        sum[2] += whole[c];
        g[j][c] *= gate[c];
        col[kColWPost][j][c] = fmaf(g[j][c], y[j][c], col[kColWPost][j][c]);
        if constexpr (BIAS) col[kColBPost][j][c] += g[j][c];
        g[j][c] *= f[c];
        sum[0] = fmaf(g[j][c], y[j][c], sum[0]);
        sum[1] += g[j][c];
      }
      if (a.gate_kind == PGG_GATE_FULL) {
        if (DT == PGG_F32 || a.p_f32)
          vec::store<PGG_F32, V>(a.d_gate, t * a.H + q * V, whole);
        else
          vec::store<DT, V>(a.d_gate, t * a.H + q * V, whole);
      }
    }
    if (a.post != PGG_NORM_NONE || a.gate_kind == PGG_GATE_TOKEN) block_sum(&s, &turn, sum);
    if (a.gate_kind == PGG_GATE_TOKEN && threadIdx.x == 0)
      static_cast<float*>(a.d_gate)[t] = sum[2];
    const float along = a.post != PGG_NORM_NONE ? sum[0] * inv_h : 0.0f;
    const float centre = a.post == PGG_NORM_LAYER ? sum[1] * inv_h : 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t q = j * static_cast<int64_t>(blockDim.x) + threadIdx.x;
      if (q >= n) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) y[j][c] = rstd * (g[j][c] - fmaf(y[j][c], along, centre));
      vec::store<DT, V>(a.h, t * a.H + q * V, y[j]);
    }
  }
#pragma unroll
  for (int k = 0; k < (BIAS ? kCols : 3); ++k) {
    const int which = BIAS ? k : (k == 2 ? static_cast<int>(kColWPre) : k);
    if (!a.d_cols[which]) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t q = j * static_cast<int64_t>(blockDim.x) + threadIdx.x;
      if (q < n)
        vec::store<PGG_F32, V>(a.partial, (static_cast<int64_t>(blockIdx.x) * kCols + which) * a.H
                                              + q * V, col[k][j]);
    }
  }
}

// ------------------------------------------------------------------ rows of any length

// Element i of n = N_post(y) and of r, from memory.
template <int DT>
__device__ __forceinline__ float at(const void* p, bool f32, int64_t i) {
  float v[1];
  vec::load_or_f32<DT, 1>(p, f32, i, v);
  return v[0];
}

struct Stat {
  float mean, rstd;
};

// Mean and 1 / deviation of value(i), i < H.
template <int M, typename F>
__device__ __forceinline__ Stat stats_of(BlockSum<M>* s, int* turn, int kind, int64_t H, float eps,
                                         F&& value) {
  Stat st = {0.0f, 1.0f};
  if (kind == PGG_NORM_NONE) return st;
  float sum[1] = {0.0f};
  if (kind == PGG_NORM_LAYER) {
    for (int64_t i = threadIdx.x; i < H; i += blockDim.x) sum[0] += value(i);
    block_sum(s, turn, sum);
    st.mean = sum[0] / static_cast<float>(H);
    sum[0] = 0.0f;
  }
  for (int64_t i = threadIdx.x; i < H; i += blockDim.x) {
    const float d = value(i) - st.mean;
    sum[0] = fmaf(d, d, sum[0]);
  }
  block_sum(s, turn, sum);
  st.rstd = 1.0f / sqrtf(sum[0] / static_cast<float>(H) + eps);
  return st;
}

template <int DT>
__global__ void __launch_bounds__(kMaxThreads) block_norm_long_kernel(const NormArgs a) {
  __shared__ BlockSum<1> s;
  int turn = 0;
  ptx::griddep_wait();
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t t0 = t * a.H;
    auto y = [&](int64_t i) { return at<DT>(a.y, a.y_f32, t0 + i); };
    const Stat post = stats_of(&s, &turn, a.post, a.H, a.eps, y);
    auto r = [&](int64_t i) {
      const float x = a.residual_scale * vec::load1<DT>(a.x, t0 + i);
      if (!a.y) return x;
      float f[1], b[1], g[1];
      affine<DT, 1>(a.w_post, a.b_post, a.p_f32, a.weight_offset, i, f, b);
      gate_at<DT, 1>(a, t, i, g);
      return fmaf(g[0], fmaf((y(i) - post.mean) * post.rstd, f[0], b[0]), x);
    };
    const Stat pre = stats_of(&s, &turn, a.pre, a.H, a.eps, r);
    // (r may be written over x, h over y: a thread reads its element before it writes it)
    for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
      const float v = r(i);
      if (a.r) vec::store1<DT>(a.r, t0 + i, v);
      if (a.pre == PGG_NORM_NONE) continue;
      float f[1], b[1];
      affine<DT, 1>(a.w_pre, a.b_pre, a.p_f32, a.weight_offset, i, f, b);
      vec::store1<DT>(a.h, t0 + i, fmaf((v - pre.mean) * pre.rstd, f[0], b[0]));
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(kMaxThreads) block_norm_grad_long_kernel(const NormArgs a) {
  __shared__ BlockSum<3> s;
  int turn = 0;
  ptx::griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->status = 0;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  float* mine = a.partial + static_cast<int64_t>(blockIdx.x) * kCols * a.H;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t t0 = t * a.H;
    const bool first = t == blockIdx.x;
    auto keep = [&](int which, int64_t i, float v) {
      if (!a.d_cols[which]) return;
      float* p = mine + which * a.H + i;
      *p = first ? v : *p + v;
    };
    auto r = [&](int64_t i) { return vec::load1<DT>(a.x, t0 + i); };
    auto y = [&](int64_t i) { return at<DT>(a.y, a.y_f32, t0 + i); };
    auto factor = [&](const void* w, int64_t i) {
      return w ? at<DT>(w, a.p_f32, i) + a.weight_offset : 1.0f;
    };
    const Stat pre = stats_of(&s, &turn, a.pre, a.H, a.eps, r);
    float along = 0.0f, centre = 0.0f;
    if (a.pre != PGG_NORM_NONE) {
      float sum[2] = {0.0f, 0.0f};
      for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float d = at<DT>(a.d_h, a.dh_f32, t0 + i), v = (r(i) - pre.mean) * pre.rstd;
        keep(kColWPre, i, d * v);
        keep(kColBPre, i, d);
        const float u = d * factor(a.w_pre, i);
        sum[0] = fmaf(u, v, sum[0]);
        sum[1] += u;
      }
      block_sum(&s, &turn, sum);
      along = sum[0] * inv_h;
      centre = a.pre == PGG_NORM_LAYER ? sum[1] * inv_h : 0.0f;
    }
    auto grad = [&](int64_t i) {  // of r
      float g = a.d_r ? vec::load1<DT>(a.d_r, t0 + i) : 0.0f;
      if (a.pre != PGG_NORM_NONE) {
        const float v = (r(i) - pre.mean) * pre.rstd;
        const float u = at<DT>(a.d_h, a.dh_f32, t0 + i) * factor(a.w_pre, i);
        g = fmaf(pre.rstd, u - fmaf(v, along, centre), g);
      }
      return g;
    };
    if (!a.y) {
      for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x)
        vec::store1<DT>(a.r, t0 + i, a.residual_scale * grad(i));
      continue;
    }
    const Stat post = stats_of(&s, &turn, a.post, a.H, a.eps, y);
    float sum[3] = {0.0f, 0.0f, 0.0f};
    for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
      const float g = grad(i), v = (y(i) - post.mean) * post.rstd, f = factor(a.w_post, i);
      const float whole = g * fmaf(v, f, a.b_post ? at<DT>(a.b_post, a.p_f32, i) : 0.0f);
      float gate[1];
      gate_at<DT, 1>(a, t, i, gate);
      const float d = g * gate[0];
      keep(kColGate, i, whole);
      keep(kColWPost, i, d * v);
      keep(kColBPost, i, d);
      sum[0] = fmaf(d * f, v, sum[0]);
      sum[1] += d * f;
      sum[2] += whole;
    }
    block_sum(&s, &turn, sum);
    if (a.gate_kind == PGG_GATE_TOKEN && threadIdx.x == 0)
      static_cast<float*>(a.d_gate)[t] = sum[2];
    const float along_y = a.post != PGG_NORM_NONE ? sum[0] * inv_h : 0.0f;
    const float centre_y = a.post == PGG_NORM_LAYER ? sum[1] * inv_h : 0.0f;
    for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
      const float g = grad(i), v = (y(i) - post.mean) * post.rstd, f = factor(a.w_post, i);
      float gate[1];
      gate_at<DT, 1>(a, t, i, gate);
      if (a.gate_kind == PGG_GATE_FULL) {
        const float whole = g * fmaf(v, f, a.b_post ? at<DT>(a.b_post, a.p_f32, i) : 0.0f);
        if (DT == PGG_F32 || a.p_f32)
          static_cast<float*>(a.d_gate)[t0 + i] = whole;
        else
          vec::store1<DT>(a.d_gate, t0 + i, whole);
      }
      vec::store1<DT>(a.r, t0 + i, a.residual_scale * g);
      vec::store1<DT>(a.h, t0 + i, post.rstd * (g * gate[0] * f - fmaf(v, along_y, centre_y)));
    }
  }
}

// d[which][i] = sum over the blocks, in their order. 32 columns x 8 shares of the blocks.
__global__ void __launch_bounds__(256) block_norm_cols_kernel(const NormArgs a, int64_t blocks) {
  __shared__ float s_sum[8][33];
  ptx::griddep_wait();
  float* out = a.d_cols[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int64_t per = (blocks + 7) / 8;
  const int64_t b1 = (share + 1) * per < blocks ? (share + 1) * per : blocks;
  float sum = 0.0f;
  if (i < a.H) {
#pragma unroll 8
    for (int64_t b = share * per; b < b1; ++b) sum += a.partial[(b * kCols + blockIdx.y) * a.H + i];
  }
  s_sum[share][lane] = sum;
  __syncthreads();
  if (share != 0 || i >= a.H) return;
  sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) sum += s_sum[k][lane];
  out[i] = sum;
}

// Vectors of a thread and threads for rows of n vectors: as few vectors as `most` threads allow.
bool shape(int64_t n, int most, int max_nv, int* nv, int* threads) {
  for (*nv = 1; *nv <= max_nv; *nv *= 2) {
    const int64_t need = ((n + *nv - 1) / *nv + 31) / 32 * 32;
    if (need <= (*nv == max_nv ? kMaxThreads : most)) {
      *threads = static_cast<int>(need);
      return true;
    }
  }
  return false;
}

template <int DT, int V>
cudaError_t launch_forward(const NormArgs& a, int num_sms, cudaStream_t stream) {
  using K = void (*)(const NormArgs);
  static const K kern[4] = {block_norm_kernel<DT, V, 1>, block_norm_kernel<DT, V, 2>,
                            block_norm_kernel<DT, V, 4>, block_norm_kernel<DT, V, 8>};
  int nv, threads;
  K k = block_norm_long_kernel<DT>;
  if (shape(a.H / V, 512, V == 1 ? 8 : 4, &nv, &threads))
    k = kern[nv == 1 ? 0 : nv == 2 ? 1 : nv == 4 ? 2 : 3];
  else
    threads = kMaxThreads;
  int64_t grid = static_cast<int64_t>(num_sms) * (2048 / threads);
  if (grid > a.T) grid = a.T;
  return launch_pdl(k, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(threads)), 0,
                    stream, 1, a);
}

template <int DT, int V>
cudaError_t launch_backward(const NormArgs& a, cudaStream_t stream) {
  using K = void (*)(const NormArgs);
  static const K kern[2][2] = {
      {block_norm_grad_kernel<DT, V, 1, false>, block_norm_grad_kernel<DT, V, 2, false>},
      {block_norm_grad_kernel<DT, V, 1, true>, block_norm_grad_kernel<DT, V, 2, true>}};
  int nv, threads;
  K k = block_norm_grad_long_kernel<DT>;
  const bool bias = a.d_cols[kColBPost] || a.d_cols[kColBPre];
  if (shape(a.H / V, kMaxThreads, 2, &nv, &threads))
    k = kern[bias ? 1 : 0][nv - 1];
  else
    threads = kMaxThreads;
  const int64_t blocks = norm_grad_blocks(a.T);
  cudaError_t err = launch_pdl(k, dim3(static_cast<unsigned>(blocks)),
                               dim3(static_cast<unsigned>(threads)), 0, stream, 1, a);
  if (err != cudaSuccess) return err;
  for (int i = 0; i < kCols; ++i)
    if (a.d_cols[i])
      return launch_pdl(block_norm_cols_kernel, dim3(static_cast<unsigned>((a.H + 31) / 32), kCols),
                        dim3(256), 0, stream, 1, a, blocks);
  return cudaSuccess;
}

}  // namespace

int64_t norm_grad_blocks(int64_t T) { return T < kGradBlocks ? T : kGradBlocks; }

cudaError_t launch_block_norm(int dtype, const NormArgs& a, bool rows16, int num_sms,
                              cudaStream_t stream) {
  if (dtype == PGG_F32)
    return rows16 ? launch_forward<PGG_F32, 4>(a, num_sms, stream)
                  : launch_forward<PGG_F32, 1>(a, num_sms, stream);
  if (dtype == PGG_F16)
    return rows16 ? launch_forward<PGG_F16, 8>(a, num_sms, stream)
                  : launch_forward<PGG_F16, 1>(a, num_sms, stream);
  if (dtype == PGG_BF16)
    return rows16 ? launch_forward<PGG_BF16, 8>(a, num_sms, stream)
                  : launch_forward<PGG_BF16, 1>(a, num_sms, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_block_norm_grad(int dtype, const NormArgs& a, bool rows16, int num_sms,
                                   cudaStream_t stream) {
  (void)num_sms;
  if (dtype == PGG_F32)
    return rows16 ? launch_backward<PGG_F32, 4>(a, stream) : launch_backward<PGG_F32, 1>(a, stream);
  if (dtype == PGG_F16)
    return rows16 ? launch_backward<PGG_F16, 8>(a, stream) : launch_backward<PGG_F16, 1>(a, stream);
  if (dtype == PGG_BF16)
    return rows16 ? launch_backward<PGG_BF16, 8>(a, stream)
                  : launch_backward<PGG_BF16, 1>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pgg
