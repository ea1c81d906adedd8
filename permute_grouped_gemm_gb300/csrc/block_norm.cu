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
// Here are the rows that block_norm_rows.cu does not take: no multiple of 16 bytes,
// or too long for a block's threads with 16 elements each. A block takes a row at a
// time; sums are fp32 (variances of the centred values), and the pre norm takes r
// before it is rounded. Rows of 16-byte vectors go through shared memory: every
// thread copies (cp.async) what it will read itself, while the row before is worked
// on, and reads it again for each pass; others are read from memory each time (the
// first level cache holds them); ones that are longer still with one element a
// thread and turn. Columns' parts of the parameters' gradients are kept over all
// rows of a block, and the blocks' sums are added in their order by a second
// launch: bitwise repeatable. Instructions bound it: 4000 x 6999 takes 273 us, its
// gradient 629 (one element a thread and turn: 301 and 708; up to eight vectors a
// thread are the rule where they fit), 4000 x 8704 (as rms norms, 16-bit) 99 and 346.

#include <atomic>
#include <cstdint>

#include "pgg_block.h"
#include "pgg_block_sum.cuh"
#include "pgg_ops_launch.h"
#include "pgg_ptx.cuh"
#include "pgg_vec.cuh"

namespace pgg {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kRingBytes = 168 * 1024;  // of shared memory: rows that are held or on their way

// The rows of up to four tensors, a thread's vectors for itself. RING: on their way through shared
// memory, vector q of a tensor at q * 16 (of 32 bytes: the second halves behind all first ones);
// else in memory.
template <int DT, int V, int NV, bool RING>
struct Rows {
  const char* base[4];
  int bytes[4];       // of a vector; 0 = no tensor
  uint32_t offset[4];
  uint32_t slot_bytes;
  int n;              // vectors of a row

  __device__ __forceinline__ void add(int i, const void* p, bool f32) {
    base[i] = static_cast<const char*>(p);
    bytes[i] = p ? V * (f32 ? 4 : vec::elem_bytes(DT)) : 0;
    offset[i] = slot_bytes;
    slot_bytes += static_cast<uint32_t>(n) * bytes[i];
  }
  // Row t into `slot` (nothing behind the last row); one group of copies.
  __device__ __forceinline__ void fetch(uint8_t* smem, int slot, int64_t t, int64_t T) const {
    if (!RING) return;
    if (t < T) {
      const uint32_t to = ptx::smem_addr(smem) + slot * slot_bytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (bytes[i] == 0) continue;
        const char* row = base[i] + t * (static_cast<int64_t>(n) * bytes[i]);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int q = j * blockDim.x + threadIdx.x;
          if (q >= n) continue;
          const uint32_t at = to + offset[i] + q * 16;
          const char* src = row + q * bytes[i];
          ptx::cp_async_16(at, src, 16);
          if (bytes[i] == 32) ptx::cp_async_16(at + n * 16, src + 16, 16);
        }
      }
    }
    ptx::cp_async_commit();
  }
  // Vector q of row t of tensor i.
  __device__ __forceinline__ void read(const uint8_t* smem, int slot, int64_t t, int i, int q,
                                       bool f32, float (&v)[V]) const {
    if constexpr (RING) {
      const uint8_t* p = smem + slot * slot_bytes + offset[i] + q * 16;
      if (DT != PGG_F32 && f32) {
        float lo[4], hi[4];
        vec::load<PGG_F32, 4>(p, 0, lo);
        vec::load<PGG_F32, 4>(p + n * 16, 0, hi);
#pragma unroll
        for (int c = 0; c < V; ++c) v[c] = c < 4 ? lo[c & 3] : hi[c & 3];
      } else {
        vec::load<DT, V>(p, 0, v);
      }
    } else {
      const char* row = base[i] + t * (static_cast<int64_t>(n) * bytes[i]);
      vec::load_or_f32<DT, V>(row, f32, q * V, v);
    }
  }
};

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

// One parameter (a weight with its offset, or a channel's gate); 1 where there is none.
template <int DT, int V>
struct Param {
  const void* p;
  float offset;
  bool f32;

  __device__ __forceinline__ void get(int q, float (&v)[V]) const {
    if (p) {
      vec::load_or_f32<DT, V>(p, f32, q * V, v);
#pragma unroll
      for (int c = 0; c < V; ++c) v[c] += offset;
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) v[c] = 1.0f;
    }
  }
};

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

// ------------------------------------------------------------------ rows held by a block

// LEAN: rms norms or none, a gate of one number a channel or none.
template <int DT, int V, int NV, bool RING, bool LEAN, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) block_norm_kernel(const NormArgs a, const int ring) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ BlockSum<1> s;
  int turn = 0, slot = 0;
  ptx::griddep_wait();
  const float inv_h = 1.0f / static_cast<float>(a.H);
  Rows<DT, V, NV, RING> rows = {};
  rows.n = static_cast<int>(a.H / V);
  const int n = rows.n, tid = threadIdx.x;
  const bool y_f32 = DT == PGG_F32 || a.y_f32, have_y = a.y != nullptr;
  rows.add(0, a.x, DT == PGG_F32);
  rows.add(1, a.y, y_f32);
  for (int i = 0; RING && i < ring; ++i)
    rows.fetch(smem, i, blockIdx.x + static_cast<int64_t>(i) * gridDim.x, a.T);
  const bool by_row = !LEAN && (a.gate_kind == PGG_GATE_FULL || a.gate_kind == PGG_GATE_TOKEN);
  const int post = LEAN && a.post != PGG_NORM_NONE ? PGG_NORM_RMS : a.post;
  const bool layer = !LEAN && a.pre == PGG_NORM_LAYER;
  const Param<DT, V> f_post = {a.w_post, a.weight_offset, a.p_f32 != 0},
                     f_pre = {a.w_pre, a.weight_offset, a.p_f32 != 0},
                     channel = {a.gate_kind == PGG_GATE_CHANNEL ? a.gate : nullptr, 0.0f,
                                a.p_f32 != 0};
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (RING) {  // (a group of copies a row: those of the `ring` - 1 rows behind may be pending)
      if (ring > 2) ptx::cp_async_wait<2>(); else if (ring == 2) ptx::cp_async_wait<1>(); else ptx::cp_async_wait<0>();
    }
    float mean = 0.0f, rstd = 1.0f;
    if (post != PGG_NORM_NONE) {
      float sum[1];
      if (!LEAN && post == PGG_NORM_LAYER) {
        sum[0] = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int q = j * blockDim.x + tid;
          if (q >= n) continue;
          float y[V];
          rows.read(smem, slot, t, 1, q, y_f32, y);
#pragma unroll
          for (int c = 0; c < V; ++c) sum[0] += y[c];
        }
        block_sum(&s, &turn, sum);
        mean = sum[0] * inv_h;
      }
      sum[0] = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int q = j * blockDim.x + tid;
        if (q >= n) continue;
        float y[V];
        rows.read(smem, slot, t, 1, q, y_f32, y);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const float v = LEAN ? y[c] : y[c] - mean;
          sum[0] = fmaf(v, v, sum[0]);
        }
      }
      block_sum(&s, &turn, sum);
      rstd = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
    }
    float r[NV][V], sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int q = j * blockDim.x + tid;
      if (q >= n) continue;
      rows.read(smem, slot, t, 0, q, DT == PGG_F32, r[j]);
#pragma unroll
      for (int c = 0; c < V; ++c) r[j][c] *= a.residual_scale;
      if (have_y) {
        float y[V];
        rows.read(smem, slot, t, 1, q, y_f32, y);
        float f[V], g[V];
        f_post.get(q, f);
        if (by_row)
          gate_at<DT, V>(a, t, q * V, g);
        else
          channel.get(q, g);
        if constexpr (LEAN) {
#pragma unroll
          for (int c = 0; c < V; ++c) r[j][c] = fmaf(y[c] * rstd, f[c] * g[c], r[j][c]);
        } else {
          float one[V], b[V];
          affine<DT, V>(nullptr, a.b_post, a.p_f32, 0.0f, q * V, one, b);
#pragma unroll
          for (int c = 0; c < V; ++c)
            r[j][c] = fmaf(g[c], fmaf((y[c] - mean) * rstd, f[c], b[c]), r[j][c]);
        }
      }
      if (a.r) vec::store<DT, V>(a.r, t * a.H + q * V, r[j]);
#pragma unroll
      for (int c = 0; c < V; ++c)
        sum[0] = layer ? sum[0] + r[j][c] : fmaf(r[j][c], r[j][c], sum[0]);
    }
    if (RING) {  // (a thread's copies go where it alone has read)
      rows.fetch(smem, slot, t + static_cast<int64_t>(ring) * gridDim.x, a.T);
      slot = slot + 1 == ring ? 0 : slot + 1;
    }
    if (a.pre == PGG_NORM_NONE) continue;
    block_sum(&s, &turn, sum);
    mean = 0.0f;
    if (layer) {
      mean = sum[0] * inv_h;
      sum[0] = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int q = j * blockDim.x + tid;
        if (q >= n) continue;
#pragma unroll
        for (int c = 0; c < V; ++c) sum[0] = fmaf(r[j][c] - mean, r[j][c] - mean, sum[0]);
      }
      block_sum(&s, &turn, sum);
    }
    rstd = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int q = j * blockDim.x + tid;
      if (q >= n) continue;
      float f[V];
      f_pre.get(q, f);
      if constexpr (LEAN) {
#pragma unroll
        for (int c = 0; c < V; ++c) r[j][c] = r[j][c] * rstd * f[c];
      } else {
        float one[V], b[V];
        affine<DT, V>(nullptr, a.b_pre, a.p_f32, 0.0f, q * V, one, b);
#pragma unroll
        for (int c = 0; c < V; ++c) r[j][c] = fmaf((r[j][c] - mean) * rstd, f[c], b[c]);
      }
      vec::store<DT, V>(a.h, t * a.H + q * V, r[j]);
    }
  }
}

// LEAN as above: no sums for a bias either.
template <int DT, int V, int NV, bool RING, bool LEAN, int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
    block_norm_grad_kernel(const NormArgs a, const int ring) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr bool BIAS = !LEAN;
  __shared__ BlockSum<4> s;
  int turn = 0, slot = 0;
  ptx::griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->status = 0;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  Rows<DT, V, NV, RING> rows = {};
  rows.n = static_cast<int>(a.H / V);
  const int n = rows.n, tid = threadIdx.x;
  const bool y_f32 = DT == PGG_F32 || a.y_f32, dh_f32 = DT == PGG_F32 || a.dh_f32;
  const bool have_y = a.y != nullptr, pre = a.pre != PGG_NORM_NONE;
  const bool token = !LEAN && a.gate_kind == PGG_GATE_TOKEN;
  const bool by_row = token || (!LEAN && a.gate_kind == PGG_GATE_FULL);
  rows.add(0, a.d_r, DT == PGG_F32);
  rows.add(1, a.y, y_f32);
  rows.add(2, pre ? a.d_h : nullptr, dh_f32);
  rows.add(3, pre ? a.x : nullptr, DT == PGG_F32);
  for (int i = 0; RING && i < ring; ++i)
    rows.fetch(smem, i, blockIdx.x + static_cast<int64_t>(i) * gridDim.x, a.T);
  float col[BIAS ? kNormCols : 3][NV][V] = {};  // without BIAS: gate, w_post, w_pre
  constexpr int kWPre = BIAS ? kColWPre : 2;
  const Param<DT, V> f_post = {a.w_post, a.weight_offset, a.p_f32 != 0},
                     f_pre = {a.w_pre, a.weight_offset, a.p_f32 != 0},
                     channel = {a.gate_kind == PGG_GATE_CHANNEL ? a.gate : nullptr, 0.0f,
                                a.p_f32 != 0};
  auto bias_at = [&](int q, float (&b)[V]) {
    float one[V];
    affine<DT, V>(nullptr, BIAS ? a.b_post : nullptr, a.p_f32, 0.0f, q * V, one, b);
  };
  auto gate_of = [&](int64_t t, int j, int q, float (&g)[V]) {
    if (by_row)
      gate_at<DT, V>(a, t, q * V, g);
    else
      channel.get(q, g);
  };
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (RING) {
      if (ring > 2) ptx::cp_async_wait<2>(); else if (ring == 2) ptx::cp_async_wait<1>(); else ptx::cp_async_wait<0>();
    }
    float mean = 0.0f, rstd = 1.0f, along = 0.0f, centre = 0.0f;
    if (pre) {
      if (!LEAN && a.pre == PGG_NORM_LAYER) {
        float sum[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int q = j * blockDim.x + tid;
          if (q >= n) continue;
          float r[V];
          rows.read(smem, slot, t, 3, q, DT == PGG_F32, r);
#pragma unroll
          for (int c = 0; c < V; ++c) sum[0] += r[c];
        }
        block_sum(&s, &turn, sum);
        mean = sum[0] * inv_h;
      }
      float sum[3] = {0.0f, 0.0f, 0.0f};  // of v^2, u v, u with v = r - mean
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int q = j * blockDim.x + tid;
        if (q >= n) continue;
        float r[V], dh[V], f[V];
        rows.read(smem, slot, t, 3, q, DT == PGG_F32, r);
        rows.read(smem, slot, t, 2, q, dh_f32, dh);
        f_pre.get(q, f);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const float v = LEAN ? r[c] : r[c] - mean, u = dh[c] * f[c];
          sum[0] = fmaf(v, v, sum[0]);
          sum[1] = fmaf(u, v, sum[1]);
          if (!LEAN) sum[2] += u;
        }
      }
      block_sum(&s, &turn, sum);
      rstd = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
      along = sum[1] * rstd * inv_h;
      centre = !LEAN && a.pre == PGG_NORM_LAYER ? sum[2] * inv_h : 0.0f;
    }
    float mean_y = 0.0f;
    if (!LEAN && a.post == PGG_NORM_LAYER) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int q = j * blockDim.x + tid;
        if (q >= n) continue;
        float y[V];
        rows.read(smem, slot, t, 1, q, y_f32, y);
#pragma unroll
        for (int c = 0; c < V; ++c) sum[0] += y[c];
      }
      block_sum(&s, &turn, sum);
      mean_y = sum[0] * inv_h;
    }
    // g, d_x, and the sums of v^2, w v, w and g b with v = y - mean, w = g gate f (and, for a
    // token's gate, g f v is w v / gate: it is taken by itself)
    float g[NV][V], sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int q = j * blockDim.x + tid;
      if (q >= n) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) g[j][c] = 0.0f;
      if (a.d_r) rows.read(smem, slot, t, 0, q, DT == PGG_F32, g[j]);
      if (pre) {
        float r[V], dh[V], f[V];
        rows.read(smem, slot, t, 3, q, DT == PGG_F32, r);
        rows.read(smem, slot, t, 2, q, dh_f32, dh);
        f_pre.get(q, f);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const float v = (LEAN ? r[c] : r[c] - mean) * rstd;
          col[kWPre][j][c] = fmaf(dh[c], v, col[kWPre][j][c]);
          if constexpr (BIAS) col[kColBPre][j][c] += dh[c];
          const float u = dh[c] * f[c];
          g[j][c] = fmaf(rstd, LEAN ? fmaf(-v, along, u) : u - fmaf(v, along, centre), g[j][c]);
        }
      }
      float d[V];
#pragma unroll
      for (int c = 0; c < V; ++c) d[c] = a.residual_scale * g[j][c];
      vec::store<DT, V>(a.r, t * a.H + q * V, d);
      if (have_y && (a.post != PGG_NORM_NONE || token)) {
        float y[V], f[V], b[V], gate[V];
        rows.read(smem, slot, t, 1, q, y_f32, y);
        f_post.get(q, f);
        if (BIAS) bias_at(q, b);
        gate_of(t, j, q, gate);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const float v = LEAN ? y[c] : y[c] - mean_y, w = g[j][c] * f[c];
          sum[0] = fmaf(v, v, sum[0]);
          if constexpr (LEAN) {
            sum[1] = fmaf(w * gate[c], v, sum[1]);
          } else {
            sum[1] = fmaf(token ? w : w * gate[c], v, sum[1]);
            sum[2] = fmaf(w, gate[c], sum[2]);
            sum[3] = fmaf(g[j][c], b[c], sum[3]);
          }
        }
      }
    }
    if (have_y) {
      float rstd_y = 1.0f, along_y = 0.0f, centre_y = 0.0f;
      if (a.post != PGG_NORM_NONE || token) {
        block_sum(&s, &turn, sum);
        if (a.post != PGG_NORM_NONE) rstd_y = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
        float tg[1] = {1.0f};
        if (token) {
          vec::load_or_f32<DT, 1>(a.gate, a.p_f32, t, tg);
          if (tid == 0) static_cast<float*>(a.d_gate)[t] = fmaf(sum[1], rstd_y, sum[3]);
        }
        if (a.post != PGG_NORM_NONE) along_y = sum[1] * tg[0] * rstd_y * inv_h;
        if (!LEAN && a.post == PGG_NORM_LAYER) centre_y = sum[2] * inv_h;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int q = j * blockDim.x + tid;
        if (q >= n) continue;
        float y[V], f[V], b[V], gate[V], whole[V];
        rows.read(smem, slot, t, 1, q, y_f32, y);
        f_post.get(q, f);
        if (BIAS) bias_at(q, b);
        gate_of(t, j, q, gate);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const float v = (LEAN ? y[c] : y[c] - mean_y) * rstd_y, d = g[j][c] * gate[c];
          whole[c] = g[j][c] * (BIAS ? fmaf(v, f[c], b[c]) : v * f[c]);
          col[kColGate][j][c] += whole[c];
          col[kColWPost][j][c] = fmaf(d, v, col[kColWPost][j][c]);
          if constexpr (BIAS) col[kColBPost][j][c] += d;
          const float u = d * f[c];
          y[c] = rstd_y * (LEAN ? fmaf(-v, along_y, u) : u - fmaf(v, along_y, centre_y));
        }
        vec::store<DT, V>(a.h, t * a.H + q * V, y);
        if (!LEAN && a.gate_kind == PGG_GATE_FULL) {
          if (DT == PGG_F32 || a.p_f32)
            vec::store<PGG_F32, V>(a.d_gate, t * a.H + q * V, whole);
          else
            vec::store<DT, V>(a.d_gate, t * a.H + q * V, whole);
        }
      }
    }
    if (RING) {  // (a thread's copies go where it alone has read)
      rows.fetch(smem, slot, t + static_cast<int64_t>(ring) * gridDim.x, a.T);
      slot = slot + 1 == ring ? 0 : slot + 1;
    }
  }
#pragma unroll
  for (int k = 0; k < (BIAS ? kNormCols : 3); ++k) {
    const int which = BIAS ? k : (k == 2 ? static_cast<int>(kColWPre) : k);
    if (!a.d_cols[which]) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int q = j * blockDim.x + tid;
      if (q < n)
        vec::store<PGG_F32, V>(a.partial, (static_cast<int64_t>(blockIdx.x) * kNormCols + which) * a.H
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
  float* mine = a.partial + static_cast<int64_t>(blockIdx.x) * kNormCols * a.H;
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
      float sum[3] = {0.0f, 0.0f, 0.0f};
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
    for (int64_t b = share * per; b < b1; ++b) sum += a.partial[(b * kNormCols + blockIdx.y) * a.H + i];
  }
  s_sum[share][lane] = sum;
  __syncthreads();
  if (share != 0 || i >= a.H) return;
  sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) sum += s_sum[k][lane];
  out[i] = sum;
}

// Rows of n vectors: vectors a thread (1, 2, 4 or, where rows are read from memory, 8) and threads;
// false: too long.
bool shape(int64_t n, bool eight, int* nv, int* threads) {
  for (*nv = 1; *nv <= (eight ? 8 : 4); *nv *= 2) {
    const int64_t need = ((n + *nv - 1) / *nv + 31) / 32 * 32;
    *threads = static_cast<int>(need);
    if (need <= (*nv == 1 ? 256 : *nv == 8 ? kMaxThreads : 512)) return true;
  }
  return false;
}

// Blocks of a kernel that an SM holds at once, by its registers and shared memory; asked once.
struct Fit {
  std::atomic<int> registers{0};
};

template <typename K>
cudaError_t blocks_that_fit(Fit* fit, K kern, int threads, int64_t smem, int* blocks) {
  int regs = fit->registers.load();
  if (regs == 0) {
    cudaFuncAttributes attr;
    const cudaError_t err = cudaFuncGetAttributes(&attr, kern);
    if (err != cudaSuccess) return err;
    regs = (attr.numRegs + 7) / 8 * 8;
    fit->registers.store(regs);
  }
  int64_t n = 65536 / (static_cast<int64_t>(regs) * threads);
  if (n > 226 * 1024 / (smem + 2048)) n = 226 * 1024 / (smem + 2048);
  *blocks = static_cast<int>(n < 1 ? 1 : n > 16 ? 16 : n);
  return cudaSuccess;
}

// Rows that a block keeps on their way: one to three, with `blocks` of them on an SM.
int ring_rows(int64_t row_bytes, int blocks) {
  const int64_t n = kRingBytes / blocks / row_bytes;
  return n < 1 ? 1 : n > 3 ? 3 : static_cast<int>(n);
}

// Bytes of a row of what the kernel reads.
template <int DT>
int64_t forward_bytes(const NormArgs& a) {
  constexpr int es = vec::elem_bytes(DT);
  return a.H * (es + (a.y ? (a.y_f32 ? 4 : es) : 0));
}
template <int DT>
int64_t backward_bytes(const NormArgs& a) {
  constexpr int es = vec::elem_bytes(DT);
  return a.H * ((a.d_r ? es : 0) + (a.y ? (a.y_f32 ? 4 : es) : 0) +
                (a.pre != PGG_NORM_NONE ? (a.dh_f32 ? 4 : es) + es : 0));
}

template <typename K>
cudaError_t launch_rows(SmemLimit* limit, K kern, int64_t grid, int threads, int64_t smem,
                        cudaStream_t stream, const NormArgs& a, int ring) {
  if (smem > 40 * 1024) {  // (beside what is static)
    const cudaError_t err = allow_smem(limit, kern, kRingBytes + 1024);
    if (err != cudaSuccess) return err;
  }
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(threads)),
                    static_cast<size_t>(smem), stream, 1, a, ring);
}

// Rms norms or none, a channel's gate or none: the kernels' short form.
bool lean(const NormArgs& a) {
  return a.post != PGG_NORM_LAYER && a.pre != PGG_NORM_LAYER &&
         (a.gate_kind == PGG_GATE_NONE || a.gate_kind == PGG_GATE_CHANNEL);
}

template <int DT, int V, int NV, bool LEAN, int THREADS>
cudaError_t launch_forward_t(const NormArgs& a, int threads, int num_sms, cudaStream_t stream) {
  constexpr bool kHeld = V >= 4;
  auto kern = block_norm_kernel<DT, V, NV, kHeld, LEAN, THREADS>;
  static Fit fit;
  static SmemLimit limit;
  int blocks;
  cudaError_t err = blocks_that_fit(&fit, kern, threads, 0, &blocks);
  if (err != cudaSuccess) return err;
  const int64_t row = forward_bytes<DT>(a);
  const int ring = kHeld ? ring_rows(row, blocks) : 0;
  err = blocks_that_fit(&fit, kern, threads, ring * row, &blocks);
  if (err != cudaSuccess) return err;
  const int64_t most = static_cast<int64_t>(num_sms) * blocks;
  return launch_rows(&limit, kern, a.T < most ? a.T : most, threads, ring * row, stream, a, ring);
}

template <int DT, int V, int NV, int THREADS>
cudaError_t launch_forward_f(const NormArgs& a, int threads, int num_sms, cudaStream_t stream) {
  if (V >= 4 && lean(a))
    return launch_forward_t<DT, V, NV, V >= 4, THREADS>(a, threads, num_sms, stream);
  return launch_forward_t<DT, V, NV, false, THREADS>(a, threads, num_sms, stream);
}

template <int DT, int V>
cudaError_t launch_forward(const NormArgs& a, int num_sms, cudaStream_t stream) {
  int nv, threads;
  if (shape(a.H / V, V < 4, &nv, &threads) && (V < 4 || forward_bytes<DT>(a) <= kRingBytes)) {
    if constexpr (V < 4) {
      if (nv == 1) return launch_forward_f<DT, V, 1, 256>(a, threads, num_sms, stream);
      if (nv == 2) return launch_forward_f<DT, V, 2, 512>(a, threads, num_sms, stream);
      if (nv == 8) return launch_forward_f<DT, V, 8, kMaxThreads>(a, threads, num_sms, stream);
    }
    return launch_forward_f<DT, V, 4, 512>(a, threads, num_sms, stream);
  }
  const int64_t grid = a.T < 2 * num_sms ? a.T : 2 * num_sms;
  return launch_pdl(block_norm_long_kernel<DT>, dim3(static_cast<unsigned>(grid)),
                    dim3(kMaxThreads), 0, stream, 1, a);
}

// Most blocks: one an SM of the longest rows (1500 x 1021, fp32: 45 us, with two 49, with four 51: each
// leaves columns' sums to add), of short ones as many as 1024 threads are (10000 x 333: 143 us, with
// half of them 170).
constexpr int64_t held_blocks(int threads) { return 152 * (threads >= 512 ? 1 : 1024 / threads); }

template <int DT, int V, int NV, bool LEAN, int THREADS>
cudaError_t launch_backward_t(const NormArgs& a, int threads, int64_t* grid, cudaStream_t stream) {
  constexpr bool kHeld = V >= 4;
  static SmemLimit limit;
  const int64_t row = backward_bytes<DT>(a), most = held_blocks(threads);
  const int64_t blocks = *grid < most ? *grid : most;
  *grid = blocks;
  const int ring = kHeld ? ring_rows(row, static_cast<int>((blocks + 151) / 152)) : 0;
  return launch_rows(&limit, block_norm_grad_kernel<DT, V, NV, kHeld, LEAN, THREADS>, blocks,
                     threads, ring * row, stream, a, ring);
}

template <int DT, int V, int NV, int THREADS>
cudaError_t launch_backward_f(const NormArgs& a, int threads, int64_t* grid, cudaStream_t stream) {
  if (V >= 4 && lean(a))
    return launch_backward_t<DT, V, NV, V >= 4, THREADS>(a, threads, grid, stream);
  return launch_backward_t<DT, V, NV, false, THREADS>(a, threads, grid, stream);
}

template <int DT, int V>
cudaError_t launch_backward(const NormArgs& a, int64_t* grid, cudaStream_t stream) {
  const int64_t n = a.H / V;
  // two vectors a thread (four: the columns' sums no longer fit the registers)
  const int nv = n <= 256 ? 1 : n <= 1024 ? 2 : n <= 2048 || V >= 4 ? 4 : 8;
  const int threads = static_cast<int>(((n + nv - 1) / nv + 31) / 32 * 32);
  if (threads <= (nv == 8 ? kMaxThreads : 512) && (V < 4 || backward_bytes<DT>(a) <= kRingBytes)) {
    if constexpr (V < 4) {
      if (nv == 1) return launch_backward_f<DT, V, 1, 256>(a, threads, grid, stream);
      if (nv == 2) return launch_backward_f<DT, V, 2, 512>(a, threads, grid, stream);
      if (nv == 8) return launch_backward_f<DT, V, 8, kMaxThreads>(a, threads, grid, stream);
    }
    return launch_backward_f<DT, V, 4, 512>(a, threads, grid, stream);
  }
  return launch_pdl(block_norm_grad_long_kernel<DT>,
                    dim3(static_cast<unsigned>(*grid)), dim3(kMaxThreads), 0, stream, 1, a);
}

}  // namespace

// One block an SM holds long rows; of short ones several do, and hide each other's sums.
int64_t norm_grad_blocks(int64_t T, int64_t H) {
  const int64_t most = 152 * (H > 4096 ? 1 : H > 1024 ? 2 : H > 512 ? 4 : 8);
  return T < most ? T : most;
}

// words: 16, 4 (two 16-bit elements, or one fp32) or 0 for rows that are read element by element.
cudaError_t launch_block_norm(int dtype, const NormArgs& a, int words, int num_sms,
                              cudaStream_t stream) {
  cudaError_t err;
  if (launch_block_norm_rows(dtype, a, words, num_sms, stream, &err)) return err;
  // (fp32 rows of 16-byte vectors come here with more than 8192 elements only: they are read one by one)
  if (dtype == PGG_F32) return launch_forward<PGG_F32, 1>(a, num_sms, stream);
  if (dtype == PGG_F16)
    return words == 16  ? launch_forward<PGG_F16, 8>(a, num_sms, stream)
           : words == 4 ? launch_forward<PGG_F16, 2>(a, num_sms, stream)
                        : launch_forward<PGG_F16, 1>(a, num_sms, stream);
  if (dtype == PGG_BF16)
    return words == 16  ? launch_forward<PGG_BF16, 8>(a, num_sms, stream)
           : words == 4 ? launch_forward<PGG_BF16, 2>(a, num_sms, stream)
                        : launch_forward<PGG_BF16, 1>(a, num_sms, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_block_norm_grad(int dtype, const NormArgs& a, int words, cudaStream_t stream) {
  cudaError_t err;
  int64_t grid = norm_grad_blocks(a.T, a.H);  // (a launch may take fewer)
  if (!launch_block_norm_rows_grad(dtype, a, words, stream, &err)) {
    if (dtype == PGG_F32)
      err = words == 16 ? launch_backward<PGG_F32, 4>(a, &grid, stream)
                        : launch_backward<PGG_F32, 1>(a, &grid, stream);
    else if (dtype == PGG_F16)
      err = words == 16  ? launch_backward<PGG_F16, 8>(a, &grid, stream)
            : words == 4 ? launch_backward<PGG_F16, 2>(a, &grid, stream)
                         : launch_backward<PGG_F16, 1>(a, &grid, stream);
    else if (dtype == PGG_BF16)
      err = words == 16  ? launch_backward<PGG_BF16, 8>(a, &grid, stream)
            : words == 4 ? launch_backward<PGG_BF16, 2>(a, &grid, stream)
                         : launch_backward<PGG_BF16, 1>(a, &grid, stream);
    else
      err = cudaErrorInvalidValue;
  }
  if (err != cudaSuccess) return err;
  for (int i = 0; i < kNormCols; ++i)
    if (a.d_cols[i])
      return launch_pdl(block_norm_cols_kernel, dim3(static_cast<unsigned>((a.H + 31) / 32), kNormCols),
                        dim3(256), 0, stream, 1, a, grid);
  return cudaSuccess;
}

}  // namespace pgg
