// The norms around a block and their gradient where a row's vectors of 16 bytes
// fit the threads of a block. With rms norms (or none) and a gate of one number a
// channel (or none), what decoder blocks use, p = gate (offset + w_post) and
// f = offset + w_pre stay in registers:
//
//     r = residual_scale x + p y^,  h = f r^,   v^ = v rstd(v)
//
//     g = d_r + rstd_r (d_h f - r^ mean(d_h f r^)),  d_x = residual_scale g
//     d_y = rstd_y (g p - y^ mean(g p y^))
//     C = sum over rows of g y^:  d_gate = (offset + w_post) C,  d_w_post = gate C
//     d_w_pre = sum over rows of d_h r^
//
// so a channel's gate and its weight share one sum. GEN: layer norms, biases and
// gates of a token or of every element too, parameters read for each row:
//
//     d = g gate where the gate belongs to the row, else g
//     C = sum d y^, D = sum d:  d_gate = (offset + w_post) C + b_post D (a channel's),
//     d_w_post, d_b_post = C, D (times a channel's gate);  d_b_pre = sum d_h
//
// Rows come through shared memory, up to four on their way. A row needs two rounds
// of sums over the block, one after the other; here row t's second round and row
// t+1's first go together, one barrier a row, so a layer norm's mean and variance
// are of one round: sums of v - k and (v - k)^2, k the mean of the row's first
// eight (four) elements. Where outliers among these have moved k by more than two
// deviations, the round is gone once more about the mean that it gave, so whatever the
// row holds, at most a factor of five is lost of the squares' precision.
//
// Memory bounds the short form (13500 x 7168, y fp32: forward 165 us, gradient 270,
// with floors of 142 and 228; y bf16 125 and 214). Two barriers a row, the sums of
// gate and weight apart and one element an instruction (now two, fma.f32x2) took
// 181 and 511. The general form, whose parameters come from the first level cache
// for each row, is bound by instructions: layer norms with biases 336 and 662, a
// gate of every element 256 and 660 (324 and 624, 252 and 627 without the second look
// at k, whose loop is written once: a round of its own for y took 806; where every row
// needs it, 18% and 22% more). It keeps fewer rows on their way (3 and 2), as shared
// memory is taken from that cache.

#include "pgg_block.h"
#include "pgg_block_sum.cuh"
#include "pgg_ops_launch.h"
#include "pgg_ptx.cuh"
#include "pgg_vec.cuh"

namespace pgg {
namespace {

// Two fp32 numbers in a pair of registers.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pair(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 both(float x) { return pair(x, x); }
__device__ __forceinline__ void split(F2 p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float added(F2 p) {
  float lo, hi;
  split(p, lo, hi);
  return lo + hi;
}

// Vector q of a row that begins at `row` in shared memory. (Rows lie there as in memory: copies of 16
// bytes whose neighbours go elsewhere are asked for one by one, which took 1.7 times as long. Vectors
// of 8 fp32 elements are read with two lanes on a bank for it.)
template <int DT, int V>
__device__ __forceinline__ void read(uint32_t row, uint32_t q, bool f32, F2 (&v)[V / 2]) {
  if (DT == PGG_F32 || f32) {
#pragma unroll
    for (int h = 0; h < V / 4; ++h)
      asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                   : "=l"(v[2 * h].v), "=l"(v[2 * h + 1].v)
                   : "r"(row + q * (V * 4) + h * 16)
                   : "memory");
  } else {
    uint32_t w[4];
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(row + q * 16)
                 : "memory");
#pragma unroll
    for (int c = 0; c < V / 2; ++c) {
      float lo, hi;
      vec::unpack2<DT == PGG_F32 ? PGG_F16 : DT>(w[c & 3], lo, hi);
      v[c] = pair(lo, hi);
    }
  }
}
// The block's vectors [first, first + threads) of a row at p, of `n` vectors, to `row`. A thread copies
// what it reads itself, but for vectors of 8 fp32 elements: there a warp copies its 1 KB chunk by
// chunk of 16 bytes in memory's order (each by its own reader would ask for every sector twice), so
// its lanes meet (__syncwarp) between the copies and the reads.
template <int DT, int V>
__device__ __forceinline__ void fetch(uint32_t row, bool f32, const char* p, int first, int n) {
  if (V == 8 && DT != PGG_F32 && f32) {
    const int chunk = (first + (threadIdx.x & ~31)) * 2 + (threadIdx.x & 31);
#pragma unroll
    for (int h = 0; h < 64; h += 32)
      if (chunk + h < 2 * n) ptx::cp_async_16(row + (chunk + h) * 16, p + (chunk + h) * 16, 16);
  } else {
    const int q = first + threadIdx.x;
    if (q < n) ptx::cp_async_16(row + q * 16, p + q * 16, 16);
  }
}
template <int DT, int V>
__device__ __forceinline__ void store(void* p, int64_t element, const F2 (&v)[V / 2]) {
  float x[V];
#pragma unroll
  for (int c = 0; c < V / 2; ++c) split(v[c], x[2 * c], x[2 * c + 1]);
  vec::store<DT, V>(p, element, x);
}

// offset + w of V columns (1 where there is no weight), or a channel's gate.
template <int DT, int V>
__device__ __forceinline__ void factor(const void* w, bool f32, float offset, int64_t i,
                                       float (&f)[V]) {
  if (w) vec::load_or_f32<DT, V>(w, f32, i, f);
#pragma unroll
  for (int c = 0; c < V; ++c) f[c] = w ? f[c] + offset : 1.0f;
}
// The product of two factors, or (w2 null) the first.
template <int DT, int V>
__device__ __forceinline__ void factors(const void* w, const void* w2, bool f32, float offset,
                                        int64_t i, F2 (&p)[V / 2]) {
  float f[V], g[V];
  factor<DT, V>(w, f32, offset, i, f);
  factor<DT, V>(w2, f32, 0.0f, i, g);
#pragma unroll
  for (int c = 0; c < V / 2; ++c) p[c] = pair(f[2 * c] * g[2 * c], f[2 * c + 1] * g[2 * c + 1]);
}

// A bias of V columns, or 0.
template <int DT, int V>
__device__ __forceinline__ void bias(const void* b, bool f32, int64_t i, F2 (&v)[V / 2]) {
  float x[V] = {};
  if (b) vec::load_or_f32<DT, V>(b, f32, i, x);
#pragma unroll
  for (int c = 0; c < V / 2; ++c) v[c] = pair(x[2 * c], x[2 * c + 1]);
}
// The mean of the V elements from `element` on, a row's first, from memory (in shared memory another warp's copies).
template <int DT, int V>
__device__ __forceinline__ float first_mean(const void* p, bool f32, int64_t element) {
  float v[V], sum = 0.0f;
  vec::load_or_f32<DT, V>(p, f32, element, v);
#pragma unroll
  for (int c = 0; c < V; ++c) sum += v[c];
  return sum * (1.0f / V);
}

// Mean and 1 / deviation from the sums of v - k and (v - k)^2; `from_k`: mean - k.
struct Stat {
  float mean, from_k, rstd;
};
__device__ __forceinline__ Stat stat_of(int kind, float k, float sum, float squares, float inv_h,
                                        float eps) {
  Stat s = {0.0f, 0.0f, 1.0f};
  if (kind == PGG_NORM_NONE) return s;
  float var = squares * inv_h;
  if (kind == PGG_NORM_LAYER) {
    s.from_k = sum * inv_h;
    s.mean = k + s.from_k;
    var = fmaf(-s.from_k, s.from_k, var);
    if (var < 0.0f) var = 0.0f;  // (NaN stays)
  }
  s.rstd = 1.0f / sqrtf(var + eps);
  return s;
}

// k lies so far from the mean that the variance has lost bits: the sums are of v - k and (v - k)^2.
__device__ __forceinline__ bool too_far(float sum, float squares, float inv_h) {
  const float from_k = sum * inv_h;
  return from_k * from_k > 4.0f * fmaf(-from_k, from_k, squares * inv_h);
}

// The copies of all rows but the `behind` last ones have landed, for the warp.
__device__ __forceinline__ void wait_rows(int behind) {
  if (behind >= 3)
    ptx::cp_async_wait<3>();
  else if (behind == 2)
    ptx::cp_async_wait<2>();
  else if (behind == 1)
    ptx::cp_async_wait<1>();
  else
    ptx::cp_async_wait<0>();
  __syncwarp();
}

// FY: y is fp32 (else of the dtype, as all of an fp32 call are); GEN: as a.y_f32 says.
template <int DT, int V, int NV, bool GEN, bool FY, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) block_norm_rows_kernel(const NormArgs a, const int ring) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ BlockSum<4> s;
  constexpr int P = V / 2, kBytes = vec::elem_bytes(DT);
  int turn = 0;
  ptx::griddep_wait();
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const int n = static_cast<int>(a.H / V), tid = threadIdx.x;
  const bool post = a.post != PGG_NORM_NONE, pre = a.pre != PGG_NORM_NONE, have_y = a.y != nullptr;
  const bool y32 = GEN ? a.y_f32 : FY, p32 = a.p_f32;
  const bool token = GEN && a.gate_kind == PGG_GATE_TOKEN, full = GEN && a.gate_kind == PGG_GATE_FULL;
  const bool post_mean = GEN && a.post == PGG_NORM_LAYER, pre_mean = GEN && a.pre == PGG_NORM_LAYER;
  const void* channel = a.gate_kind == PGG_GATE_CHANNEL ? a.gate : nullptr;
  const uint32_t part = n * 16, base = ptx::smem_addr(smem), wide = DT == PGG_F32 ? 1 : 2;
  const uint32_t y_at = part, gate_at = y_at + (have_y ? part * (y32 ? wide : 1) : 0);
  const uint32_t slot_bytes = gate_at + (full ? part * (p32 ? wide : 1) : 0);
  const int64_t step = gridDim.x * a.H;
  const F2 scale = both(a.residual_scale);
  auto fetch_row = [&](uint32_t slot, int64_t t) {
    __syncwarp();
    if (t < a.T) {
      const int64_t e = t * a.H;
      const char *x = static_cast<const char*>(a.x) + e * kBytes,
                 *y = static_cast<const char*>(a.y) + e * (y32 ? 4 : kBytes),
                 *gate = static_cast<const char*>(a.gate) + e * (p32 ? 4 : kBytes);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int q = j * blockDim.x;
        fetch<DT, V>(base + slot, false, x, q, n);
        if (have_y) fetch<DT, V>(base + slot + y_at, y32, y, q, n);
        if (full) fetch<DT, V>(base + slot + gate_at, p32, gate, q, n);
      }
    }
    ptx::cp_async_commit();
  };
  int64_t t = blockIdx.x, e = t * a.H + tid * V;  // the row, and the thread's first element of it
  for (int i = 0; i < ring; ++i) fetch_row(i * slot_bytes, t + i * gridDim.x);
  F2 p[GEN ? 1 : NV][P], f[GEN ? 1 : NV][P];
#pragma unroll
  for (int j = 0; !GEN && j < NV; ++j) {
    const int q = j * blockDim.x + tid;
    if (q >= n) continue;
    factors<DT, V>(a.w_post, channel, p32, a.weight_offset, q * V, p[GEN ? 0 : j]);
    factors<DT, V>(a.w_pre, nullptr, p32, a.weight_offset, q * V, f[GEN ? 0 : j]);
  }
  float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // of y - k, (y - k)^2 (the next row's); r, r^2
  // of row t: k, and its token's gate
  auto scalars = [&](int64_t t, float& k, float& gate) {
    float one[1] = {1.0f};
    if (token) vec::load_or_f32<DT, 1>(a.gate, p32, t, one);
    gate = one[0];
    k = post_mean ? first_mean<DT, V>(a.y, y32, t * a.H) : 0.0f;
  };
  float k, token_gate, k_next = 0.0f, gate_next = 1.0f;
  scalars(t, k, token_gate);
  // the first two sums of the row in `slot`
  auto first_pass = [&](uint32_t slot, float k) {
    F2 sum = both(0.0f), squares = both(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t q = j * blockDim.x + tid;
      if (static_cast<int>(q) >= n) continue;
      F2 y[P];
      read<DT, V>(base + slot + y_at, q, y32, y);
#pragma unroll
      for (int c = 0; c < P; ++c) {
        if constexpr (GEN) {
          y[c] = add2(y[c], both(-k));
          sum = add2(sum, y[c]);
        }
        squares = fma2(y[c], y[c], squares);
      }
    }
    sums[0] = GEN ? added(sum) : 0.0f;
    sums[1] = added(squares);
  };
  wait_rows(ring - 1);
#pragma unroll 1
  for (bool again = false; post; again = true) {
    first_pass(0, k);
    block_sum(&s, &turn, sums);
    if (!GEN || again || !post_mean || !too_far(sums[0], sums[1], inv_h)) break;
    k = fmaf(sums[0], inv_h, k);
  }
  uint32_t slot = 0;
  for (; t < a.T; t += gridDim.x, e += step) {
    const Stat of_y = stat_of(a.post, k, sums[0], sums[1], inv_h, a.eps);
    const F2 rstd_y = both(of_y.rstd), mean_y = both(-of_y.mean), row_gate = both(token_gate);
    const uint32_t next = slot + slot_bytes == ring * slot_bytes ? 0 : slot + slot_bytes;
    if (GEN && t + gridDim.x < a.T) scalars(t + gridDim.x, k_next, gate_next);
    F2 r[NV][P], sum = both(0.0f), squares = both(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t q = j * blockDim.x + tid;
      if (static_cast<int>(q) >= n) continue;
      read<DT, V>(base + slot, q, false, r[j]);
#pragma unroll
      for (int c = 0; c < P; ++c) r[j][c] = mul2(r[j][c], scale);
      if (have_y) {
        F2 y[P];
        read<DT, V>(base + slot + y_at, q, y32, y);
        if constexpr (GEN) {
          F2 w[P], b[P];
          factors<DT, V>(a.w_post, nullptr, p32, a.weight_offset, q * V, w);
          bias<DT, V>(a.b_post, p32, q * V, b);
#pragma unroll
          for (int c = 0; c < P; ++c)
            y[c] = fma2(mul2(add2(y[c], mean_y), rstd_y), w[c], b[c]);
          if (full)
            read<DT, V>(base + slot + gate_at, q, p32, w);
          else
            factors<DT, V>(nullptr, channel, p32, 0.0f, q * V, w);
#pragma unroll
          for (int c = 0; c < P; ++c) r[j][c] = fma2(y[c], token ? row_gate : w[c], r[j][c]);
        } else {
#pragma unroll
          for (int c = 0; c < P; ++c) r[j][c] = fma2(mul2(y[c], rstd_y), p[j][c], r[j][c]);
        }
      }
      if (a.r) store<DT, V>(a.r, e + j * blockDim.x * V, r[j]);
#pragma unroll
      for (int c = 0; c < P; ++c) {
        if constexpr (GEN) sum = add2(sum, r[j][c]);
        squares = fma2(r[j][c], r[j][c], squares);
      }
    }
    sums[0] = sums[1] = 0.0f;
    sums[2] = GEN ? added(sum) : 0.0f;
    sums[3] = added(squares);
    fetch_row(slot, t + ring * gridDim.x);
    wait_rows(ring - 1);
    const bool more = post && t + gridDim.x < a.T;
#pragma unroll 1
    for (bool again = false;; again = true) {
      if (more) first_pass(next, k_next);
      if (post || pre) block_sum(&s, &turn, sums);
      // (the same bits in every thread, so all of them go again or none)
      if (!GEN || again || !post_mean || !more || !too_far(sums[0], sums[1], inv_h)) break;
      k_next = fmaf(sums[0], inv_h, k_next);
      if (tid != 0) sums[2] = sums[3] = 0.0f;  // (r's are there already, once)
    }
    if (pre) {
      float mean = 0.0f, var = sums[3] * inv_h;
      if (pre_mean) {
        mean = sums[2] * inv_h;
        F2 centred = both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (static_cast<int>(j * blockDim.x + tid) >= n) continue;
#pragma unroll
          for (int c = 0; c < P; ++c) {
            const F2 d = add2(r[j][c], both(-mean));
            centred = fma2(d, d, centred);
          }
        }
        float one[1] = {added(centred)};
        block_sum(&s, &turn, one);
        var = one[0] * inv_h;
      }
      const F2 rstd = both(1.0f / sqrtf(var + a.eps));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t q = j * blockDim.x + tid;
        if (static_cast<int>(q) >= n) continue;
        if constexpr (GEN) {
          F2 w[P], b[P];
          factors<DT, V>(a.w_pre, nullptr, p32, a.weight_offset, q * V, w);
          bias<DT, V>(a.b_pre, p32, q * V, b);
#pragma unroll
          for (int c = 0; c < P; ++c)
            r[j][c] = fma2(mul2(add2(r[j][c], both(-mean)), rstd), w[c], b[c]);
        } else {
#pragma unroll
          for (int c = 0; c < P; ++c) r[j][c] = mul2(mul2(r[j][c], rstd), f[j][c]);
        }
        store<DT, V>(a.h, e + j * blockDim.x * V, r[j]);
      }
    }
    slot = next;
    k = k_next;
    token_gate = gate_next;
  }
}

// FY, FH: y, d_h are fp32; GEN: as a.y_f32 and a.dh_f32 say.
template <int DT, int V, int NV, bool GEN, bool FY, bool FH, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 1 : 2)
    block_norm_rows_grad_kernel(const NormArgs a, const int ring) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int P = V / 2, kBytes = vec::elem_bytes(DT), kSums = GEN ? 8 : 4;
  __shared__ BlockSum<kSums> s;
  int turn = 0;
  ptx::griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->status = 0;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const int n = static_cast<int>(a.H / V), tid = threadIdx.x;
  const bool post = a.post != PGG_NORM_NONE, pre = a.pre != PGG_NORM_NONE;
  const bool have_y = a.y != nullptr, have_dr = a.d_r != nullptr;
  const bool y32 = GEN ? a.y_f32 : FY, h32 = GEN ? a.dh_f32 : FH, p32 = a.p_f32;
  const bool token = GEN && a.gate_kind == PGG_GATE_TOKEN, full = GEN && a.gate_kind == PGG_GATE_FULL;
  const bool post_mean = GEN && a.post == PGG_NORM_LAYER, pre_mean = GEN && a.pre == PGG_NORM_LAYER;
  const void* channel = a.gate_kind == PGG_GATE_CHANNEL ? a.gate : nullptr;
  const uint32_t part = n * 16, base = ptx::smem_addr(smem), wide = DT == PGG_F32 ? 1 : 2;
  const uint32_t h_at = part, g_at = h_at + part * (h32 ? wide : 1), y_at = g_at + part;
  const uint32_t gate_at = y_at + part * (y32 ? wide : 1);
  const uint32_t slot_bytes = gate_at + (full ? part * (p32 ? wide : 1) : 0);
  const int64_t step = gridDim.x * a.H;
  const F2 scale = both(a.residual_scale);
  auto fetch_row = [&](uint32_t slot, int64_t t) {
    __syncwarp();
    if (t < a.T) {
      const int64_t e = t * a.H;
      const char *r = static_cast<const char*>(a.x) + e * kBytes,
                 *dh = static_cast<const char*>(a.d_h) + e * (h32 ? 4 : kBytes),
                 *dr = static_cast<const char*>(a.d_r) + e * kBytes,
                 *y = static_cast<const char*>(a.y) + e * (y32 ? 4 : kBytes),
                 *gate = static_cast<const char*>(a.gate) + e * (p32 ? 4 : kBytes);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int q = j * blockDim.x;
        if (pre) {
          fetch<DT, V>(base + slot, false, r, q, n);
          fetch<DT, V>(base + slot + h_at, h32, dh, q, n);
        }
        if (have_dr) fetch<DT, V>(base + slot + g_at, false, dr, q, n);
        if (have_y) fetch<DT, V>(base + slot + y_at, y32, y, q, n);
        if (full) fetch<DT, V>(base + slot + gate_at, p32, gate, q, n);
      }
    }
    ptx::cp_async_commit();
  };
  int64_t t = blockIdx.x, e = t * a.H + tid * V;
  for (int i = 0; i < ring; ++i) fetch_row(i * slot_bytes, t + i * gridDim.x);
  F2 p[NV][P], f[NV][P];  // (GEN: used up between two barriers, not kept)
  F2 c_post[NV][P], c_pre[NV][P], d_post[GEN ? NV : 1][P], d_pre[GEN ? NV : 1][P];
  auto load_p = [&](int j, uint32_t q) {
    factors<DT, V>(a.w_post, channel, p32, a.weight_offset, q * V, p[j]);
  };
  auto load_f = [&](int j, uint32_t q) {
    factors<DT, V>(a.w_pre, nullptr, p32, a.weight_offset, q * V, f[j]);
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int q = j * blockDim.x + tid;
#pragma unroll
    for (int c = 0; c < P; ++c) {
      c_post[j][c] = c_pre[j][c] = both(0.0f);
      if constexpr (GEN) d_post[j][c] = d_pre[j][c] = both(0.0f);
    }
    if (GEN || q >= n) continue;
    load_p(j, q);
    load_f(j, q);
  }
  // of the next row r^2, d_h f r; of the row y^2, g p y. GEN: of the next row (r - k)^2, d_h f (r - k),
  // r - k, d_h f, (y - k)^2, y - k; of the row g p (y - mean), g p
  constexpr int kYY = GEN ? 4 : 2, kY1 = GEN ? 5 : 0, kWY = GEN ? 6 : 3, kW1 = GEN ? 7 : 0;
  constexpr int kR1 = GEN ? 2 : 0, kU1 = GEN ? 3 : 0;
  float sums[kSums] = {};
  // of row t: r's k, y's k, and its token's gate
  struct Scalars {
    float r, y, gate;
  };
  auto scalars = [&](int64_t t) {
    float one[1] = {1.0f};
    if (token) vec::load_or_f32<DT, 1>(a.gate, p32, t, one);
    return Scalars{pre_mean ? first_mean<DT, V>(a.x, false, t * a.H) : 0.0f,
                   post_mean ? first_mean<DT, V>(a.y, y32, t * a.H) : 0.0f, one[0]};
  };
  Scalars now = scalars(t), later = {0.0f, 0.0f, 1.0f};
  // those of the next row, in `slot`
  auto first_pass = [&](uint32_t slot, const Scalars& of) {
    F2 rr = both(0.0f), ur = both(0.0f), r1 = both(0.0f), u1 = both(0.0f);
    F2 yy = both(0.0f), y1 = both(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t q = j * blockDim.x + tid;
      if (static_cast<int>(q) >= n) continue;
      if (pre) {
        F2 r[P], dh[P];
        read<DT, V>(base + slot, q, false, r);
        read<DT, V>(base + slot + h_at, q, h32, dh);
        if constexpr (GEN) load_f(j, q);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          const F2 u = mul2(dh[c], f[j][c]);
          if constexpr (GEN) {
            r[c] = add2(r[c], both(-of.r));
            r1 = add2(r1, r[c]);
            u1 = add2(u1, u);
          }
          rr = fma2(r[c], r[c], rr);
          ur = fma2(u, r[c], ur);
        }
      }
      if (GEN && post) {
        F2 y[P];
        read<DT, V>(base + slot + y_at, q, y32, y);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          y[c] = add2(y[c], both(-of.y));
          y1 = add2(y1, y[c]);
          yy = fma2(y[c], y[c], yy);
        }
      }
    }
    sums[0] = added(rr);
    sums[1] = added(ur);
    if constexpr (GEN) {
      sums[kR1] = added(r1);
      sums[kU1] = added(u1);
      sums[kYY] = added(yy);
      sums[kY1] = added(y1);
    }
  };
  // The block's sums, with the next row's (in `slot`, where there is one) gone over once more about
  // the means where k was too far from one of them: the same bits in every thread, so all go or none.
  auto sum_up = [&](uint32_t slot, bool there, Scalars& of) {
#pragma unroll 1
    for (bool again = false;; again = true) {
      if (there) first_pass(slot, of);
      block_sum(&s, &turn, sums);
      if (!GEN || again || !there) break;
      const bool far_r = pre_mean && too_far(sums[kR1], sums[0], inv_h);
      const bool far_y = post_mean && too_far(sums[kY1], sums[kYY], inv_h);
      if (!far_r && !far_y) break;
      if (far_r) of.r = fmaf(sums[kR1], inv_h, of.r);
      if (far_y) of.y = fmaf(sums[kY1], inv_h, of.y);
      if (tid != 0) sums[kWY] = sums[kW1] = 0.0f;  // (the row's are there already, once)
    }
  };
  wait_rows(ring - 1);
  if (pre || (GEN && post)) sum_up(0, true, now);
  uint32_t slot = 0;
  for (; t < a.T; t += gridDim.x, e += step) {
    const Stat of_r = stat_of(a.pre, now.r, GEN ? sums[kR1] : 0.0f, sums[0], inv_h, a.eps);
    Stat of_y = {};
    if constexpr (GEN) of_y = stat_of(a.post, now.y, sums[kY1], sums[kYY], inv_h, a.eps);
    const float u_r = GEN ? sums[kU1] : 0.0f, uv = fmaf(-of_r.from_k, u_r, sums[1]);
    const F2 rstd_r = both(of_r.rstd), mean_r = both(-of_r.mean),
             along_r = both(-(uv * of_r.rstd * inv_h) * of_r.rstd),
             centre_r = both(pre_mean ? -u_r * inv_h * of_r.rstd : 0.0f);
    const uint32_t next = slot + slot_bytes == ring * slot_bytes ? 0 : slot + slot_bytes;
    if (GEN && t + gridDim.x < a.T) later = scalars(t + gridDim.x);
    F2 g[NV][P], yy = both(0.0f), wy = both(0.0f), w1 = both(0.0f), gb = both(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t q = j * blockDim.x + tid;
      if (static_cast<int>(q) >= n) continue;
      if (have_dr) {
        read<DT, V>(base + slot + g_at, q, false, g[j]);
      } else {
#pragma unroll
        for (int c = 0; c < P; ++c) g[j][c] = both(0.0f);
      }
      if (pre) {
        F2 r[P], dh[P];
        read<DT, V>(base + slot, q, false, r);
        read<DT, V>(base + slot + h_at, q, h32, dh);
        if constexpr (GEN) load_f(j, q);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          if constexpr (GEN) {
            r[c] = add2(r[c], mean_r);
            d_pre[j][c] = add2(d_pre[j][c], dh[c]);
            g[j][c] = add2(g[j][c], centre_r);
          }
          const F2 v = mul2(r[c], rstd_r);
          c_pre[j][c] = fma2(dh[c], v, c_pre[j][c]);
          g[j][c] = fma2(v, along_r, fma2(mul2(dh[c], f[j][c]), rstd_r, g[j][c]));
        }
      }
      F2 d[P];
#pragma unroll
      for (int c = 0; c < P; ++c) d[c] = mul2(g[j][c], scale);
      store<DT, V>(a.r, e + j * blockDim.x * V, d);
      if (post || token) {
        F2 y[P];
        read<DT, V>(base + slot + y_at, q, y32, y);
        if constexpr (GEN) {
          load_p(j, q);
          if (full) {
            read<DT, V>(base + slot + gate_at, q, p32, d);
#pragma unroll
            for (int c = 0; c < P; ++c) p[j][c] = mul2(p[j][c], d[c]);
          }
          if (token && a.b_post) {
            bias<DT, V>(a.b_post, p32, q * V, d);
#pragma unroll
            for (int c = 0; c < P; ++c) gb = fma2(g[j][c], d[c], gb);
          }
        }
#pragma unroll
        for (int c = 0; c < P; ++c) {
          const F2 w = mul2(g[j][c], p[j][c]);
          if constexpr (GEN) {
            y[c] = add2(y[c], both(-of_y.mean));
            w1 = add2(w1, w);
          } else {
            yy = fma2(y[c], y[c], yy);
          }
          wy = fma2(w, y[c], wy);
        }
      }
    }
    if constexpr (!GEN) sums[kYY] = added(yy);
    sums[kWY] = added(wy);
    if constexpr (GEN) sums[kW1] = added(w1);
    wait_rows(ring - 2);
    if (post || pre || token) sum_up(next, (pre || GEN) && t + gridDim.x < a.T, later);
    if (have_y) {
      if constexpr (!GEN) of_y = stat_of(a.post, 0.0f, 0.0f, sums[kYY], inv_h, a.eps);
      const float w_sum = GEN ? sums[kW1] : 0.0f, wv = sums[kWY];
      if (token) {
        float b[1] = {added(gb)};
        if (a.b_post) block_sum(&s, &turn, b);
        if (tid == 0) static_cast<float*>(a.d_gate)[t] = fmaf(wv, of_y.rstd, b[0]);
      }
      const F2 rstd_y = both(of_y.rstd), mean_y = both(-of_y.mean), row_gate = both(now.gate),
               along_y = both(-(wv * now.gate * of_y.rstd * inv_h) * of_y.rstd),
               centre_y = both(post_mean ? -w_sum * now.gate * inv_h * of_y.rstd : 0.0f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t q = j * blockDim.x + tid;
        if (static_cast<int>(q) >= n) continue;
        F2 y[P], d[P];
        read<DT, V>(base + slot + y_at, q, y32, y);
        if constexpr (GEN) {
          F2 gate[P];
          load_p(j, q);
          if (full) read<DT, V>(base + slot + gate_at, q, p32, gate);
#pragma unroll
          for (int c = 0; c < P; ++c) {
            y[c] = mul2(add2(y[c], mean_y), rstd_y);
            d[c] = full ? mul2(g[j][c], gate[c]) : token ? mul2(g[j][c], row_gate) : g[j][c];
            c_post[j][c] = fma2(d[c], y[c], c_post[j][c]);
            d_post[j][c] = add2(d_post[j][c], d[c]);
          }
          if (full) {
            bias<DT, V>(a.b_post, p32, q * V, gate);
#pragma unroll
            for (int c = 0; c < P; ++c) gate[c] = mul2(g[j][c], fma2(y[c], p[j][c], gate[c]));
            if (p32)
              store<PGG_F32, V>(a.d_gate, e + j * blockDim.x * V, gate);
            else
              store<DT, V>(a.d_gate, e + j * blockDim.x * V, gate);
          }
#pragma unroll
          for (int c = 0; c < P; ++c) {
            d[c] = mul2(mul2(d[c], p[j][c]), rstd_y);
            if (post) d[c] = add2(fma2(y[c], along_y, d[c]), centre_y);
          }
        } else {
#pragma unroll
          for (int c = 0; c < P; ++c) {
            const F2 v = mul2(y[c], rstd_y);
            c_post[j][c] = fma2(g[j][c], v, c_post[j][c]);
            d[c] = mul2(mul2(g[j][c], p[j][c]), rstd_y);
            if (post) d[c] = fma2(v, along_y, d[c]);
          }
        }
        store<DT, V>(a.h, e + j * blockDim.x * V, d);
      }
    }
    fetch_row(slot, t + ring * gridDim.x);
    slot = next;
    now = later;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int q = j * blockDim.x + tid;
    if (q >= n) continue;
    float* at = a.partial + static_cast<int64_t>(blockIdx.x) * kNormCols * a.H + q * V;
    F2 w[P], out[P];
    if (a.d_cols[kColGate]) {
      factors<DT, V>(a.w_post, nullptr, p32, a.weight_offset, q * V, w);
#pragma unroll
      for (int c = 0; c < P; ++c) out[c] = mul2(c_post[j][c], w[c]);
      if constexpr (GEN) {
        bias<DT, V>(a.b_post, p32, q * V, w);
#pragma unroll
        for (int c = 0; c < P; ++c) out[c] = fma2(d_post[j][c], w[c], out[c]);
      }
      store<PGG_F32, V>(at + kColGate * a.H, 0, out);
    }
    factors<DT, V>(nullptr, channel, p32, 0.0f, q * V, w);
    if (a.d_cols[kColWPost]) {
#pragma unroll
      for (int c = 0; c < P; ++c) out[c] = mul2(c_post[j][c], w[c]);
      store<PGG_F32, V>(at + kColWPost * a.H, 0, out);
    }
    if (a.d_cols[kColWPre]) store<PGG_F32, V>(at + kColWPre * a.H, 0, c_pre[j]);
    if constexpr (GEN) {
      if (a.d_cols[kColBPost]) {
#pragma unroll
        for (int c = 0; c < P; ++c) out[c] = mul2(d_post[j][c], w[c]);
        store<PGG_F32, V>(at + kColBPost * a.H, 0, out);
      }
      if (a.d_cols[kColBPre]) store<PGG_F32, V>(at + kColBPre * a.H, 0, d_pre[j]);
    }
  }
}

// Shared memory of a block with `blocks` of them on an SM, beside what is static.
constexpr int64_t ring_bytes(int64_t blocks) { return 228 * 1024 / blocks - 3 * 1024; }

template <typename K>
cudaError_t launch_ring(SmemLimit* limit, K kern, int64_t grid, int threads, int64_t row,
                        int64_t blocks, int most, cudaStream_t stream, const NormArgs& a) {
  const cudaError_t err = allow_smem(limit, kern, ring_bytes(1));
  if (err != cudaSuccess) return err;
  const int64_t rows = ring_bytes(blocks) / row;
  const int ring = static_cast<int>(rows < most ? rows : most);
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(threads)),
                    static_cast<size_t>(ring * row), stream, 1, a, ring);
}

struct Shape {
  int threads, nv;
  int64_t row;  // bytes of a slot
  bool fits, general;
};

constexpr int kThreads = 512;  // of a block, at most, with 16 elements each

Shape shape_of(const NormArgs& a, int dtype, int words, bool backward) {
  const int es = dtype == PGG_F32 ? 4 : 2;
  const int64_t n = a.H / (16 / es);
  Shape s;
  s.nv = n <= 256 ? 1 : es == 2 || n <= 1024 ? 2 : 4;
  s.threads = static_cast<int>(((n + s.nv - 1) / s.nv + 31) / 32 * 32);
  const int y = a.y_f32 ? 4 : es, gate = a.gate_kind != PGG_GATE_FULL ? 0 : a.p_f32 ? 4 : es;
  // (the gradient's slot has room for all tensors)
  s.row = a.H * (gate + (backward ? 2 * es + (a.dh_f32 ? 4 : es) + y : es + (a.y ? y : 0)));
  s.general = a.post == PGG_NORM_LAYER || a.pre == PGG_NORM_LAYER || a.b_post || a.b_pre ||
              a.d_cols[kColBPost] || a.d_cols[kColBPre] || a.gate_kind == PGG_GATE_TOKEN ||
              a.gate_kind == PGG_GATE_FULL;
  s.fits = words == 16 && n <= s.nv * kThreads &&
           2 * s.row <= ring_bytes(1);
  return s;
}

// So many blocks on an SM that each has room for two rows.
int64_t blocks_for(const Shape& s, int64_t blocks) {
  while (blocks > 1 && ring_bytes(blocks) < 2 * s.row) --blocks;
  return blocks;
}

template <int DT, int V, int NV, bool GEN, bool FY, int THREADS>
cudaError_t forward(const NormArgs& a, const Shape& s, int num_sms, cudaStream_t stream) {
  static SmemLimit limit;
  // (64 registers a thread, 92 and 104)
  int64_t blocks = (GEN ? 576 : NV * V <= 8 ? 1024 : 704) / s.threads;
  blocks = blocks_for(s, blocks < 1 ? 1 : blocks > 8 ? 8 : blocks);
  const int64_t most = blocks * num_sms;
  return launch_ring(&limit, block_norm_rows_kernel<DT, V, NV, GEN, FY, THREADS>,
                     a.T < most ? a.T : most, s.threads, s.row, blocks, GEN ? 3 : 4, stream, a);
}
template <int DT, int V, bool GEN, bool FY>
cudaError_t forward_of(const NormArgs& a, const Shape& s, int num_sms, cudaStream_t stream) {
  if (s.nv == 1) return forward<DT, V, 1, GEN, FY, 256>(a, s, num_sms, stream);
  if constexpr (V == 4)
    if (s.nv == 4) return forward<DT, V, 4, GEN, FY, kThreads>(a, s, num_sms, stream);
  return forward<DT, V, 2, GEN, FY, kThreads>(a, s, num_sms, stream);
}
template <int DT>
cudaError_t forward_16(const NormArgs& a, const Shape& s, int num_sms, cudaStream_t stream) {
  if (s.general) return forward_of<DT, 8, true, false>(a, s, num_sms, stream);
  return a.y_f32 ? forward_of<DT, 8, false, true>(a, s, num_sms, stream)
                 : forward_of<DT, 8, false, false>(a, s, num_sms, stream);
}

template <int DT, int V, int NV, bool GEN, bool FY, bool FH, int THREADS>
cudaError_t backward(const NormArgs& a, const Shape& s, cudaStream_t stream) {
  static SmemLimit limit;
  const int64_t grid = norm_grad_blocks(a.T, a.H);
  return launch_ring(&limit, block_norm_rows_grad_kernel<DT, V, NV, GEN, FY, FH, THREADS>, grid,
                     s.threads, s.row, blocks_for(s, (grid + 151) / 152), GEN ? 2 : 4,
                     stream, a);
}
template <int DT, int V, bool GEN, bool FY, bool FH>
cudaError_t backward_of(const NormArgs& a, const Shape& s, cudaStream_t stream) {
  if (s.nv == 1) return backward<DT, V, 1, GEN, FY, FH, 256>(a, s, stream);
  if constexpr (V == 4)
    if (s.nv == 4) return backward<DT, V, 4, GEN, FY, FH, kThreads>(a, s, stream);
  return backward<DT, V, 2, GEN, FY, FH, kThreads>(a, s, stream);
}
template <int DT>
cudaError_t backward_16(const NormArgs& a, const Shape& s, cudaStream_t stream) {
  if (s.general) return backward_of<DT, 8, true, false, false>(a, s, stream);
  if (a.y_f32)
    return a.dh_f32 ? backward_of<DT, 8, false, true, true>(a, s, stream)
                    : backward_of<DT, 8, false, true, false>(a, s, stream);
  return a.dh_f32 ? backward_of<DT, 8, false, false, true>(a, s, stream)
                  : backward_of<DT, 8, false, false, false>(a, s, stream);
}

}  // namespace

bool launch_block_norm_rows(int dtype, const NormArgs& a, int words, int num_sms,
                            cudaStream_t stream, cudaError_t* err) {
  const Shape s = shape_of(a, dtype, words, false);
  if (!s.fits) return false;
  if (dtype == PGG_F32)
    *err = s.general ? forward_of<PGG_F32, 4, true, false>(a, s, num_sms, stream)
                     : forward_of<PGG_F32, 4, false, false>(a, s, num_sms, stream);
  else
    *err = dtype == PGG_F16 ? forward_16<PGG_F16>(a, s, num_sms, stream)
                            : forward_16<PGG_BF16>(a, s, num_sms, stream);
  return true;
}

bool launch_block_norm_rows_grad(int dtype, const NormArgs& a, int words, cudaStream_t stream,
                                 cudaError_t* err) {
  const Shape s = shape_of(a, dtype, words, true);
  if (!s.fits) return false;
  if (dtype == PGG_F32)
    *err = s.general ? backward_of<PGG_F32, 4, true, false, false>(a, s, stream)
                     : backward_of<PGG_F32, 4, false, false, false>(a, s, stream);
  else
    *err = dtype == PGG_F16 ? backward_16<PGG_F16>(a, s, stream) : backward_16<PGG_BF16>(a, s, stream);
  return true;
}

}  // namespace pgg
