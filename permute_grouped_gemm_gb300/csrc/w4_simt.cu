// Products with 4-bit expert weights on the FP32 pipes, for every dtype, size
// and alignment, and the combination of a token's rows:
//
//     w[g, n, k] = scale[g, n, k / group] (code - zero)
//     rows      y[i, n] = sum_k x[token(i), k] w[g(i), n, k]
//     gated     h[i, f] = prob silu(gate) up, gate and up the columns f and F + f
//     combined  out[b, n] = sum over the rows i of token b of sum_k x[i, k] w[g(i), n, k]
//
// Tile: 32 rows of one expert x 64 columns (gated: 32 gates and their 32 ups),
// twice 128 threads with a 4 x 4 block each, which take every other step of 32 k;
// the latter's sums are added to the former's. Bytes of codes are read one by one,
// so that rows of any length will do; a step's are loaded while the one before is
// worked on, and its scale once for sixteen of k. Few tiles leave it waiting for
// memory (450 rows, 7 experts, 1021 x 286, fp32: 45 us; one half, nothing ahead,
// a scale for every k: 103). Sums are fp32, each output is rounded once.

#include <cstdint>

#include "pgg_block.h"
#include "pgg_ptx.cuh"
#include "pgg_vec.cuh"

namespace pgg {
namespace {

constexpr int kHalf = 128;        // threads that take every other step of k
constexpr int kThr = 2 * kHalf;
constexpr int kRows = 32;
constexpr int kCols = 64;
constexpr int kKc = 32;

struct Smem {
  float x[kKc][kRows + 4];
  float w[kKc][kCols + 4];
};

template <int DT>
__device__ __forceinline__ float scale_at(const W4Args& a, int64_t i) {
  return a.scale_f32 ? static_cast<const float*>(a.scales)[i] : vec::load1<DT>(a.scales, i);
}

template <int DT>
__global__ void __launch_bounds__(kThr) w4_simt_kernel(const W4Args a, const uint32_t n_blocks) {
  ptx::griddep_wait();
  __shared__ __align__(16) Smem both[2];
  const int half = threadIdx.x / kHalf, tid = threadIdx.x % kHalf, tx = tid & 15, ty = tid >> 4;
  Smem& sm = both[half];
  const uint32_t st_word = a.hdr->status;
  const bool gated = a.product == PGG_W4_GATED, combined = a.product == PGG_W4_COMBINED;
  if (st_word != 0) {  // validation failed: the result is defined as zeros (combined: by the sum)
    const int64_t n = combined ? 0 : a.M * a.N;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThr;
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * kThr + threadIdx.x; q < n; q += stride) {
      if (a.out_f32)
        static_cast<float*>(a.out)[q] = 0.0f;
      else
        vec::store1<DT>(a.out, q, 0.0f);
    }
    return;
  }
  const int tile_n = gated ? 32 : kCols;
  const bool one_group = a.group % 16 == 0;
  const int64_t C = gated ? 2 * a.N : a.N;
  const uint32_t total = a.hdr->n_row_blocks * n_blocks;
  for (uint32_t t = blockIdx.x; t < total; t += gridDim.x) {
    const int4 e = a.rblist[t / n_blocks];
    const int64_t g = check_index(a.hdr, e.x, a.G, 160);
    const int64_t n0 = static_cast<int64_t>(t % n_blocks) * tile_n;
    // this thread's column while it loads: gates in the first 32, ups in the second
    const int lc = tid >> 1;
    const int64_t n = n0 + (gated ? lc & 31 : lc);
    const int64_t col = g * C + n + (gated && lc >= 32 ? a.N : 0);
    const bool have_col = n < a.N;
    for (int p0 = 0; p0 < e.z; p0 += kRows) {
      const int R = e.z - p0 < kRows ? e.z - p0 : kRows;
      const int lr = tid >> 2;  // row while loading
      const int64_t row = static_cast<int64_t>(e.y) + p0 + lr;
      int64_t xrow = -1;
      if (lr < R) xrow = combined ? row : check_index(a.hdr, a.rowinfo[row].token, a.batch, 161);
      float acc[4][4] = {};
      // a step's values, loaded while the one before is worked on: x, 16 codes and (where a group
      // has whole sixteens of k) their scale and zero
      float nx[8], ns = 0.0f, nz = 8.0f;
      uint8_t nc[8];
      const int kw = 16 * (tid & 1);
      auto fetch = [&](int64_t k0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t k = k0 + (tid & 3) + 4 * j;
          nx[j] = xrow >= 0 && k < a.K ? vec::load1<DT>(a.x, xrow * a.K + k) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t k = k0 + kw + 2 * j;
          nc[j] = have_col && k < a.K ? a.codes[col * a.row_bytes + (k >> 1)] : 0;
        }
        if (one_group && have_col && k0 + kw < a.K) {
          const int64_t q = col * a.groups + static_cast<uint32_t>(k0 + kw) /
                                                 static_cast<uint32_t>(a.group);
          ns = scale_at<DT>(a, q);
          if (a.zeros) nz = static_cast<float>(a.zeros[q]);
        }
      };
      fetch(half * kKc);
      for (int64_t k0 = half * kKc; k0 < a.K; k0 += 2 * kKc) {
        ptx::named_bar_sync(1 + half, kHalf);
#pragma unroll
        for (int j = 0; j < 8; ++j) sm.x[(tid & 3) + 4 * j][lr] = nx[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t k = k0 + kw + 2 * j + h;
            float w = 0.0f;  // (behind the end x is 0, but 0 inf is not)
            if (have_col && k < a.K) {
              const float code = static_cast<float>((nc[j] >> (4 * h)) & 15);
              if (one_group) {
                w = ns * (code - nz);
              } else {
                const int64_t q = col * a.groups +
                                  static_cast<uint32_t>(k) / static_cast<uint32_t>(a.group);
                w = scale_at<DT>(a, q) *
                    (code - static_cast<float>(a.zeros ? a.zeros[q] : 8));
              }
            }
            sm.w[kw + 2 * j + h][lc] = w;
          }
        }
        ptx::named_bar_sync(1 + half, kHalf);
        if (k0 + 2 * kKc < a.K) fetch(k0 + 2 * kKc);
#pragma unroll 8
        for (int kk = 0; kk < kKc; ++kk) {
          const float4 xv = *reinterpret_cast<const float4*>(&sm.x[kk][4 * ty]);
          const float2 w0 = *reinterpret_cast<const float2*>(&sm.w[kk][2 * tx]);
          const float2 w1 = *reinterpret_cast<const float2*>(&sm.w[kk][32 + 2 * tx]);
          const float xs[4] = {xv.x, xv.y, xv.z, xv.w};
          const float ws[4] = {w0.x, w0.y, w1.x, w1.y};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ws[j], acc[i][j]);
        }
      }
      // the second half's sums to the first's
      __syncthreads();
      float* sums = &both[1].w[0][0];
      if (half == 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[i * kHalf + tid] = acc[i / 4][i % 4];
      }
      __syncthreads();
      if (half == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i / 4][i % 4] += sums[i * kHalf + tid];
      }
      __syncthreads();  // (the second half's next step goes where they stood)
      if (half == 1) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= R) continue;
        const int64_t row_i = static_cast<int64_t>(e.y) + p0 + r;
        const int64_t pos = check_index(a.hdr, a.rowinfo[row_i].rank, a.M, 162);
        if (gated) {
          const float p = a.probs ? a.probs[pos] : 1.0f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int64_t f = n0 + 2 * tx + j;
            if (f >= a.N) continue;
            const float gate = acc[i][j], up = acc[i][2 + j];
            vec::store1<DT>(a.out, row_i * a.N + f, p * (gate / (1.0f + expf(-gate)) * up));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t f = n0 + (j < 2 ? 2 * tx + j : 32 + 2 * tx + j - 2);
            if (f >= a.N) continue;
            if (combined)
              static_cast<float*>(a.out)[pos * a.N + f] = acc[i][j];
            else if (a.out_f32)
              static_cast<float*>(a.out)[row_i * a.N + f] = acc[i][j];
            else
              vec::store1<DT>(a.out, row_i * a.N + f, acc[i][j]);
          }
        }
      }
    }
  }
}

// One thread per four (or, ragged, one) of a token's columns.
template <int V>
__global__ void __launch_bounds__(256) w4_combine_kernel(const float* rows, const WsHeader* hdr,
                                                         int64_t batch, int64_t top_k, int64_t N,
                                                         float* out) {
  ptx::griddep_wait();
  const bool failed = hdr->status != 0;
  const int64_t per = N / V, total = batch * per;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; q < total;
       q += stride) {
    const int64_t b = q / per, n = (q - b * per) * V;
    float sum[V] = {};
    if (!failed) {
      const float* p = rows + b * top_k * N + n;
#pragma unroll 8
      for (int64_t j = 0; j < top_k; ++j) {
        float v[V];
        vec::load<PGG_F32, V>(p, j * N, v);
#pragma unroll
        for (int c = 0; c < V; ++c) sum[c] += v[c];
      }
    }
    vec::store<PGG_F32, V>(out, b * N + n, sum);
  }
}

template <int DT>
cudaError_t launch_t(const W4Args& a, int num_sms, cudaStream_t stream) {
  const int tile_n = a.product == PGG_W4_GATED ? 32 : kCols;
  const int64_t n_blocks = (a.N + tile_n - 1) / tile_n;
  int64_t grid = a.max_row_blocks * n_blocks;
  if (grid > num_sms * 8) grid = num_sms * 8;
  return launch_pdl(w4_simt_kernel<DT>, dim3(static_cast<unsigned>(grid)), dim3(kThr), 0, stream,
                    1, a, static_cast<uint32_t>(n_blocks));
}

}  // namespace

cudaError_t launch_w4_simt(int dtype, const W4Args& a, int num_sms, cudaStream_t stream) {
  if (dtype == PGG_F32) return launch_t<PGG_F32>(a, num_sms, stream);
  if (dtype == PGG_F16) return launch_t<PGG_F16>(a, num_sms, stream);
  if (dtype == PGG_BF16) return launch_t<PGG_BF16>(a, num_sms, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_w4_combine(const float* rows, const WsHeader* hdr, int64_t batch, int64_t top_k,
                              int64_t N, float* out, int num_sms, cudaStream_t stream) {
  const bool vec4 = N % 4 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
  const int64_t items = batch * (vec4 ? N / 4 : N);
  int64_t blocks = (items + 255) / 256;
  if (blocks > num_sms * 8) blocks = num_sms * 8;
  return launch_pdl(vec4 ? w4_combine_kernel<4> : w4_combine_kernel<1>,
                    dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, 1, rows, hdr, batch,
                    top_k, N, out);
}

}  // namespace pgg
