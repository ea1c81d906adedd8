// Products over ragged rows on the FP32 pipes: the gated product, the
// adapters' low-rank rows and the projection with adapters, for every dtype,
// size and alignment. fp32 inputs, odd widths and unaligned pointers run here;
// 16-bit inputs whose rows the tensor-memory-access unit can stream run on the
// tensor cores instead.
//
//     gated    gate_up[i, :] = x[token(i)] W[g(i)];  h = prob * silu(gate) * up
//     shrink   u[i, :] = scale[g(i)] * x[token(i)] a[g(i)]
//     adapt    y[token(i), :] = x[token(i)] W + u[i] b[g(i)]^T   (W as [K, N] or [N, K])
//
// Tile: 64 rows of one group x 128 columns (gated: 64 gates and the 64 ups
// that belong to them, so that a thread holds both), 128 threads with an 8 x 8
// block each, 32 of the reduction index a step through two shared-memory
// buffers. All sums are 32-bit fused multiply-adds in increasing k; 16-bit
// outputs are rounded once. Rows of one tile belong to one group, so what
// another adapter's weights hold never meets them.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pgg_ops.h"
#include "pgg_ops_mma.cuh"
#include "pgg_ptx.cuh"

namespace pgg {
namespace {

constexpr int kThr = 128;
constexpr int kRows = 64;
constexpr int kCols = 128;
constexpr int kKc = 32;
constexpr int kAS = kRows + 4;   // strides of the shared tiles [k][row] and [k][col]
constexpr int kBS = kCols + 4;

struct Smem {
  float a[2][kKc * kAS];
  float b[2][kKc * kBS];
};

template <int DT>
__device__ __forceinline__ float ld(const void* p, int64_t i) {
  if constexpr (DT == PGG_F32) return __ldg(static_cast<const float*>(p) + i);
  if constexpr (DT == PGG_F16) return __half2float(__ldg(static_cast<const __half*>(p) + i));
  if constexpr (DT == PGG_BF16)
    return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + i));
}

template <int DT>
__device__ __forceinline__ void st(void* p, int64_t i, float v) {
  if constexpr (DT == PGG_F32) static_cast<float*>(p)[i] = v;
  if constexpr (DT == PGG_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  if constexpr (DT == PGG_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Rank n of a low-rank row (a.N ranks).
template <int DT>
__device__ __forceinline__ void store_low(const RowsArgs& a, int64_t row, int64_t n, float v) {
  if (a.low_form == kLowFloat) {
    static_cast<float*>(a.out)[row * a.N + n] = v;
  } else if (a.low_form == kLowRounded) {
    st<DT>(a.out, row * a.N + n, v);
  } else if constexpr (DT != PGG_F32) {
    uint16_t* p = static_cast<uint16_t*>(a.out) + row * low_width(a.N) + n / 32 * 64 + n % 32;
    split16<DT>(v, p, p + 32);
  }
}

// A [row][k] and B by element: column c of the tile at bcol[c-part] + k * kstride.
struct Operand {
  const void* a;
  const void* b;
  int64_t lda, K;
  int64_t b0;       // B offset of (k 0, tile column 0)
  int64_t bk, bn;   // strides of B along k and along the columns; one of them is 1
  int64_t ncols;    // valid columns of the tile (of each half when gated)
  int64_t half;     // gated: offset of the second half's columns; else 0
};

template <int DA, int DT, bool HALVES, bool KMAJOR>
__device__ __forceinline__ void load_step(const Operand& o, const int32_t (&arow)[4], int64_t k0,
                                          int warp, int lane, float (&ra)[16], float (&rb)[32]) {
  const int l_k = lane & 7, l_r = lane >> 3;
#pragma unroll
  for (int it = 0; it < 4; ++it)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t k = k0 + 8 * q + l_k;
      ra[4 * it + q] = arow[it] >= 0 && k < o.K ? ld<DA>(o.a, arow[it] * o.lda + k) : 0.0f;
    }
  if constexpr (KMAJOR) {  // 8 k x 4 columns an instruction
#pragma unroll
    for (int it = 0; it < 8; ++it)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t k = k0 + 8 * q + l_k;
        const int c = it * 16 + warp * 4 + l_r;
        rb[4 * it + q] = c < o.ncols && k < o.K ? ld<DT>(o.b, o.b0 + c * o.bn + k) : 0.0f;
      }
  } else {  // one k, 32 columns an instruction
#pragma unroll
    for (int it = 0; it < 8; ++it)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int64_t k = k0 + 4 * it + warp;
        const int c = 32 * h + lane;
        const int in_half = HALVES ? c & 63 : c;
        const int64_t off = HALVES && c >= 64 ? o.half + in_half : in_half;
        rb[4 * it + h] =
            in_half < o.ncols && k < o.K ? ld<DT>(o.b, o.b0 + k * o.bk + off) : 0.0f;
      }
  }
}

template <bool KMAJOR>
__device__ __forceinline__ void store_step(float* sa, float* sb, int warp, int lane,
                                           const float (&ra)[16], const float (&rb)[32]) {
  const int l_k = lane & 7, l_r = lane >> 3;
#pragma unroll
  for (int it = 0; it < 4; ++it)
#pragma unroll
    for (int q = 0; q < 4; ++q) sa[(8 * q + l_k) * kAS + it * 16 + warp * 4 + l_r] = ra[4 * it + q];
  if constexpr (KMAJOR) {
#pragma unroll
    for (int it = 0; it < 8; ++it)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sb[(8 * q + l_k) * kBS + it * 16 + warp * 4 + l_r] = rb[4 * it + q];
  } else {
#pragma unroll
    for (int it = 0; it < 8; ++it)
#pragma unroll
      for (int h = 0; h < 4; ++h) sb[(4 * it + warp) * kBS + 32 * h + lane] = rb[4 * it + h];
  }
}

// acc += A B over the operand's whole reduction (A of dtype DA, B of DT).
template <int DA, int DT, bool HALVES, bool KMAJOR>
__device__ __forceinline__ void product(Smem& sm, const Operand& o, const int32_t (&arow)[4],
                                        float (&acc)[8][8]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tx = tid & 15, ty = tid >> 4;
  float ra[16], rb[32];
  load_step<DA, DT, HALVES, KMAJOR>(o, arow, 0, warp, lane, ra, rb);
  __syncthreads();  // earlier reads of buffer 0 are done
  store_step<KMAJOR>(sm.a[0], sm.b[0], warp, lane, ra, rb);
  __syncthreads();
  int buf = 0;
  for (int64_t k0 = 0; k0 < o.K; k0 += kKc) {
    const bool more = k0 + kKc < o.K;
    if (more) load_step<DA, DT, HALVES, KMAJOR>(o, arow, k0 + kKc, warp, lane, ra, rb);
    const float* pa = sm.a[buf];
    const float* pb = sm.b[buf];
#pragma unroll 4
    for (int kk = 0; kk < kKc; ++kk) {
      const float4 a0 = *reinterpret_cast<const float4*>(&pa[kk * kAS + 8 * ty]);
      const float4 a1 = *reinterpret_cast<const float4*>(&pa[kk * kAS + 8 * ty + 4]);
      const float4 b0 = *reinterpret_cast<const float4*>(&pb[kk * kBS + 4 * tx]);
      const float4 b1 = *reinterpret_cast<const float4*>(&pb[kk * kBS + 64 + 4 * tx]);
      const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
      const float bv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    if (more) store_step<KMAJOR>(sm.a[buf ^ 1], sm.b[buf ^ 1], warp, lane, ra, rb);
    __syncthreads();
    buf ^= 1;
  }
}

template <int DT, int MODE>
__device__ void zero_outputs(const RowsArgs& a) {
  const int64_t n = MODE == kShrink ? 0 : a.M * a.N;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; q < n;
       q += stride) {
    st<DT>(a.out, q, 0.0f);
    if (MODE == kGated && a.gate_up) {
      st<DT>(a.gate_up, 2 * q, 0.0f);
      st<DT>(a.gate_up, 2 * q + 1, 0.0f);
    }
  }
}

template <int DT, int MODE>
__global__ void __launch_bounds__(kThr, 3) rows_simt_kernel(const RowsArgs a) {
  ptx::griddep_wait();
  extern __shared__ __align__(16) uint8_t rows_simt_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(rows_simt_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tx = tid & 15, ty = tid >> 4;
  // validation failed: the result is defined as zeros
  const uint32_t st_word = a.hdr->status;
  if (st_word == kStIndex || st_word == kStGroupSum || st_word == kStNotPerm) {
    zero_outputs<DT, MODE>(a);
    return;
  }
  constexpr bool kHalves = MODE == kGated;
  constexpr int kTileN = kHalves ? 64 : kCols;
  const uint32_t nb = static_cast<uint32_t>(a.n_blocks);
  const uint32_t total = a.hdr->n_row_blocks * nb;
  for (uint32_t t = blockIdx.x; t < total; t += gridDim.x) {
    const int4 e = a.rblist[t / nb];
    const int64_t g = e.x, n0 = static_cast<int64_t>(t % nb) * kTileN;
    const bool none = MODE != kGated && g >= a.G;  // tokens without an adapter
    if (MODE == kShrink && none) continue;
    for (int p0 = 0; p0 < e.z; p0 += kRows) {
      const int R = e.z - p0 < kRows ? e.z - p0 : kRows;
      int32_t tok[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int r = it * 16 + warp * 4 + (lane >> 3);
        tok[it] = r < R ? a.rowinfo[static_cast<int64_t>(e.y) + p0 + r].token : -1;
      }
      float acc[8][8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
      Operand o;
      o.a = a.x;
      o.b = a.w;
      o.lda = a.K;
      o.K = a.K;
      o.half = 0;
      o.ncols = a.N - n0 < kTileN ? a.N - n0 : kTileN;
      if (MODE == kGated) {
        o.bk = 2 * a.N;
        o.bn = 1;
        o.half = a.N;
        o.b0 = g * a.K * 2 * a.N + n0;
      } else if (MODE == kAdaptT) {
        o.bk = 1;
        o.bn = a.K;
        o.b0 = n0 * a.K;
      } else {
        o.bk = a.N;
        o.bn = 1;
        o.b0 = (MODE == kShrink ? g * a.K * a.N : 0) + n0;
      }
      product<DT, DT, kHalves, MODE == kAdaptT>(sm, o, tok, acc);
      if ((MODE == kAdapt || MODE == kAdaptT) && !none) {
        // the low-rank part: rows of u are in order, b [A, N, R] has the rank innermost
        int32_t urow[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int r = it * 16 + warp * 4 + (lane >> 3);
          urow[it] = r < R ? e.w + p0 + r : -1;
        }
        o.a = a.u;
        o.b = a.b;
        o.lda = a.R;
        o.K = a.R;
        o.bk = 1;
        o.bn = a.R;
        o.b0 = (g * a.N + n0) * a.R;
        if (a.low_form == kLowFloat)
          product<PGG_F32, DT, false, true>(sm, o, urow, acc);
        else
          product<DT, DT, false, true>(sm, o, urow, acc);
      }
      const float sc = MODE == kShrink && a.scale ? a.scale[g] : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 8 * ty + i;
        if (r >= R) continue;
        const int64_t row = static_cast<int64_t>(e.y) + p0 + r;
        if (MODE == kGated) {
          const float p = a.probs ? a.probs[a.rowinfo[row].rank] : 1.0f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int64_t f = n0 + 4 * tx + c;
            if (f >= a.N) continue;
            const float gate = acc[i][c], up = acc[i][4 + c];
            st<DT>(a.out, row * a.N + f, p * (gate / (1.0f + expf(-gate)) * up));
            if (a.gate_up) {
              st<DT>(a.gate_up, row * 2 * a.N + f, gate);
              st<DT>(a.gate_up, row * 2 * a.N + a.N + f, up);
            }
          }
        } else {
          const int64_t orow = MODE == kShrink ? static_cast<int64_t>(e.w) + p0 + r
                                               : a.rowinfo[row].token;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int64_t n = n0 + (j < 4 ? 4 * tx + j : 64 + 4 * tx + j - 4);
            if (n >= a.N) continue;
            if (MODE == kShrink)
              store_low<DT>(a, orow, n, acc[i][j] * sc);
            else
              st<DT>(a.out, orow * a.N + n, acc[i][j]);
          }
        }
      }
    }
  }
}

template <int DT>
cudaError_t launch_t(RowsMode mode, const RowsArgs& a, int num_sms, cudaStream_t stream) {
  using K = void (*)(const RowsArgs);
  static const K kern[4] = {rows_simt_kernel<DT, kGated>, rows_simt_kernel<DT, kShrink>,
                            rows_simt_kernel<DT, kAdapt>, rows_simt_kernel<DT, kAdaptT>};
  constexpr int smem = static_cast<int>(sizeof(Smem));
  cudaError_t err = cudaFuncSetAttribute(kern[mode], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem);
  if (err != cudaSuccess) return err;
  int64_t grid = static_cast<int64_t>(num_sms) * 3;
  const int64_t tiles = a.max_row_blocks * a.n_blocks;
  if (tiles < grid) grid = tiles;
  return launch_pdl(kern[mode], dim3(static_cast<unsigned>(grid)), dim3(kThr),
                    static_cast<size_t>(smem), stream, 1, a);
}

}  // namespace

cudaError_t launch_rows_simt(int dtype, RowsMode mode, RowsArgs a, int num_sms,
                             cudaStream_t stream) {
  const int64_t tile_n = mode == kGated ? 64 : kCols;
  a.n_blocks = static_cast<int32_t>((a.N + tile_n - 1) / tile_n);
  if (dtype == PGG_F32) return launch_t<PGG_F32>(mode, a, num_sms, stream);
  if (dtype == PGG_F16) return launch_t<PGG_F16>(mode, a, num_sms, stream);
  if (dtype == PGG_BF16) return launch_t<PGG_BF16>(mode, a, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pgg
