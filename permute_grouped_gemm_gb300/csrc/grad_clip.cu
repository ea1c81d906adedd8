// The global norm of a list of gradients, and the gradients clipped to it:
//
//     norm = |scale| sqrt(sum over all tensors of g^2)
//     out  = g c,  c = scale min(1, max_norm / (norm + eps))
//
// Two passes over the gradients (the second is needed because the first's
// result scales it), each bound by memory. A launch takes a table of up to 512
// tensors as its parameters, cut into chunks of 16384 elements; the blocks walk
// the chunks, the table is searched by bisection once a chunk.
//
// Squares are summed in fp32 over the 32 elements that a thread holds, and
// these sums in fp64 in a fixed order: bitwise repeatable. A sum of 32 that
// over- or underflows fp32 is taken again with the elements scaled by a power
// of two, so the norm is right wherever it is an fp32 number.

#include <cstdint>

#include "pgg_block.h"
#include "pgg_ptx.cuh"
#include "pgg_vec.cuh"

namespace pgg {
namespace {

constexpr int kThr = 512;
constexpr int kHold = 32;                   // elements of a thread and chunk
constexpr int kChunk = kThr * kHold;

__device__ __forceinline__ int tensor_of(const ClipTable& t, uint32_t chunk) {
  int lo = 0, hi = t.tensors - 1;  // the last tensor whose first chunk is not behind `chunk`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Sum of the squares of N values.
template <int N>
__device__ __forceinline__ double squares(const float (&v)[N]) {
  float s[4] = {};
#pragma unroll
  for (int i = 0; i < N; ++i) s[i & 3] = fmaf(v[i], v[i], s[i & 3]);
  const float sum = (s[0] + s[1]) + (s[2] + s[3]);
  // (squares below 2^-126 lose bits: 32 of them are nothing beside a sum of 2^-80)
  if (sum > 8.2718061e-25f && sum < 3.0e38f) return sum;
  const float by = sum < 1.0f ? 0x1p96f : 0x1p-70f;  // (NaN: either)
  const double back = sum < 1.0f ? 0x1p-192 : 0x1p140;
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float u = v[i] * by;
    s[i & 3] = fmaf(u, u, s[i & 3]);
  }
  return static_cast<double>((s[0] + s[1]) + (s[2] + s[3])) * back;
}

template <int DT>
__device__ __forceinline__ double chunk_squares(const void* in, int64_t at, int64_t n) {
  constexpr int V = 16 / vec::elem_bytes(DT);
  const bool vectors = reinterpret_cast<uintptr_t>(in) % 16 == 0 && at + kChunk <= n;
  float v[kHold];
  if (vectors) {
#pragma unroll
    for (int j = 0; j < kHold / V; ++j) {
      float u[V];
      vec::load<DT, V>(in, at + (static_cast<int64_t>(j) * kThr + threadIdx.x) * V, u);
#pragma unroll
      for (int c = 0; c < V; ++c) v[j * V + c] = u[c];
    }
  } else {
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      const int64_t i = at + static_cast<int64_t>(j) * kThr + threadIdx.x;
      v[j] = i < n ? vec::load1<DT>(in, i) : 0.0f;
    }
  }
  return squares(v);
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s_part[kThr / 32];
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  double sum = 0.0;
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) sum += s_part[i];
  return sum;
}

__global__ void __launch_bounds__(kThr) clip_squares_kernel(const __grid_constant__ ClipTable t,
                                                            WsHeader* hdr, double* partial) {
  ptx::griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) hdr->status = 0;
  double sum = 0.0;
  const uint32_t chunks = t.first[t.tensors];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = static_cast<int64_t>(c - t.first[i]) * kChunk;
    if (t.dtype[i] == PGG_F32)
      sum += chunk_squares<PGG_F32>(t.in[i], at, t.n[i]);
    else if (t.dtype[i] == PGG_F16)
      sum += chunk_squares<PGG_F16>(t.in[i], at, t.n[i]);
    else
      sum += chunk_squares<PGG_BF16>(t.in[i], at, t.n[i]);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThr) clip_norm_kernel(const double* partial, int64_t count,
                                                         float scale, float* norm) {
  ptx::griddep_wait();
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += kThr) sum += partial[i];
  sum = block_sum(sum);
  if (threadIdx.x == 0)
    *norm = static_cast<float>(sqrt(sum) * fabs(static_cast<double>(scale)));
}

template <int DT>
__device__ __forceinline__ void chunk_apply(const void* in, void* out, int64_t at, int64_t n,
                                            float by) {
  constexpr int V = 16 / vec::elem_bytes(DT);
  const bool vectors = reinterpret_cast<uintptr_t>(in) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(out) % 16 == 0 && at + kChunk <= n;
  if (vectors) {
    float v[kHold / V][V];
#pragma unroll
    for (int j = 0; j < kHold / V; ++j)
      vec::load<DT, V>(in, at + (static_cast<int64_t>(j) * kThr + threadIdx.x) * V, v[j]);
#pragma unroll
    for (int j = 0; j < kHold / V; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) v[j][c] *= by;
      vec::store<DT, V>(out, at + (static_cast<int64_t>(j) * kThr + threadIdx.x) * V, v[j]);
    }
  } else {
#pragma unroll 8
    for (int j = 0; j < kHold; ++j) {
      const int64_t i = at + static_cast<int64_t>(j) * kThr + threadIdx.x;
      if (i < n) vec::store1<DT>(out, i, vec::load1<DT>(in, i) * by);
    }
  }
}

__global__ void __launch_bounds__(kThr) clip_apply_kernel(const __grid_constant__ ClipTable t,
                                                          const float* norm, float max_norm,
                                                          float eps, float scale) {
  ptx::griddep_wait();
  const float n = *norm;
  float by = scale;
  if (n < __int_as_float(0x7F800000)) {  // (not NaN, not infinite)
    const float ratio = max_norm / (n + eps);
    if (ratio < 1.0f) by = scale * ratio;
  }
  const uint32_t chunks = t.first[t.tensors];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    if (by == 1.0f && t.in[i] == t.out[i]) continue;
    const int64_t at = static_cast<int64_t>(c - t.first[i]) * kChunk;
    if (t.dtype[i] == PGG_F32)
      chunk_apply<PGG_F32>(t.in[i], t.out[i], at, t.n[i], by);
    else if (t.dtype[i] == PGG_F16)
      chunk_apply<PGG_F16>(t.in[i], t.out[i], at, t.n[i], by);
    else
      chunk_apply<PGG_BF16>(t.in[i], t.out[i], at, t.n[i], by);
  }
}

}  // namespace

int64_t clip_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }

cudaError_t launch_clip_squares(const ClipTable& t, WsHeader* hdr, double* partial, int blocks,
                                cudaStream_t stream) {
  return launch_pdl(clip_squares_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThr), 0,
                    stream, 1, t, hdr, partial);
}

cudaError_t launch_clip_norm(const double* partial, int64_t count, float scale, float* norm,
                             cudaStream_t stream) {
  return launch_pdl(clip_norm_kernel, dim3(1), dim3(kThr), 0, stream, 1, partial, count, scale,
                    norm);
}

cudaError_t launch_clip_apply(const ClipTable& t, const float* norm, float max_norm, float eps,
                              float scale, int blocks, cudaStream_t stream) {
  return launch_pdl(clip_apply_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThr), 0, stream,
                    1, t, norm, max_norm, eps, scale);
}

}  // namespace pgg
