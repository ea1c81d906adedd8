// The global norm of a list of gradients, and the gradients clipped to it:
//
//     norm = |scale| sqrt(sum over all tensors of g^2)
//     out  = g c,  c = scale min(1, max_norm / (norm + eps))
//
// Two passes over the gradients (the second is needed because the first's
// result scales it), each bound by memory. A launch takes a table of up to 512
// tensors as its parameters, cut into chunks of 64 KB; the blocks walk the
// chunks, the table is searched by bisection once a chunk. A thread loads its
// eight 16-byte words of a chunk before it uses one, with the hint for data that is
// not read again: the norm alone is faster by it (400 M elements: 197 us, 203 without),
// and of what the first pass read last the second-level cache keeps little, so that
// the second pass, which walks the chunks backwards to find it, gains 2 of 520 us (537 M
// bf16 elements; without the hint 517).
//
// Squares are summed in fp32 over the elements that a thread holds, and these
// sums in fp64 in a fixed order: bitwise repeatable. A sum that over- or
// underflows fp32 is taken again with the elements scaled by a power of two, so
// the norm is right wherever it is an fp32 number.

#include <cstdint>

#include "pgg_block.h"
#include "pgg_ptx.cuh"
#include "pgg_vec.cuh"

namespace pgg {
namespace {

constexpr int kThr = 512;
constexpr int kWords = 8;                        // of 16 bytes, a thread and chunk
constexpr int64_t kChunkBytes = kThr * kWords * 16;

__host__ __device__ constexpr int64_t chunk_of(int dtype) {  // elements
  return kChunkBytes / vec::elem_bytes(dtype);
}

__device__ __forceinline__ int tensor_of(const ClipTable& t, uint32_t chunk) {
  int lo = 0, hi = t.tensors - 1;  // the last tensor whose first chunk is not behind `chunk`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// What a thread holds of a chunk: words that are whole, and (an unaligned tensor, or the one that
// the end cuts) single elements.
template <int DT>
struct Piece {
  static constexpr int V = 16 / vec::elem_bytes(DT);
  uint4 w[kWords];
  int64_t i0;    // first element of word 0; words are kThr * V apart
  int64_t n;     // of the tensor
  bool aligned;

  __device__ __forceinline__ int64_t at(int j) const {
    return i0 + static_cast<int64_t>(j) * kThr * V;
  }
  __device__ __forceinline__ bool whole(int j) const { return aligned && at(j) + V <= n; }
  __device__ __forceinline__ void load(const void* in, int64_t first, int64_t size, bool words) {
    i0 = first + static_cast<int64_t>(threadIdx.x) * V;
    n = size;
    aligned = words;
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      w[j] = make_uint4(0, 0, 0, 0);
      if (whole(j))
        w[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(in) +
                                                     at(j) * vec::elem_bytes(DT)));
    }
  }
  __device__ __forceinline__ void values(int j, float (&v)[V]) const {
    vec::load<DT, V>(&w[j], 0, v);
  }
};

template <int DT>
__device__ __forceinline__ float sum_squares(const Piece<DT>& p, const void* in, float by) {
  constexpr int V = Piece<DT>::V;
  float s[4] = {};
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    float v[V];
    p.values(j, v);
#pragma unroll
    for (int c = 0; c < V; ++c) s[c & 3] = fmaf(v[c] * by, v[c] * by, s[c & 3]);
  }
  if (!p.whole(kWords - 1)) {
#pragma unroll 1
    for (int j = 0; j < kWords; ++j)
      if (!p.whole(j))
#pragma unroll
        for (int c = 0; c < V; ++c)
          if (p.at(j) + c < p.n) {
            const float v = vec::load1<DT>(in, p.at(j) + c) * by;
            s[c & 3] = fmaf(v, v, s[c & 3]);  // (the order of whole words: an alignment's bits)
          }
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

template <int DT>
__device__ __forceinline__ double chunk_squares(const void* in, int64_t at, int64_t n) {
  Piece<DT> p;
  p.load(in, at, n, reinterpret_cast<uintptr_t>(in) % 16 == 0);
  const float sum = sum_squares<DT>(p, in, 1.0f);
  // (squares below 2^-126 lose bits: so few of them are nothing beside a sum of 2^-80)
  if (sum > 8.2718061e-25f && sum < 3.0e38f) return sum;
  if (sum < 1.0f)
    return static_cast<double>(sum_squares<DT>(p, in, 0x1p96f)) * 0x1p-192;
  return static_cast<double>(sum_squares<DT>(p, in, 0x1p-70f)) * 0x1p140;  // (NaN, too)
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
    const int64_t at = static_cast<int64_t>(c - t.first[i]) * chunk_of(t.dtype[i]);
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

// The norm from the partial sums (the whole block, the same bits in every thread).
__device__ __forceinline__ float norm_of(const double* partial, int64_t count, float scale) {
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += kThr) sum += partial[i];
  return static_cast<float>(sqrt(block_sum(sum)) * fabs(static_cast<double>(scale)));
}

__global__ void __launch_bounds__(kThr) clip_norm_kernel(const double* partial, int64_t count,
                                                         float scale, float* norm) {
  ptx::griddep_wait();
  const float n = norm_of(partial, count, scale);
  if (threadIdx.x == 0) *norm = n;
}

template <int DT>
__device__ __forceinline__ void chunk_apply(const void* in, void* out, int64_t at, int64_t n,
                                            float by) {
  constexpr int V = Piece<DT>::V;
  Piece<DT> p;
  p.load(in, at, n,
         (reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) % 16 == 0);
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    if (!p.whole(j)) continue;
    float v[V];
    p.values(j, v);
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] *= by;
    uint4 w;
    vec::store<DT, V>(&w, 0, v);
    __stcs(reinterpret_cast<uint4*>(static_cast<char*>(out) + p.at(j) * vec::elem_bytes(DT)), w);
  }
  if (p.whole(kWords - 1)) return;
#pragma unroll 1
  for (int j = 0; j < kWords; ++j)
    if (!p.whole(j))
#pragma unroll
      for (int c = 0; c < V; ++c)
        if (p.at(j) + c < n)
          vec::store1<DT>(out, p.at(j) + c, vec::load1<DT>(in, p.at(j) + c) * by);
}

// Every block takes the norm from the partial sums itself, in their order: one launch less.
__global__ void __launch_bounds__(kThr) clip_apply_kernel(const __grid_constant__ ClipTable t,
                                                          const double* partial, int64_t count,
                                                          float max_norm, float eps, float scale,
                                                          float* norm) {
  ptx::griddep_wait();
  const float n = norm_of(partial, count, scale);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  float by = scale;
  if (n < __int_as_float(0x7F800000)) {  // (not NaN, not infinite)
    const float ratio = max_norm / (n + eps);
    if (ratio < 1.0f) by = scale * ratio;
  }
  const uint32_t chunks = t.first[t.tensors];
  for (uint32_t q = blockIdx.x; q < chunks; q += gridDim.x) {
    const uint32_t c = chunks - 1 - q;
    const int i = tensor_of(t, c);
    if (by == 1.0f && t.in[i] == t.out[i]) continue;
    const int64_t at = static_cast<int64_t>(c - t.first[i]) * chunk_of(t.dtype[i]);
    if (t.dtype[i] == PGG_F32)
      chunk_apply<PGG_F32>(t.in[i], t.out[i], at, t.n[i], by);
    else if (t.dtype[i] == PGG_F16)
      chunk_apply<PGG_F16>(t.in[i], t.out[i], at, t.n[i], by);
    else
      chunk_apply<PGG_BF16>(t.in[i], t.out[i], at, t.n[i], by);
  }
}

}  // namespace

int64_t clip_chunks(int64_t n, int dtype) {
  return (n + chunk_of(dtype) - 1) / chunk_of(dtype);
}

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

cudaError_t launch_clip_apply(const ClipTable& t, const double* partial, int64_t count,
                              float max_norm, float eps, float scale, float* norm, int blocks,
                              cudaStream_t stream) {
  return launch_pdl(clip_apply_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThr), 0, stream,
                    1, t, partial, count, max_norm, eps, scale, norm);
}

}  // namespace pgg
