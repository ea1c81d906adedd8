// Low-rank rows of a few tokens, each with its own adapter:
//
//     u[t, :] = scale[ad] * x[t, :] a[ad],   ad = adapter[t],   u fp32 [T, R]
//
// One cluster of eight CTAs per token, each over an eighth of K: a[ad] is read
// 16 bytes a thread, R / 8 neighbouring threads to a k, so that a warp reads
// one contiguous piece, and multiplied with x in fp32. The CTAs' sums meet in
// the first one's shared memory and are added in order. Nothing is sorted and
// nothing but the caller's tensors is read, so one launch does it, and the
// projection's launch behind it may start streaming its weight at once
// (launch_dependents): the operator takes as long as that stream. K R
// multiply-adds a token on the FP32 pipes are far below what the same bytes of
// `a` cost to read.
//
// The first CTA also checks every id and writes the status word.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pgg_ops.h"
#include "pgg_ops_cluster.cuh"
#include "pgg_ops_mma.cuh"
#include "pgg_ptx.cuh"

namespace pgg {
namespace {

constexpr int kSplit = 8;
constexpr int kThreads = 256;
constexpr int kMaxR = static_cast<int>(kMaxRank);

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) few_shrink_kernel(const RowsArgs a) {
  cluster_started();
  ptx::griddep_wait();
  // all that came before has completed; the launch behind this one reads only the caller's x and
  // weight until its own wait
  launch_dependents();
  extern __shared__ float s_mem[];  // [threads along k][R], then [kSplit][R]
  __shared__ float s_out[kSplit][kMaxR];
  const int tid = threadIdx.x;
  const uint32_t rank = ptx::cluster_ctarank();
  const int64_t t = blockIdx.x / kSplit;
  if (blockIdx.x == 0) {
    bool bad = false;
    for (int64_t i = tid; i < a.M; i += kThreads) {
      const int64_t id = a.adapter[i];
      bad = bad || id < -1 || id >= a.G;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      a.hdr->status = bad ? kStIndex : 0u;
      a.hdr->timeout_site = 0;
    }
  }
  const int64_t ad = a.adapter[t];
  const bool on = ad >= 0 && ad < a.G;  // the same in all of the cluster
  const int R = static_cast<int>(a.N), oct = R / 8, nk = kThreads / oct;
  const int64_t per = (a.K / 8 + kSplit - 1) / kSplit * 8;
  const int64_t k0 = per * rank, k1 = k0 + per < a.K ? k0 + per : a.K;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  const int ro = tid % oct, kk = tid / oct;
  if (on && kk < nk) {
    const uint4* f = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w) +
                                                    (ad * a.K) * R) + ro;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + t * a.K;
    // eight loads under way at once, also where fewer are left (a chain of single ones cost 2 us:
    // one token 15.5 -> 13.7, 48 tokens 24.0 -> 22.9 for the whole call)
    for (int64_t k = k0 + kk; k < k1; k += 8 * nk) {
      uint4 q[8];
      uint16_t xs[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t ki = k + i * nk;
        const bool in = ki < k1;
        q[i] = in ? __ldg(f + ki * oct) : make_uint4(0, 0, 0, 0);
        xs[i] = in ? __ldg(x + ki) : static_cast<uint16_t>(0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xv = unpack2<DT>(xs[i]).x;
        const float2 p0 = unpack2<DT>(q[i].x), p1 = unpack2<DT>(q[i].y);
        const float2 p2 = unpack2<DT>(q[i].z), p3 = unpack2<DT>(q[i].w);
        acc[0] = fmaf(xv, p0.x, acc[0]);
        acc[1] = fmaf(xv, p0.y, acc[1]);
        acc[2] = fmaf(xv, p1.x, acc[2]);
        acc[3] = fmaf(xv, p1.y, acc[3]);
        acc[4] = fmaf(xv, p2.x, acc[4]);
        acc[5] = fmaf(xv, p2.y, acc[5]);
        acc[6] = fmaf(xv, p3.x, acc[6]);
        acc[7] = fmaf(xv, p3.y, acc[7]);
      }
    }
  }
  if (kk < nk) {
    float4* s = reinterpret_cast<float4*>(s_mem + kk * R + ro * 8);
    s[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    s[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
  __syncthreads();
  // the threads' sums of each rank: `parts` threads a rank, then one
  const int parts = R >= kThreads ? 1 : kThreads / R;
  const int r = tid % R, part = tid / R;
  float v = 0.0f;
  if (part < parts)
    for (int i = part; i < nk; i += parts) v += s_mem[i * R + r];
  __syncthreads();
  if (part < parts) s_mem[part * R + r] = v;
  __syncthreads();
  cluster_all_started();
  if (tid < R) {
    v = 0.0f;
    for (int i = 0; i < parts; ++i) v += s_mem[i * R + tid];
    st_cluster_f32(ptx::mapa(&s_out[rank][tid], 0), v);
  }
  ptx::cluster_sync();
  if (rank == 0 && tid < R && on) {
    v = 0.0f;
#pragma unroll
    for (int c = 0; c < kSplit; ++c) v += s_out[c][tid];
    static_cast<float*>(a.out)[t * R + tid] = v * (a.scale ? a.scale[ad] : 1.0f);
  }
}

}  // namespace

cudaError_t launch_few_shrink(int dtype, const RowsArgs& a, cudaStream_t stream) {
  const int R = static_cast<int>(a.N);
  const int nk = kThreads / (R / 8);
  const size_t smem = static_cast<size_t>(nk > 1 ? nk : 1) * R * 4;  // 8 KB
  return launch_pdl(dtype == PGG_BF16 ? few_shrink_kernel<PGG_BF16> : few_shrink_kernel<PGG_F16>,
                    dim3(static_cast<unsigned>(a.M * kSplit)), dim3(kThreads), smem, stream,
                    kSplit, a);
}

}  // namespace pgg
