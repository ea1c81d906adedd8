// Gradient of the gated product's activation, from d_h and the kept
// pre-activations gate_up = [gate | up]:
//
//     sig = 1 / (1 + exp(-gate)),  act = gate * sig
//     d_up   = p d_h act
//     d_gate = p d_h up sig (1 + gate (1 - sig))
//     d_prob = sum over f of d_h act up          (by original position)
//     h      = p act up                          (the operand of the weight gradient)
//
// with p the row's routing weight (1 without weights). One pass: three 16-byte
// reads and up to three 16-byte writes per eight 16-bit elements, one warp per
// row, d_prob one fixed-order 32-bit sum. 12 bytes move per gate, so HBM is
// what bounds it. d_prob is fp32 whatever the rows' dtype, so the exponential is
// the accurate one for all of them (108000 x 2048 bf16 takes 415 us with it and
// with the fast one, whose error grows with |gate|; 4096 x 2048 22.0 and 21.1);
// the 16-bit dtypes take a reciprocal within one unit for the quotient.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pgg_ops.h"
#include "pgg_ptx.cuh"

namespace pgg {
namespace {

constexpr int kThreads = 256;

template <int DT>
struct Vec {  // 16 bytes of elements
  static constexpr int n = DT == PGG_F32 ? 4 : 8;
  float v[n];
};

template <int DT>
__device__ __forceinline__ void unpack(const uint4& q, Vec<DT>* o) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == PGG_F32) {
      o->v[i] = __uint_as_float(w[i]);
    } else if constexpr (DT == PGG_BF16) {
      o->v[2 * i] = __uint_as_float(w[i] << 16);
      o->v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      o->v[2 * i] = f.x;
      o->v[2 * i + 1] = f.y;
    }
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack(const Vec<DT>& o) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == PGG_F32) {
      w[i] = __float_as_uint(o.v[i]);
    } else if constexpr (DT == PGG_BF16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(o.v[2 * i], o.v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      const __half2 p = __floats2half2_rn(o.v[2 * i], o.v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (DT == PGG_F32) return static_cast<const float*>(p)[i];
  if constexpr (DT == PGG_F16) return __half2float(static_cast<const __half*>(p)[i]);
  if constexpr (DT == PGG_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (DT == PGG_F32) static_cast<float*>(p)[i] = v;
  if constexpr (DT == PGG_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  if constexpr (DT == PGG_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// 1 / x within one unit of the last place, from its smallest to its largest values.
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// One element: d_gate, d_up and h in place of gate, up and d_h; returns its part of d_prob.
template <int DT>
__device__ __forceinline__ float element(float& g, float& u, float& d, float p) {
  const float sig = DT == PGG_F32 ? 1.0f / (1.0f + expf(-g)) : reciprocal(1.0f + expf(-g));
  const float act = g * sig, y = act * u;
  const float part = d * y, pd = p * d;
  const float d_gate = pd * u * (sig * fmaf(g, 1.0f - sig, 1.0f));
  u = pd * act;
  g = d_gate;
  d = p * y;
  return part;
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) gated_grad_kernel(const GatedGradArgs a) {
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  const bool failed = a.hdr->status != 0;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
       q < a.M; q += warps) {
    if (failed) {  // the index is not a permutation: the results are defined as zeros
      for (int64_t f = lane; f < a.F; f += 32) {
        store1<DT>(a.d_gate_up, q * 2 * a.F + f, 0.0f);
        store1<DT>(a.d_gate_up, q * 2 * a.F + a.F + f, 0.0f);
        if (a.h) store1<DT>(a.h, q * a.F + f, 0.0f);
      }
      if (a.d_probs && lane == 0) a.d_probs[q] = 0.0f;
      continue;
    }
    const int64_t v = a.idx[q];
    const int64_t row = a.row_idx_type == 0 ? q : v;
    const int64_t pos = a.row_idx_type == 0 ? v : q;
    const float p = a.probs ? a.probs[pos] : 1.0f;
    float part = 0.0f;
    if constexpr (VEC) {
      constexpr int kV = Vec<DT>::n;
      constexpr int es = 16 / kV;
      const int64_t n = a.F / kV;  // 16-byte units of a row
      const uint4* pg = reinterpret_cast<const uint4*>(static_cast<const char*>(a.gate_up) +
                                                       row * 2 * a.F * es);
      const uint4* pu = pg + n;
      const uint4* pd = reinterpret_cast<const uint4*>(static_cast<const char*>(a.d_h) +
                                                       row * a.F * es);
      uint4* og = reinterpret_cast<uint4*>(static_cast<char*>(a.d_gate_up) + row * 2 * a.F * es);
      uint4* oh = a.h ? reinterpret_cast<uint4*>(static_cast<char*>(a.h) + row * a.F * es) : nullptr;
      for (int64_t i = lane; i < n; i += 32) {
        Vec<DT> g, u, d;
        unpack<DT>(pg[i], &g);
        unpack<DT>(pu[i], &u);
        unpack<DT>(pd[i], &d);
#pragma unroll
        for (int c = 0; c < kV; ++c) part += element<DT>(g.v[c], u.v[c], d.v[c], p);
        og[i] = pack<DT>(g);
        og[n + i] = pack<DT>(u);
        if (oh) oh[i] = pack<DT>(d);
      }
    } else {
      for (int64_t f = lane; f < a.F; f += 32) {
        float g = load1<DT>(a.gate_up, row * 2 * a.F + f);
        float u = load1<DT>(a.gate_up, row * 2 * a.F + a.F + f);
        float d = load1<DT>(a.d_h, row * a.F + f);
        part += element<DT>(g, u, d, p);
        store1<DT>(a.d_gate_up, row * 2 * a.F + f, g);
        store1<DT>(a.d_gate_up, row * 2 * a.F + a.F + f, u);
        if (a.h) store1<DT>(a.h, row * a.F + f, d);
      }
    }
    if (a.d_probs) {
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, s);
      if (lane == 0) a.d_probs[pos] = part;
    }
  }
}

template <int DT>
cudaError_t launch_t(const GatedGradArgs& a, bool vec, int num_sms, cudaStream_t stream) {
  int64_t blocks = (a.M + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = static_cast<int64_t>(num_sms) * 8;
  if (blocks > cap) blocks = cap;
  return launch_pdl(vec ? gated_grad_kernel<DT, true> : gated_grad_kernel<DT, false>,
                    dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, 1, a);
}

}  // namespace

cudaError_t launch_gated_grad(int dtype, const GatedGradArgs& a, bool vec, int num_sms,
                              cudaStream_t stream) {
  if (dtype == PGG_F32) return launch_t<PGG_F32>(a, vec, num_sms, stream);
  if (dtype == PGG_F16) return launch_t<PGG_F16>(a, vec, num_sms, stream);
  if (dtype == PGG_BF16) return launch_t<PGG_BF16>(a, vec, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pgg
