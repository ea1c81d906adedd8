// Device pieces shared by the tensor-core kernels of the gated product and the adapters.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pgg_ops.h"
#include "pgg_ops_cluster.cuh"
#include "pgg_ptx.cuh"

namespace pgg {

__device__ __forceinline__ void raise_status(WsHeader* hdr, uint32_t code, uint32_t site) {
  if (atomicCAS(&hdr->status, 0u, code) == 0u) hdr->timeout_site = site;
}

// The preparation found the caller's routing or adapter ids not valid.
__device__ __forceinline__ bool routing_failed(const WsHeader* hdr) {
  const uint32_t st = hdr->status;
  return st == kStIndex || st == kStGroupSum || st == kStNotPerm;
}

// Zeros to every element of the 16-bit outputs (the whole grid).
__device__ __forceinline__ void zero_rows16(const RowsArgs& a) {
  const int64_t n = a.M * a.N;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; q < n;
       q += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    static_cast<uint16_t*>(a.out)[q] = 0;
    if (a.gate_up) {
      static_cast<uint16_t*>(a.gate_up)[2 * q] = 0;
      static_cast<uint16_t*>(a.gate_up)[2 * q + 1] = 0;
    }
  }
}

// First token of `rows` compact rows of one adapter from row0 if they are neighbouring tokens, else
// -1. (An adapter's rows are in token order, so the ends tell.)
__device__ __forceinline__ int32_t box_of_rows(const RowInfo* order, int64_t row0, int rows) {
  if (rows <= 0) return -1;
  const int32_t t0 = order[row0].token;
  return order[row0 + rows - 1].token - t0 == rows - 1 ? t0 : -1;
}

// Two 16-bit values of a 32-bit word <-> fp32 (round to nearest even).
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == PGG_BF16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  } else {
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
}

template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (DT == PGG_BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// v as the sum of two 16-bit values (see LowRankForm): hi is v cut off, lo the rounded rest. Both have
// v's sign and (but for the smallest numbers) neither is 0, so that times an infinity they are the
// same infinity, and their sum is what v times it is; where nothing is left, hi gives one unit to lo.
template <int DT>
__device__ __forceinline__ void split16(float v, uint16_t* hi, uint16_t* lo) {
  const bool finite = fabsf(v) < INFINITY;
  uint32_t h;
  float left;
  if constexpr (DT == PGG_BF16) {
    const uint32_t b = __float_as_uint(v);
    h = b >> 16;
    if (finite && (b & 0xFFFFu) == 0 && (h & 0x7FFFu) != 0) --h;
    left = v - __uint_as_float(h << 16);
    *lo = __bfloat16_as_ushort(__float2bfloat16_rn(left));
  } else {
    h = __half_as_ushort(__float2half_rz(v));
    left = v - __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
    if (finite && fabsf(left) <= 0x1p-25f && (h & 0x7FFFu) != 0) {  // (would round to 0)
      --h;
      left = v - __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
    }
    *lo = __half_as_ushort(__float2half_rn(left));
  }
  if (!finite) *lo = static_cast<uint16_t>(h);
  *hi = static_cast<uint16_t>(h);
}

// ptx::mapa of a shared-memory address.
__device__ __forceinline__ uint32_t mapa_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Programmatic dependent launch: the launch behind this one may start.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A launch and the one behind it that does not read what it writes may run side by side, so that the
// second fills the multiprocessors that the first leaves idle. The first (early) waits for all
// before it and then lets the second start; the second (late) starts at once: what it reads was
// complete when the first let it. It waits for the first before it ends, so that the launch behind
// both finds both complete.
__device__ __forceinline__ void launch_order(bool early, bool late) {
  if (!late) ptx::griddep_wait();
  if (early) launch_dependents();
}

__device__ __forceinline__ void launch_end(bool late) {
  if (late && blockIdx.x == 0) ptx::griddep_wait();
}

// p * silu(g) * u for a 16-bit output: the fast exponential, within 2 + |1.2 g| units of 2^-23 (2^-19
// of the result at g = -8, 2^-16 at -85; where g is positive it hardly counts), and a quotient
// within two (0 below g = -87.3). That stays well below the one rounding of the result, 2^-9 in
// bf16 and 2^-12 in fp16.
__device__ __forceinline__ float gate(float g, float u, float p) {
  return p * (g * __fdividef(1.0f, 1.0f + __expf(-g)) * u);
}

// Pair MMA (see ptx::mma_f16_pair) that leaves the accumulator lanes of the set mask bits as they
// are: bit b of word i is lane 32 i + b of the pair's 256.
__device__ __forceinline__ void mma_f16_pair_lanes(uint32_t d_tmem, uint64_t a_desc,
                                                   uint64_t b_desc, uint32_t idesc,
                                                   const uint32_t (&m)[8], uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3,"
      " {%5, %6, %7, %8, %9, %10, %11, %12}, p;\n"
      "}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(m[0]), "r"(m[1]), "r"(m[2]),
      "r"(m[3]), "r"(m[4]), "r"(m[5]), "r"(m[6]), "r"(m[7])
      : "memory");
}

}  // namespace pgg
