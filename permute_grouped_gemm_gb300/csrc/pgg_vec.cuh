// Elements of the three dtypes as fp32: one at a time, and in vectors of
// 16-byte loads and stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pgg.h"

namespace pgg {
namespace vec {

__host__ __device__ constexpr int elem_bytes(int dtype) { return dtype == PGG_F32 ? 4 : 2; }

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

// The two 16-bit elements of a word (the lower half first).
template <int DT>
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
  if constexpr (DT == PGG_BF16) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = f.x;
    b = f.y;
  }
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == PGG_BF16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  } else {
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
}

// V (1, 2, 4 or 8) consecutive elements from element i on, aligned to their size or to 16 bytes.
template <int DT, int V>
__device__ __forceinline__ void load(const void* p, int64_t i, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = load1<DT>(p, i);
  } else if constexpr (DT == PGG_F32 && V == 2) {
    const float2 f = *reinterpret_cast<const float2*>(static_cast<const float*>(p) + i);
    v[0] = f.x;
    v[1] = f.y;
  } else if constexpr (V == 2) {
    unpack2<DT>(*reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + i), v[0], v[1]);
  } else if constexpr (DT == PGG_F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const float4 f = q[j];
      v[4 * j] = f.x;
      v[4 * j + 1] = f.y;
      v[4 * j + 2] = f.z;
      v[4 * j + 3] = f.w;
    }
  } else if constexpr (V == 4) {
    const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    unpack2<DT>(q.x, v[0], v[1]);
    unpack2<DT>(q.y, v[2], v[3]);
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    unpack2<DT>(q.x, v[0], v[1]);
    unpack2<DT>(q.y, v[2], v[3]);
    unpack2<DT>(q.z, v[4], v[5]);
    unpack2<DT>(q.w, v[6], v[7]);
  }
}

template <int DT, int V>
__device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[V]) {
  if constexpr (V == 1) {
    store1<DT>(p, i, v[0]);
  } else if constexpr (DT == PGG_F32 && V == 2) {
    *reinterpret_cast<float2*>(static_cast<float*>(p) + i) = make_float2(v[0], v[1]);
  } else if constexpr (V == 2) {
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p) + i) = pack2<DT>(v[0], v[1]);
  } else if constexpr (DT == PGG_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
#pragma unroll
    for (int j = 0; j < V / 4; ++j)
      q[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]));
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                   pack2<DT>(v[6], v[7]));
  }
}

// The same where the dtype is DT or fp32, known at run time and alike for a whole launch.
template <int DT, int V>
__device__ __forceinline__ void load_or_f32(const void* p, bool f32, int64_t i, float (&v)[V]) {
  if (DT == PGG_F32 || f32)
    load<PGG_F32, V>(p, i, v);
  else
    load<DT, V>(p, i, v);
}

}  // namespace vec
}  // namespace pgg
