// Shared by the row quantisations: loads of the element types that they take.
#pragma once

#include "layer_ops.h"

namespace moe {

template <int DT>
struct Elem {
  using type = uint16_t;
};
template <>
struct Elem<MOE_DTYPE_F32> {
  using type = float;
};
template <int DT>
__device__ __forceinline__ float widen(typename Elem<DT>::type v) {
  if constexpr (DT == MOE_DTYPE_F32)
    return v;
  else if constexpr (DT == MOE_DTYPE_BF16)
    return bf16_bits_to_f32(v);
  else
    return (float)__builtin_bit_cast(_Float16, v);
}

// 8 consecutive elements
template <int DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::type* p, float (&v)[8]) {
  if constexpr (DT == MOE_DTYPE_F32) {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = widen<DT>((uint16_t)(w[i] & 0xffffu));
      v[2 * i + 1] = widen<DT>((uint16_t)(w[i] >> 16));
    }
  }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

}  // namespace moe
