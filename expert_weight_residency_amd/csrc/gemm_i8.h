// Shared by the two families of 8-bit products.
#pragma once

#include <type_traits>

#include "layer_ops.h"

namespace moe {

hipError_t launch_gemm_i8_tile(const I8Args& a, hipStream_t stream);
bool gemm_i8_tile_fits(const I8Args& a);
hipError_t launch_gemm_i8_stream(const I8Args& a, hipStream_t stream);
bool gemm_i8_use_stream(const I8Args& a);

__device__ __forceinline__ void store1(const I8Args& a, int64_t row, int n, float y) {
  if (a.dtype == MOE_DTYPE_F32)
    static_cast<float*>(a.y)[row * a.ldy + n] = y;
  else if (a.dtype == MOE_DTYPE_BF16)
    static_cast<uint16_t*>(a.y)[row * a.ldy + n] = (uint16_t)f32_to_bf16_bits(y);
  else
    static_cast<_Float16*>(a.y)[row * a.ldy + n] = (_Float16)y;
}

// Outputs n .. n+3 (n a multiple of 4) of a row in type DT. VEC: N is a multiple
// of 4 and every such group is aligned for one store; else the outputs past N
// are left out one by one.
template <int DT, bool VEC>
__device__ __forceinline__ void store4(const I8Args& a, int64_t row, int n, const float (&y)[4]) {
  if constexpr (DT == MOE_DTYPE_F32) {
    float* p = static_cast<float*>(a.y) + row * a.ldy + n;
    if constexpr (VEC) {
      *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (n + v < a.N) p[v] = y[v];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(a.y) + row * a.ldy + n;
    uint32_t b[4];
#pragma unroll
    for (int v = 0; v < 4; ++v)
      b[v] = DT == MOE_DTYPE_BF16 ? f32_to_bf16_bits(y[v])
                                  : (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)y[v]);
    if constexpr (VEC) {
      *reinterpret_cast<uint2*>(p) = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (n + v < a.N) p[v] = (uint16_t)b[v];
    }
  }
}

// f(type, vec) for the launch's output type and alignment, both compile-time in
// f: the branches sit around one copy of the epilogue each. (Inside it, at every
// store, they made the 256 x 256 tile's epilogue thousands of instructions.)
template <typename F>
__device__ __forceinline__ void with_output(const I8Args& a, F f) {
  const bool vec = ((a.ldy | a.N) & 3) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.y) & (4 * dtype_bytes(a.dtype) - 1)) == 0;
  auto by_type = [&](auto v) {
    if (a.dtype == MOE_DTYPE_BF16) f(std::integral_constant<int, MOE_DTYPE_BF16>(), v);
    else if (a.dtype == MOE_DTYPE_F16) f(std::integral_constant<int, MOE_DTYPE_F16>(), v);
    else f(std::integral_constant<int, MOE_DTYPE_F32>(), v);
  };
  if (vec) by_type(std::true_type());
  else by_type(std::false_type());
}

}  // namespace moe
