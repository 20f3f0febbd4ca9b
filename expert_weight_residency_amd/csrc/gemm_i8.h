// Shared by the two families of 8-bit products.
#pragma once

#include "layer_ops.h"

namespace moe {

hipError_t launch_gemm_i8_tile(const I8Args& a, hipStream_t stream);
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

// Outputs n .. n+3 (n a multiple of 4) of a row; the ones past N are left out.
__device__ __forceinline__ void store4(const I8Args& a, int64_t row, int n, const float (&y)[4]) {
  const int es = dtype_bytes(a.dtype);
  // rows whose groups of 4 are aligned; wave-uniform
  const bool vec = (a.ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(a.y) & (4 * es - 1)) == 0;
  if (vec && n + 4 <= a.N) {
    if (a.dtype == MOE_DTYPE_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.y) + row * a.ldy + n) =
          make_float4(y[0], y[1], y[2], y[3]);
    } else {
      uint32_t b[4];
#pragma unroll
      for (int v = 0; v < 4; ++v)
        b[v] = a.dtype == MOE_DTYPE_BF16
                   ? f32_to_bf16_bits(y[v])
                   : (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)y[v]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + row * a.ldy + n) =
          make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
    }
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (n + v < a.N) store1(a, row, n + v, y[v]);
  }
}

}  // namespace moe
