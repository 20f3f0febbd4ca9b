// Shared by the two families of 8-bit products.
#pragma once

#include "gemm_tile.h"

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

}  // namespace moe
