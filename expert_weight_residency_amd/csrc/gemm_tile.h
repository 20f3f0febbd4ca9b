// Shared by the tiled products (8-bit integers, 8-bit floating point, products
// grouped by expert): waits for global-to-LDS copies, the order of tiles over the
// XCDs, and the epilogue's stores.
#pragma once

#include <type_traits>

#include "layer_ops.h"

namespace moe {

// Source of the granules past the end of a row.
static __device__ __align__(16) const uint8_t kZeros[16] = {};

// s_waitcnt immediate: at most n vector-memory operations and no LDS operation
// outstanding.
constexpr int vm_lds(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

#define tile_barrier(W)                                    \
  do {                                                     \
    __builtin_amdgcn_sched_barrier(0);                     \
    __builtin_amdgcn_s_waitcnt(W);                         \
    __builtin_amdgcn_s_barrier();                          \
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup"); \
    __builtin_amdgcn_sched_barrier(0);                     \
  } while (0)

// Workgroups go round the 8 XCDs in turn, each with its own L2: XCD x takes the
// x-th eighth of the items, so that neighbours, which share rows, meet in one
// L2. The item of this workgroup, -1: none.
constexpr int kXcds = 8;
__device__ __forceinline__ int xcd_item(int items) {
  const int per = (items + kXcds - 1) / kXcds, at = blockIdx.x / kXcds;
  const int item = (blockIdx.x % kXcds) * per + at;
  return at < per && item < items ? item : -1;
}

// 16 bytes per lane from p to LDS, lane after lane.
__device__ __forceinline__ void copy16(uint8_t* buf, const uint8_t* p) {
  asm volatile("" : "+v"(p));  // a select, not a branch around two copies
  __builtin_amdgcn_global_load_lds(p, buf, 16, 0, 0);
}

// 16 bytes per lane from base + off to LDS, zeros where off is not below bytes. base and
// bytes are the same in all lanes.
__device__ __forceinline__ void copy16(uint8_t* buf, const uint8_t* base, uint32_t bytes,
                                       uint32_t off) {
  auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes, 0x27000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rsrc, (__attribute__((address_space(3))) void*)buf, 16, off, 0, 0, 0);
}

// Two values rounded to a 16-bit type, the first one low.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == MOE_DTYPE_BF16) {
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    const f16x2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
}

// Outputs n .. n+3 (n a multiple of 4) of a row in type DT. VEC: N is a multiple
// of 4 and every such group is aligned for one store; else the outputs past N
// are left out one by one.
template <int DT, bool VEC, typename A>
__device__ __forceinline__ void store4(const A& a, int64_t row, int n, const float (&y)[4]) {
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
// BITS: 16 or 32 where only such types come here.
template <int BITS = 0, typename A, typename F>
__device__ __forceinline__ void with_output(const A& a, F f) {
  const bool vec = ((a.ldy | a.N) & 3) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.y) & (4 * dtype_bytes(a.dtype) - 1)) == 0;
  auto by_type = [&](auto v) {
    if constexpr (BITS != 32) {
      if (a.dtype == MOE_DTYPE_BF16) return f(std::integral_constant<int, MOE_DTYPE_BF16>(), v);
      if (BITS == 16 || a.dtype == MOE_DTYPE_F16)
        return f(std::integral_constant<int, MOE_DTYPE_F16>(), v);
    }
    if constexpr (BITS != 16) f(std::integral_constant<int, MOE_DTYPE_F32>(), v);
  };
  if (vec) by_type(std::true_type());
  else by_type(std::false_type());
}

}  // namespace moe
