// Rows to 8-bit floating point (E4M3) with one scale per 128 elements: s =
// max|x| / 448 (fp32) over the group, q = the E4M3 value nearest to 448 x /
// max|x|, ties to the even code.
//
// The nearest value is decided exactly. r = x * (448 / max|x|) in fp32 is within
// 2^-22 of the real quotient (relative), so where r (1 - 2^-21) and r (1 + 2^-21)
// convert to one code, that is the answer; only else (about one element in
// 30000, and true ties) 448 |x| is compared with the middle of the two codes'
// values times max|x| in fp64, where both products are exact (3 + 24 and 5 + 24
// bits).
//
// 16 lanes take one group, 8 elements each, so that nothing crosses a wavefront. Bound by
// the rows' bytes: 4096 x 4096 bf16 14.7 us (51 MB, 3.5 TB/s), 24576 x 2880 fp32 rows of a
// split 76 us (356 MB, 4.7 TB/s); one row of 4096 3.1 us, of which nearly all is launch.
#include "quantize.h"

namespace moe {
namespace {

struct QuantF8Args {
  const void* x;
  int64_t ld;
  int rows, K, blocks;      // blocks: groups per row
  int shift;                // a workgroup's 16 groups: 1 << shift of each row
  const int32_t* n_active;  // null: rows 0 .. rows - 1
  const int32_t* row_off;   // else the rows slots[0 .. row_off[n_active])
  const int32_t* slots;
  uint8_t* q;
  float* scale;
};

// The code of 448 |x| / most, with x's sign, where two neighbours (lower one lo)
// are left.
__device__ uint32_t decide(float x, float most, uint32_t lo) {
  const double a = (double)__builtin_amdgcn_cvt_f32_fp8((int)lo, 0);
  const double b = (double)__builtin_amdgcn_cvt_f32_fp8((int)lo + 1, 0);
  const double d = 448.0 * (double)__builtin_fabsf(x) - 0.5 * (a + b) * (double)most;
  const uint32_t c = lo + (d > 0.0 || (d == 0.0 && (lo & 1)) ? 1 : 0);
  return c | (__float_as_uint(x) >> 24 & 0x80u);
}

__device__ __forceinline__ uint32_t pack4(const float* v) {
  int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], p, true);
}

// VEC: 8 consecutive elements of a lane are one aligned load and store
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void quantize_f8(QuantF8Args a) {
  using T = typename Elem<DT>::type;
  const int g = threadIdx.x >> 4, l = threadIdx.x & 15;
  int row = (blockIdx.x << (4 - a.shift)) + (g >> a.shift);
  const int listed = a.n_active ? a.row_off[*a.n_active] : a.rows;
  if (row >= listed) return;  // whole groups of 16 lanes
  if (a.n_active) row = a.slots[row];
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  uint8_t* q = a.q + row * (int64_t)a.K;
  for (int blk = (blockIdx.y << a.shift) + (g & ((1 << a.shift) - 1)); blk < a.blocks;
       blk += gridDim.y << a.shift) {
    // element i of this lane: e + i (VEC) or e + 16 i
    const int e = blk * 128 + (VEC ? 8 * l : l);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if constexpr (VEC) {
      if (e < a.K) load8<DT>(x + e, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + 16 * i < a.K) v[i] = widen<DT>(x[e + 16 * i]);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 16));
    const float most = __uint_as_float(m);
    float scale = most / 448.0f;
    // a group with an infinity or NaN: zeros with scale NaN, so that what is
    // computed from it is NaN; one whose scale would be subnormal: zeros, scale 0
    const bool bad = m >= 0x7f800000u;
    const bool zero = bad || scale < 1.17549435e-38f;
    if (bad) scale = __uint_as_float(0x7fc00000u);
    else if (zero) scale = 0.0f;
    if (l == 0) a.scale[row * (int64_t)a.blocks + blk] = scale;
    const float inv = zero ? 0.0f : 448.0f / most;
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = zero ? 0.0f : v[i] * inv;
      lo[i] = r * (1.0f - 0x1p-21f);
      hi[i] = r * (1.0f + 0x1p-21f);
    }
    uint32_t w[2] = {pack4(lo), pack4(lo + 4)};
    const uint32_t up[2] = {pack4(hi), pack4(hi + 4)};
    if (__builtin_expect((w[0] ^ up[0]) | (w[1] ^ up[1]), 0)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = 8 * (i & 3);
        const uint32_t c = w[i >> 2] >> at & 0xffu;
        if (c != (up[i >> 2] >> at & 0xffu))
          w[i >> 2] = (w[i >> 2] & ~(0xffu << at)) | decide(v[i], most, c & 0x7fu) << at;
      }
    }
    if constexpr (VEC) {
      if (e < a.K) *reinterpret_cast<uint2*>(q + e) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + 16 * i < a.K) q[e + 16 * i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
  }
}

template <int DT>
hipError_t pick(QuantF8Args a, hipStream_t s) {
  const int es = dtype_bytes(DT);
  const bool vec = a.K % 8 == 0 && (a.ld * es) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.q) % 8 == 0;
  a.shift = 0;
  while (a.shift < 4 && (1 << a.shift) < a.blocks) ++a.shift;
  const int per = 16 >> a.shift;  // rows of a workgroup
  const unsigned gx = (unsigned)((a.rows + per - 1) / per);
  // a row's groups go over gridDim.y, unless the rows alone are a full grid
  const unsigned gy = a.rows > 1 << 16 ? 1u : (unsigned)((a.blocks + 15) / 16);
  if (vec)
    hipLaunchKernelGGL((quantize_f8<DT, true>), dim3(gx, gy), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((quantize_f8<DT, false>), dim3(gx, gy), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_f8(const void* x, int dtype, int64_t ld, int rows, int K,
                              const moe_split* split, uint8_t* q, float* scale,
                              hipStream_t stream) {
  QuantF8Args a = {x, ld, rows, K, (K + 127) / 128, 0, nullptr, nullptr, nullptr, q, scale};
  if (split) {
    a.n_active = split->n_active;
    a.row_off = split->row_off;
    a.slots = split->slots;
  }
  switch (dtype) {
    case MOE_DTYPE_BF16: return pick<MOE_DTYPE_BF16>(a, stream);
    case MOE_DTYPE_F16: return pick<MOE_DTYPE_F16>(a, stream);
    default: return pick<MOE_DTYPE_F32>(a, stream);
  }
}

}  // namespace moe
