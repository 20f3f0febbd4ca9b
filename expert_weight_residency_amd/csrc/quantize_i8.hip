// Rows to 8-bit integers with one scale each: s = max|x| / 127 (fp32), q = the
// integer nearest to 127 x / max|x|, ties to even.
//
// The quotient is decided exactly. r = |x| * (127 / max|x|) in fp32 is within
// 127 * 2^-22 of the real quotient, so its nearest integer is right unless r
// lies within 2^-13 of half way between two; only then (about one element in
// 4000, and true ties) 127 |x| is compared with (n + 1/2) max|x| in fp64, where
// both products are exact (7 + 24 and 8 + 24 bits). Equal inputs give equal
// integers in any kernel or step, and nothing hangs on how a division rounds.
//
// One workgroup per row (a wavefront for rows of at most 512 elements), the row
// held in registers between the maximum and the rounding (up to 8192 elements;
// longer rows are read twice, the second time from the L2). Bound by its traffic
// at prefill sizes (4096 rows of 4096 bf16: 15.5 us, 50 MB at 3.2 TB/s; 24576
// rows of 2880 fp32: 69 us, 354 MB at 5.1 TB/s), by one round trip to memory for a
// few rows (3.1 us for one).
#include "layer_ops.h"

namespace moe {
namespace {

struct QuantArgs {
  const void* x;
  int64_t ld;
  int K;
  const int32_t* n_active;  // null: rows 0 .. gridDim.x - 1
  const int32_t* row_off;   // else the rows slots[0 .. row_off[n_active])
  const int32_t* slots;
  int8_t* q;
  float* scale;
};

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

// round-half-even of 127 |x| / most, with x's sign; most > 0 finite, inv = 127 / most
__device__ __forceinline__ int quant1(float x, float inv, float most) {
  const float a = __builtin_fabsf(x), r = a * inv;
  float n = __builtin_rintf(r);
  if (__builtin_expect(__builtin_fabsf(__builtin_fabsf(r - n) - 0.5f) < 0.000125f, 0)) {
    const double lo = __builtin_floor((double)r);  // the two candidates: lo, lo + 1
    const double d = 127.0 * (double)a - (lo + 0.5) * (double)most;
    const bool up = d > 0.0 || (d == 0.0 && ((int)lo & 1));
    n = (float)lo + (up ? 1.0f : 0.0f);
  }
  const int q = (int)n;
  return x < 0.0f ? -q : q;
}

// Largest |x| bits over the threads of one row (THREADS of them; NaN orders
// above infinity, which orders above every number).
template <int THREADS>
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  if constexpr (THREADS > 64) {
    __shared__ uint32_t part[THREADS / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) m = max(m, part[i]);
  }
  return m;
}

// NV: 8-element vectors each thread keeps (the whole row); 0: the row is read
// twice, element by element (long or unaligned rows)
template <int DT, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void quantize_rows(QuantArgs a) {
  using T = typename Elem<DT>::type;
  int64_t row = blockIdx.x;
  if (a.n_active) {
    if ((int)blockIdx.x >= a.row_off[*a.n_active]) return;  // the whole workgroup
    row = a.slots[blockIdx.x];
  }
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  int8_t* q = a.q + row * (int64_t)a.K;
  const int tid = threadIdx.x;
  float v[NV > 0 ? NV : 1][8];
  uint32_t m = 0;
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * THREADS + tid) * 8;
      if (e < a.K) {
        load8<DT>(x + e, v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
      }
    }
  } else {
    for (int e = tid; e < a.K; e += THREADS) m = max(m, abs_bits(widen<DT>(x[e])));
  }
  m = row_max<THREADS>(m);
  const float most = __uint_as_float(m);
  float scale = most / 127.0f;
  // a row with an infinity or NaN: zeros with scale NaN, so that what is
  // computed from it is NaN; one whose scale would be subnormal: zeros, scale 0
  const bool bad = m >= 0x7f800000u;
  const bool zero = bad || scale < 1.17549435e-38f;
  if (bad) scale = __uint_as_float(0x7fc00000u);
  else if (zero) scale = 0.0f;
  const float inv = zero ? 0.0f : 127.0f / most;
  if (tid == 0) a.scale[row] = scale;
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * THREADS + tid) * 8;
      if (e < a.K) {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int n = zero ? 0 : quant1(v[i][j], inv, most);
          w[j >> 2] |= (uint32_t)(n & 0xff) << (8 * (j & 3));
        }
        *reinterpret_cast<uint2*>(q + e) = make_uint2(w[0], w[1]);
      }
    }
  } else {
    for (int e = tid; e < a.K; e += THREADS)
      q[e] = (int8_t)(zero ? 0 : quant1(widen<DT>(x[e]), inv, most));
  }
}

template <int DT, int THREADS, int NV>
hipError_t go(const QuantArgs& a, int rows, hipStream_t s) {
  hipLaunchKernelGGL((quantize_rows<DT, THREADS, NV>), dim3((unsigned)rows), dim3(THREADS), 0, s,
                     a);
  return hipGetLastError();
}

template <int DT>
hipError_t pick(const QuantArgs& a, int rows, hipStream_t s) {
  const int es = dtype_bytes(DT);
  const bool vec = a.K % 8 == 0 && (a.ld * es) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.q) % 8 == 0;
  if (!vec || a.K > 8192) return go<DT, 256, 0>(a, rows, s);
  if (a.K <= 512) return go<DT, 64, 1>(a, rows, s);
  if (a.K <= 2048) return go<DT, 256, 1>(a, rows, s);
  if (a.K <= 4096) return go<DT, 256, 2>(a, rows, s);
  return go<DT, 256, 4>(a, rows, s);
}

}  // namespace

hipError_t launch_quantize_rows(const void* x, int dtype, int64_t ld, int rows, int K,
                                const moe_split* split, int8_t* q, float* scale,
                                hipStream_t stream) {
  QuantArgs a = {x, ld, K, nullptr, nullptr, nullptr, q, scale};
  if (split) {
    a.n_active = split->n_active;
    a.row_off = split->row_off;
    a.slots = split->slots;
  }
  switch (dtype) {
    case MOE_DTYPE_BF16: return pick<MOE_DTYPE_BF16>(a, rows, stream);
    case MOE_DTYPE_F16: return pick<MOE_DTYPE_F16>(a, rows, stream);
    default: return pick<MOE_DTYPE_F32>(a, rows, stream);
  }
}

}  // namespace moe
