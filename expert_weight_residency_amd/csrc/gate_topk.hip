// The router's gate: the k largest logits of each token in descending order
// (ties to the lower expert id) and their softmax weights.
//
// One wavefront per token. Lane l holds the logits of experts l, l + 64, ... in
// registers, as unsigned keys that order like the numbers (a masked expert,
// -inf or NaN, has key 0; both zeros share one key). A pick is a wave-wide
// maximum of the keys followed by a wave-wide minimum of the expert ids that
// hold it; the winner's key is then set to 0. The softmax is taken against the
// first pick, which is the row's maximum; all sums are in fp32.
//
// Bound: a step of a few tokens is one round trip to memory and k dependent
// picks (7 tokens, 384 experts, top-6: 4.0 us, most of it the launch); at 4096
// tokens the picks' cross-lane steps bound it (7.2 us), not the reads (3 MB).
// Above 2048 experts a lane holds 64 logits and the comparisons' masks spill 141
// scalar registers: 4096 tokens of 2048 experts 17.2 us, of 2049 42.5, of 4096
// 59.4 (7 tokens: 9.9, 13.8, 18.0).
#include "layer_ops.h"

namespace moe {
namespace {

constexpr int kWaves = 4;  // tokens per workgroup

// f over all 64 lanes, in every lane: within rows of 16 by DPP (quad
// permutations, mirrors), then across rows and halves with the lane swaps, all
// of them VALU operations (the LDS-based shuffles took most of the kernel's
// time: 5.7 us for 7 tokens, 9.0 for 4096).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, F f) {
  v = f(v, dpp<0xb1>(v));   // quad_perm [1,0,3,2]
  v = f(v, dpp<0x4e>(v));   // quad_perm [2,3,0,1]
  v = f(v, dpp<0x141>(v));  // row_half_mirror
  v = f(v, dpp<0x140>(v));  // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = f(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return f(b[0], b[1]);
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int dtype) {
  if (dtype == MOE_DTYPE_F32) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  if (dtype == MOE_DTYPE_BF16) return bf16_bits_to_f32(b);
  return (float)__builtin_bit_cast(_Float16, b);
}

__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > -__builtin_inff())) return 0;  // -inf and NaN
  const uint32_t b = v == 0.0f ? 0u : __float_as_uint(v);
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key >> 31) ? key & 0x7fffffffu : ~key);
}

template <int V>  // logits per lane
__global__ __launch_bounds__(64 * kWaves) void topk_gate(const void* __restrict__ logits,
                                                         int dtype, int64_t ld, int T, int E,
                                                         int k, int norm,
                                                         int32_t* __restrict__ ids,
                                                         float* __restrict__ w) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= T) return;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < E ? order_key(load_as_f32(logits, (int64_t)t * ld + e, dtype)) : 0u;
  }
  int my_id = -1;      // lane j: pick j
  uint32_t my_key = 0;
  float top = 0.0f, all = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, key[i]);
    m = wave_reduce(m, [](uint32_t a, uint32_t b) { return max(a, b); });
    if (m == 0) break;  // wave-uniform: nothing is left
    uint32_t e = 0xffffffffu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) e = key[i] == m ? (uint32_t)(lane + 64 * i) : e;
    e = wave_reduce(e, [](uint32_t a, uint32_t b) { return min(a, b); });
    if (j == 0) {
      top = key_value(m);
      if (norm == MOE_GATE_NORM_ALL) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (key[i]) s += key[i] == m ? 1.0f : expf(key_value(key[i]) - top);
        all = wave_sum(s);
      }
    }
    if (lane == j) {
      my_id = (int)e;
      my_key = m;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = (uint32_t)(lane + 64 * i) == e ? 0u : key[i];
  }
  // equal to the maximum: weight exp(0), also for an infinite one
  const float v = my_key ? key_value(my_key) : 0.0f;
  const float p = my_key ? (v == top ? 1.0f : expf(v - top)) : 0.0f;
  const float total = norm == MOE_GATE_NORM_ALL ? all : wave_sum(p);
  if (lane < k) {
    ids[(int64_t)t * k + lane] = my_id;
    w[(int64_t)t * k + lane] = my_key ? p / total : 0.0f;
  }
}

template <int V>
hipError_t go(const void* logits, int dtype, int64_t ld, int T, int E, int k, int norm,
              int32_t* ids, float* w, hipStream_t stream) {
  hipLaunchKernelGGL((topk_gate<V>), dim3((unsigned)((T + kWaves - 1) / kWaves)),
                     dim3(64 * kWaves), 0, stream, logits, dtype, ld, T, E, k, norm, ids, w);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_topk_gate(const void* logits, int dtype, int64_t ld, int T, int E, int k,
                            int norm, int32_t* ids, float* w, hipStream_t stream) {
  const int per = (E + 63) / 64;  // at most 64: E <= MOE_MAX_EXPERTS
  const auto f = per <= 1    ? go<1>
                 : per <= 2  ? go<2>
                 : per <= 4  ? go<4>
                 : per <= 6  ? go<6>
                 : per <= 8  ? go<8>
                 : per <= 16 ? go<16>
                 : per <= 32 ? go<32>
                             : go<64>;
  return f(logits, dtype, ld, T, E, k, norm, ids, w, stream);
}

}  // namespace moe
