// Products of 8-bit floating point (E4M3) rows with a scale per 128 elements of an
// activation row and per 128 x 128 block of the weights, in tiles, dense and
// grouped by expert.
//
//   y[r][n] = sum over blocks b of (sa[r][b] * sw[n / 128][b]) * p_b[r][n],
//   p_b[r][n] = sum over k in block b of a[r][k] w[n][k]
//
// Weights are the A operand (result rows), activations the B operand (result
// columns), so that a lane ends with 4 consecutive outputs of one activation row,
// which share one scale; p_b starts from zero and is added to the accumulator with
// one fma per output. Which element of its block a lane's byte is does not matter to
// the sum, as long as both operands agree: lane (r, q) holds granules q and 4 + q of
// row r.
//
// The FP8 matrix instruction adds products in groups of 8 of which each is cut at
// 2^-13 of the group's largest (measured: 2^16 + 2^2 gives 2^16; bits of other
// groups stay down to 2^-24), about 3e-5 of a sum of Gaussian terms. That is far
// below a 16-bit output's rounding, so products with such outputs use it, one
// v_mfma_f32_16x16x128_f8f6f4 per tile and block. Outputs in 32 bits, and gate/up,
// whose h is quantized again, take EXACT: both operands widened to bf16 (which holds
// every E4M3 value), 4 v_mfma_f32_16x16x32_bf16 per tile and block, at half the rate.
//
// Copies, buffers, swizzle and the order of tiles are those of gemm_i8_tile: a
// step takes 128 bytes, so one block, of each row of the tile.
#include "gemm_tile.h"
#include "mxfp4_common.h"
#include "tile_items.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// One operand of a tile: 32 bytes of a row per lane, or those as bf16.
template <bool EXACT>
struct Frag {
  i32x8 v;
  __device__ __forceinline__ Frag() {}
  __device__ __forceinline__ explicit Frag(i32x8 x) : v(x) {}
};
template <>
struct Frag<true> {
  bf16x8 v[4];
  __device__ __forceinline__ Frag() {}
  __device__ __forceinline__ explicit Frag(i32x8 x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * i], 1.0f, false);
      const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * i], 1.0f, true);
      const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * i + 1], 1.0f, false);
      const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * i + 1], 1.0f, true);
      v[i] = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
  }
};

__device__ __forceinline__ f32x4 block_product(const Frag<true>& a, const Frag<true>& b) {
  f32x4 p = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], p, 0, 0, 0);
  return p;
}

__device__ __forceinline__ f32x4 block_product(const Frag<false>& a, const Frag<false>& b) {
  // scale operands of 0 select the form without block scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4{0, 0, 0, 0}, 0, 0, 0, 0,
                                                          0, 0);
}

__device__ __forceinline__ float from_lane(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_ds_bpermute(4 * lane, __float_as_int(v)));
}

// TN x TM tile (weight rows x activation rows), WN x WM wavefronts, S buffers.
template <int TN, int TM, int WN, int WM, int S, bool GU, bool EXACT>
__global__ __launch_bounds__(64 * WN * WM, WN * WM / 2) void gemm_f8_tile(F8Args a, int tiles_n) {
  constexpr int kW = WN * WM, kRows = TN + TM, kCopies = kRows / 8 / kW;
  static_assert(kRows % (8 * kW) == 0 && TN % (8 * kW) == 0 && (S == 3 || S == 4),
                "whole copies per wavefront");
  static_assert((GU ? TN / 2 : TN) <= 128 && 128 % (GU ? TN / 2 : TN) == 0,
                "a tile's outputs lie in one block of weight rows");
  constexpr int NF = TN / WN / 16, MF = TM / WM / 16;  // MFMA tiles per wavefront
  static_assert(!GU || NF % 2 == 0, "gate and up tiles in pairs");
  constexpr int kSides = GU ? 2 : 1;
  __shared__ __align__(128) uint8_t buf0[kRows * 128];
  __shared__ __align__(128) uint8_t buf1[kRows * 128];
  __shared__ __align__(128) uint8_t buf2[kRows * 128];
  __shared__ __align__(128) uint8_t buf3[S > 3 ? kRows * 128 : 16];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K, blocks = (K + 127) / 128, nblocks = (N + 127) / 128;

  // which tile: [m0, m1) of the group's slots, outputs from n0
  int m0, m1, n0;
  const uint8_t* w = a.w;
  const float* sw = a.sw;
  if (a.slots) {
    extern __shared__ int tpre[];  // [n_active + 1]
    __shared__ int wsum[kW];
    const int na = *a.n_active;
    tiles::build_tile_prefix<TM, kW>(a.row_off, na, tpre, wsum);
    const int item = xcd_item(tpre[na] * tiles_n);
    if (item < 0) return;  // the whole workgroup
    // items of one expert: weight rows outermost, so that its tiles meet a
    // block of weights together
    const int e = tiles::row_of_tile(tpre, na, item / tiles_n);
    const int local = item - tpre[e] * tiles_n, nt = tpre[e + 1] - tpre[e];
    const int nb = local / nt, mt = local - nb * nt;
    m0 = a.row_off[e] + mt * TM;
    m1 = min(m0 + TM, a.row_off[e + 1]);
    n0 = nb * (GU ? TN / 2 : TN);
    const int64_t row = a.active_rows[e];
    w += row * kSides * N * (int64_t)K;
    sw += row * kSides * nblocks * (int64_t)blocks;
  } else {
    const int item = xcd_item((a.M + TM - 1) / TM * tiles_n);
    if (item < 0) return;
    const int mt = item / tiles_n, nb = item - mt * tiles_n;
    m0 = mt * TM;
    m1 = min(m0 + TM, a.M);
    n0 = nb * TN;
  }
  sw += (n0 / 128) * (int64_t)blocks;
  // weight row of tile row r (clamped into the matrix; such outputs are not
  // stored). Gate/up: 16 gate rows and the same 16 up rows in turn.
  auto wrow = [&](int r) {
    if constexpr (GU) return min(n0 + (r >> 5) * 16 + (r & 15), N - 1) + ((r >> 4) & 1) * N;
    else return min(n0 + r, N - 1);
  };
  auto arow = [&](int m) -> int64_t {
    if (!a.slots) return m;
    const int s = a.slots[m];
    return a.by_token ? s / a.k : s;
  };

  // copies: wavefront wv copies rows 8 (wv + kW i) .. + 7; lane l granule l % 8
  // of row l / 8, from where the swizzle has it
  const int gran = (lane & 7) ^ (lane >> 3);
  const uint8_t* src[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int r = 8 * (wv + kW * i) + (lane >> 3);
    const uint8_t* p = r < TN ? w + (int64_t)wrow(r) * K
                              : a.a + arow(min(m0 + (r - TN), m1 - 1)) * a.lda;
    src[i] = p + 16 * gran;
  }
  auto copy = [&](uint8_t* buf, int k0) {
    const bool in = k0 + 16 * gran < K;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const uint8_t* p = in ? src[i] + k0 : kZeros;
      // a select, not a branch around two copies
      asm volatile("" : "+v"(p));
      __builtin_amdgcn_global_load_lds(p, buf + 1024 * (wv + kW * i), 16, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  f32x4 acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const int wn = wv % WN, wm = wv / WN, r = lane & 15, q = lane >> 4;

  // scales of S steps at a time: lane (r, q) holds those of step s + q for the
  // rows 16 j + r of its tiles, 0 past the end of K (the copies bring zeros there)
  const float* xs[MF];
#pragma unroll
  for (int j = 0; j < MF; ++j)
    xs[j] = a.sa + arow(min(m0 + (wm * MF + j) * 16 + r, m1 - 1)) * blocks;
  auto scales = [&](int s, float (&x)[MF], float (&v)[kSides]) {
    const int b = min(s + q, blocks - 1);
    const bool in = s + q < blocks;
#pragma unroll
    for (int j = 0; j < MF; ++j) x[j] = in ? xs[j][b] : 0.0f;
#pragma unroll
    for (int h = 0; h < kSides; ++h) v[h] = in ? sw[h * nblocks * (int64_t)blocks + b] : 0.0f;
  };
  float nx[MF], nw[kSides], cur[kSides][MF];

  auto frag = [&](const uint8_t* buf, int row) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(buf + row * 128 + 16 * (q ^ (row & 7)));
    const i32x4 hi = *reinterpret_cast<const i32x4*>(buf + row * 128 + 16 * ((4 + q) ^ (row & 7)));
    return Frag<EXACT>(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto compute = [&](const uint8_t* buf, int step) {
    Frag<EXACT> bf[MF], af[NF];
#pragma unroll
    for (int j = 0; j < MF; ++j) bf[j] = frag(buf, TN + (wm * MF + j) * 16 + r);
#pragma unroll
    for (int i = 0; i < NF; ++i) af[i] = frag(buf, (wn * NF + i) * 16 + r);
    float sc[kSides][MF];
#pragma unroll
    for (int h = 0; h < kSides; ++h)
#pragma unroll
      for (int j = 0; j < MF; ++j) sc[h][j] = from_lane(cur[h][j], 16 * step + r);
    f32x4 p[NF][MF];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < MF; ++j) p[i][j] = block_product(af[i], bf[j]);
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < MF; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[i][j][v] = __builtin_fmaf(sc[GU ? i & 1 : 0][j], p[i][j][v], acc[i][j][v]);
  };

  scales(0, nx, nw);
  // past the end of K a copy brings zeros, which the products ignore
  copy(buf0, 0);
  copy(buf1, 128);
  if constexpr (S > 3) copy(buf2, 256);
  for (int s = 0; s < blocks; s += S) {
#pragma unroll
    for (int h = 0; h < kSides; ++h)
#pragma unroll
      for (int j = 0; j < MF; ++j) cur[h][j] = nx[j] * nw[h];
    scales(s + S, nx, nw);
    // each step: its copies (the oldest) have arrived for every wavefront, and
    // the buffer the last step read is free for the copies S - 1 steps ahead
    tile_barrier(vm_lds((S - 2) * kCopies));
    copy(S == 3 ? buf2 : buf3, (s + S - 1) * 128);
    compute(buf0, 0);
    tile_barrier(vm_lds((S - 2) * kCopies));
    copy(buf0, (s + S) * 128);
    compute(buf1, 1);
    tile_barrier(vm_lds((S - 2) * kCopies));
    copy(buf1, (s + S + 1) * 128);
    compute(buf2, 2);
    if constexpr (S > 3) {
      tile_barrier(vm_lds((S - 2) * kCopies));
      copy(buf2, (s + S + 2) * 128);
      compute(buf3, 3);
    }
  }

  __builtin_amdgcn_s_waitcnt(vm_lds(0));  // no copy outlives the workgroup's LDS

  // lane (r, q): outputs 16 i + 4 q + v of activation row 16 j + r
  auto rows = [&](auto f) {
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int m = m0 + (wm * MF + j) * 16 + r;
      if (m >= m1) continue;
      f(j, a.slots ? (int64_t)a.slots[m] : (int64_t)m);
    }
  };
  if constexpr (GU) {
    rows([&](int j, int64_t orow) {
#pragma unroll
      for (int i = 0; i < NF; i += 2) {
        const int n = n0 + (wn * NF + i) * 8 + 4 * q;
        if (n >= N) continue;  // N is a multiple of 64
        float h[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) h[v] = mx::silu_f32(acc[i][j][v]) * acc[i + 1][j][v];
        *reinterpret_cast<float4*>(static_cast<float*>(a.y) + orow * a.ldy + n) =
            make_float4(h[0], h[1], h[2], h[3]);
      }
    });
  } else {
    with_output(a, [&](auto type, auto vec) {
      rows([&](int j, int64_t orow) {
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          const int n = n0 + (wn * NF + i) * 16 + 4 * q;
          if (n >= N) continue;
          const float y[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
          store4<type(), vec()>(a, orow, n, y);
        }
      });
    });
  }
}

template <int TN, int TM, int WN, int WM, int S, bool GU, bool EXACT>
hipError_t go(const F8Args& a, hipStream_t stream) {
  const int per = GU ? TN / 2 : TN;
  const int64_t tiles_n = (a.N + per - 1) / per;
  int64_t tiles_m, lds = 0;
  if (a.slots) {
    // at most one part-filled tile per active row
    const int64_t cap = a.n_rows < a.M ? a.n_rows : a.M;
    tiles_m = cap + a.M / TM;
    lds = (cap + 1) * sizeof(int);
  } else {
    tiles_m = (a.M + TM - 1) / TM;
  }
  const unsigned grid = (unsigned)((tiles_m * tiles_n + kXcds - 1) / kXcds * kXcds);
  hipLaunchKernelGGL((gemm_f8_tile<TN, TM, WN, WM, S, GU, EXACT>), dim3(grid), dim3(64 * WN * WM), lds,
                     stream, a, (int)tiles_n);
  return hipGetLastError();
}

}  // namespace

// The finest tiles any of the kernels takes for such a call, times its threads.
bool gemm_f8_fits(const F8Args& a) {
  const int64_t limit = ((int64_t)1 << 32) - 512 * kXcds;
  if (a.slots) {
    const int64_t cap = a.n_rows < a.M ? a.n_rows : a.M;
    return (cap + a.M / 64) * ((a.N + 63) / 64) * 512 < limit;
  }
  return ((a.M + 63) / 64) * (int64_t)((a.N + 31) / 32) * 256 < limit;
}

hipError_t launch_gemm_f8(const F8Args& a, hipStream_t s) {
  if (a.gate_up) return go<128, 64, 4, 2, 3, true, true>(a, s);
  if (a.slots) return go<128, 64, 4, 2, 3, false, false>(a, s);
  const int cus = device_cus();
  auto tiles = [&](int tn, int tm) {
    return (int64_t)((a.N + tn - 1) / tn) * ((a.M + tm - 1) / tm);
  };
  const bool wide = a.dtype == MOE_DTYPE_F32;
  if (tiles(128, 64) >= cus)
    return wide ? go<128, 64, 4, 2, 3, false, true>(a, s) : go<128, 64, 4, 2, 3, false, false>(a, s);
  if (tiles(64, 64) >= cus)
    return wide ? go<64, 64, 2, 2, 3, false, true>(a, s) : go<64, 64, 2, 2, 3, false, false>(a, s);
  return wide ? go<32, 64, 2, 2, 4, false, true>(a, s) : go<32, 64, 2, 2, 4, false, false>(a, s);
}

}  // namespace moe
