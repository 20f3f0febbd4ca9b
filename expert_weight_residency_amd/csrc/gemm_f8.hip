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
// Every sum is taken in fp32. The FP8 matrix instructions do not: they cut each product at
// 2^-13 of the largest of the 8 that they add first (measured, for v_mfma_f32_16x16x128_f8f6f4
// and v_mfma_f32_16x16x32_fp8_fp8 alike: 2^16 + 2^2 gives 2^16, and 448 * 448 - 448 * 448 + 90
// gives 0), so that nothing bounds a sum's error by its own size; an activation of a hundred
// times its neighbours alone takes it to 2.7e-4 of the products' magnitudes. So both operands
// are widened to bf16, which holds every E4M3 value, for 4 v_mfma_f32_16x16x32_bf16 per tile
// and block, at half the rate: these keep 24 bits below the largest of 8 (1e-8 of a sum of
// Gaussian terms). 4096 x 5760 x 4096 106 us with the FP8 instruction, 172 so; one row 9.5 and
// 11.3; the down product of 4096 tokens 1,353 and 1,526.
//
// Copies, buffers, swizzle and the order of tiles are those of gemm_i8_tile: a
// step takes 128 bytes, so one block, of each row of the tile.
//
// Bounds (times of a trace). Few rows: the weights' bytes (384 experts, H 4096, I 2880, 7
// tokens: 141 + 80 us, 5.7 and 5.1 TB/s). One row of 5760 x 4096, 12.8 us: bytes in flight, 180
// workgroups on 256 CUs with 12 KB of weights each, half of every copy being the one
// activation row again. The FFN of 4096 tokens: gate/up 2.71 ms (9.1 GB) and down 1.52 (4.5
// GB): copies into LDS at 3.4 and 3.0 TB/s from HBM, and the widening; the matrix cores are
// busy for 0.35 and 0.33 of the CUs' busy cycles. 128 x 64 tiles on 2 x 2 wavefronts (4,155 us
// for that FFN while down took the FP8 instruction; then 4 x 2 4,425, 64 x 64 4,715, 128 x 32
// 4,840, 128 x 128 5,586). Large dense products: gemm_f8_big.
#include <algorithm>

#include "gemm_tile.h"
#include "mxfp4_common.h"
#include "tile_items.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// One operand of a tile: a lane's 32 bytes of a row, as bf16.
struct Frag {
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

// Quarter i of a block's product: the four in order are the block's sum.
__device__ __forceinline__ f32x4 quarter(const Frag& a, const Frag& b, int i, f32x4 p) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], p, 0, 0, 0);
}

__device__ __forceinline__ f32x4 block_product(const Frag& a, const Frag& b) {
  f32x4 p = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) p = quarter(a, b, i, p);
  return p;
}

__device__ __forceinline__ float from_lane(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_ds_bpermute(4 * lane, __float_as_int(v)));
}

// TN x TM tile (weight rows x activation rows), WN x WM wavefronts, S buffers; W32:
// outputs of 32 bits (gate/up's h among them), else 16.
template <int TN, int TM, int WN, int WM, int S, bool GU, bool W32>
__global__ __launch_bounds__(64 * WN * WM, WN * WM / 2) void gemm_f8_tile(F8Args a, int tiles_n) {
  constexpr int kW = WN * WM, kRows = TN + TM, kCopies = kRows / 8 / kW;
  static_assert(kRows % (8 * kW) == 0 && TN % (8 * kW) == 0 && (S == 3 || S == 4),
                "whole copies per wavefront");
  static_assert((GU ? TN / 2 : TN) <= 128 && 128 % (GU ? TN / 2 : TN) == 0,
                "a tile's outputs lie in one block of weight rows");
  constexpr int NF = TN / WN / 16, MF = TM / WM / 16;  // MFMA tiles per wavefront
  static_assert(!GU || (NF % 2 == 0 && W32), "gate and up tiles in pairs, h in 32 bits");
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

  // scales of S steps at a time: lane (r, q) holds those of step s + q for the rows 16 j
  // + r of its tiles, taken as 0 past the end of K (the copies bring zeros there) only
  // once they are used: a select at the loads would wait for them, and for every copy
  const float* xs[MF];
#pragma unroll
  for (int j = 0; j < MF; ++j)
    xs[j] = a.sa + arow(min(m0 + (wm * MF + j) * 16 + r, m1 - 1)) * blocks;
  auto scales = [&](int s, float (&x)[MF], float (&v)[kSides]) {
    const int b = min(s + q, blocks - 1);
#pragma unroll
    for (int j = 0; j < MF; ++j) x[j] = xs[j][b];
#pragma unroll
    for (int h = 0; h < kSides; ++h) v[h] = sw[h * nblocks * (int64_t)blocks + b];
  };
  float nx[MF], nw[kSides], cur[kSides][MF];

  auto frag = [&](const uint8_t* buf, int row) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(buf + row * 128 + 16 * (q ^ (row & 7)));
    const i32x4 hi = *reinterpret_cast<const i32x4*>(buf + row * 128 + 16 * ((4 + q) ^ (row & 7)));
    return Frag(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto compute = [&](const uint8_t* buf, int step) {
    Frag bf[MF], af[NF];
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
      for (int j = 0; j < MF; ++j) cur[h][j] = s + q < blocks ? nx[j] * nw[h] : 0.0f;
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
    with_output<W32 ? 32 : 16>(a, [&](auto type, auto vec) {
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

// Dense products with 16-bit outputs, large enough to fill the card with wide tiles: 8
// wavefronts (2 x 4) of TN/2 x TM/4 outputs, S buffers of 128 bytes, one block, per row.
// The weights' operand of one or two tiles on is read from LDS while a row of tiles is
// multiplied, and the row before it is scaled and added; the one barrier per step sits
// after the last read of the step's buffer. Copies go out one row of tiles at a time: a
// step's, asked for at once by all wavefronts, hold the products up. 4096 x 5760 x 4096: 172
// us, 1.12 PFLOP/s (130 at the rate of the largest library products in bf16); the matrix
// cores are busy for 0.53 of the CUs' busy cycles: the widening (16 conversions per operand
// and lane), operand reads, the scales' fma on every tile and the last round of tiles.
template <int TN, int TM, int S>
__global__ __launch_bounds__(512, 2) void gemm_f8_big(F8Args a, int tiles_n) {
  constexpr int WN = 2, WM = 4, kW = 8;
  constexpr int kCopiesA = TN / 8 / kW, kCopiesB = TM / 8 / kW, kCopies = kCopiesA + kCopiesB;
  static_assert(TN % (8 * kW) == 0 && TM % (8 * kW) == 0 && (S == 2 || S == 3), "whole copies");
  constexpr int NF = TN / WN / 16, MF = TM / WM / 16;
  static_assert(128 % (TN / WN) == 0, "a wavefront's weight rows lie in one block");
  __shared__ __align__(128) uint8_t buf0[(TN + TM) * 128];
  __shared__ __align__(128) uint8_t buf1[(TN + TM) * 128];
  __shared__ __align__(128) uint8_t buf2[S > 2 ? (TN + TM) * 128 : 16];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wv % WN, wm = wv / WN, r = lane & 15, q = lane >> 4;
  const int N = a.N, K = a.K, M = a.M, blocks = (K + 127) / 128;
  // items in groups of 8 rows of tiles, column by column, so that an XCD's share is
  // about square and its L2 meets few rows of either operand
  const int tiles_m = (M + TM - 1) / TM;
  const int item = xcd_item(tiles_m * tiles_n);
  if (item < 0) return;
  const int group = item / (8 * tiles_n), local = item - group * 8 * tiles_n;
  const int gm = min(8, tiles_m - 8 * group);
  const int m0 = (8 * group + local % gm) * TM, n0 = local / gm * TN;

  constexpr uint32_t kOutside = 1u << 31;  // above the bytes of any copy
  const int gran = (lane & 7) ^ (lane >> 3);
  const uint8_t *wbase = a.w + (int64_t)n0 * K, *abase = a.a + m0 * a.lda;
  uint32_t offa[kCopiesA], offb[kCopiesB];
#pragma unroll
  for (int i = 0; i < kCopiesA; ++i)
    offa[i] = min(8 * (wv + kW * i) + (lane >> 3), N - 1 - n0) * K + 16 * gran;
#pragma unroll
  for (int i = 0; i < kCopiesB; ++i)
    offb[i] = min(8 * (wv + kW * i) + (lane >> 3), M - 1 - m0) * (int)a.lda + 16 * gran;
  // copies [from, to) of step s's: weights first
  auto copy = [&](uint8_t* buf, int s, int from, int to) __attribute__((always_inline)) {
    const bool in = s * 128 + 16 * gran < K;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      if (i < from || i >= to) continue;
      if (i < kCopiesA)
        copy16(buf + 1024 * (wv + kW * i), wbase + (int64_t)s * 128, kOutside,
               in ? offa[i < kCopiesA ? i : 0] : kOutside);
      else
        copy16(buf + TN * 128 + 1024 * (wv + kW * (i - kCopiesA)), abase + (int64_t)s * 128,
               kOutside, in ? offb[i < kCopiesA ? 0 : i - kCopiesA] : kOutside);
    }
  };

  // scales of 4 steps at a time, as in gemm_f8_tile
  const int block = min((n0 + wn * (TN / WN)) / 128, (N - 1) / 128);
  const float* sw = a.sw + block * (int64_t)blocks;
  const float* sbase = a.sa + m0 * (int64_t)blocks;
  uint32_t offs[MF];
#pragma unroll
  for (int j = 0; j < MF; ++j)
    offs[j] = min((wm * MF + j) * 16 + r, M - 1 - m0) * blocks;
  float nx[MF], nw, cur[MF];
  auto scales = [&](int s) {
    const int b = min(s + q, blocks - 1);
#pragma unroll
    for (int j = 0; j < MF; ++j) nx[j] = sbase[offs[j] + b];
    nw = sw[b];
  };
  auto take = [&](int s) {
    const bool in = s + q < blocks;
#pragma unroll
    for (int j = 0; j < MF; ++j) cur[j] = in ? nx[j] * nw : 0.0f;
  };

  f32x4 acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const int off0 = r * 128 + 16 * (q ^ (r & 7)), off1 = r * 128 + 16 * ((4 + q) ^ (r & 7));
  auto frag = [&](const uint8_t* p) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(p + off0);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(p + off1);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto fa = [&](const uint8_t* buf, int i) { return frag(buf + (wn * NF + i) * 2048); };
  auto fb = [&](const uint8_t* buf, int j) { return frag(buf + (TN / 16 + wm * MF + j) * 2048); };

  // The columns of tiles are taken kHeld at a time, so that their operands stay widened in
  // registers (the largest tiles go over their rows twice). Rows of a step: NF for each such
  // part. w: the weights' operands of rows i .. i + kAhead, widened as they are multiplied.
  constexpr int kHeld = NF * MF >= 32 ? MF / 2 : MF, kRows = NF * (MF / kHeld);
  constexpr int kAhead = NF * MF >= 24 ? 1 : 2, kRing = kAhead == 1 ? 2 : 4;
  static_assert(NF % kRing == 0, "the ring starts over with a step");
  i32x8 braw[kHeld], w[kRing];
  f32x4 p[kHeld];  // block products of a row of tiles
  float sc[MF];    // the step's scales
#pragma unroll
  for (int j = 0; j < kHeld; ++j) p[j] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < MF; ++j) sc[j] = 0.0f;
  // to the sums of row i of a step, what p has for its tile j
  auto add = [&](int i, int j) __attribute__((always_inline)) {
    const int at = i / NF * kHeld + j;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      acc[i % NF][at][v] = __builtin_fmaf(sc[at], p[j][v], acc[i % NF][at][v]);
  };
  int s = 0;
  // step s out of `here`; phase: its place among the 4 whose scales are in cur. False
  // after the last. The order of instructions is fixed: the products of a row of tiles,
  // with the sums of the row before.
  auto step = [&](auto phase, uint8_t* before, uint8_t* here, const uint8_t* next)
                  __attribute__((always_inline)) {
    if constexpr (phase() == 0) {
      take(s);
      scales(s + 4);
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) add(kRows - 1, j);  // of the step before
#pragma unroll
    for (int j = 0; j < MF; ++j) sc[j] = from_lane(cur[j], 16 * phase() + r);
    Frag b[kHeld];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i == kRows - kAhead) {
        tile_barrier(vm_lds((S - 2) * kCopies));  // the next step's copies have arrived
      }
      // a share of the copies for the step S on, into the buffer that this step, and
      // before the barrier the one before, has read
      const int at = i + kAhead < kRows ? i + kAhead : i + kAhead - kRows;
      if (i < kRows - kAhead)
        copy(before, s - 1 + S, at * kCopies / kRows, (at + 1) * kCopies / kRows);
      else
        copy(here, s + S, at * kCopies / kRows, (at + 1) * kCopies / kRows);
      w[at % kRing] = i + kAhead < kRows ? fa(here, at % NF) : fa(next, at);
      if (i % NF == 0) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) b[j] = Frag(braw[j]);
      }
      const Frag wide(w[i % kRing]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
          if (h == 0 && i > 0) add(i - 1, j);
          p[j] = quarter(wide, b[j], h, h ? p[j] : f32x4{0, 0, 0, 0});
          if (h == 3 && i % NF == NF - 1)
            braw[j] = i < kRows - 1 ? fb(here, (i / NF + 1) * kHeld + j) : fb(next, j);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
    return ++s < blocks;
  };
  scales(0);
  copy(buf0, 0, 0, kCopies);
  if constexpr (S > 2) copy(buf1, 1, 0, kCopies);
  // the first step brings the others
  copy(S > 2 ? buf2 : buf1, S - 1, 0, kAhead * kCopies / kRows);
  tile_barrier(vm_lds((S - 2) * kCopies + kAhead * kCopies / kRows));
#pragma unroll
  for (int j = 0; j < kHeld; ++j) braw[j] = fb(buf0, j);
  w[0] = fa(buf0, 0);
  if constexpr (kAhead > 1) w[1] = fa(buf0, 1);
  constexpr std::integral_constant<int, 0> p0;
  constexpr std::integral_constant<int, 1> p1;
  constexpr std::integral_constant<int, 2> p2;
  constexpr std::integral_constant<int, 3> p3;
  if constexpr (S == 2) {
    while (step(p0, buf1, buf0, buf1) && step(p1, buf0, buf1, buf0) &&
           step(p2, buf1, buf0, buf1) && step(p3, buf0, buf1, buf0)) {
    }
  } else {
    while (step(p0, buf2, buf0, buf1) && step(p1, buf0, buf1, buf2) &&
           step(p2, buf1, buf2, buf0) && step(p3, buf2, buf0, buf1) &&
           step(p0, buf0, buf1, buf2) && step(p1, buf1, buf2, buf0) &&
           step(p2, buf2, buf0, buf1) && step(p3, buf0, buf1, buf2) &&
           step(p0, buf1, buf2, buf0) && step(p1, buf2, buf0, buf1) &&
           step(p2, buf0, buf1, buf2) && step(p3, buf1, buf2, buf0)) {
    }
  }
  __builtin_amdgcn_s_waitcnt(vm_lds(0));  // no copy outlives the workgroup's LDS
#pragma unroll
  for (int j = 0; j < kHeld; ++j) add(kRows - 1, j);
  with_output<16>(a, [&](auto type, auto vec) {
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int m = m0 + (wm * MF + j) * 16 + r;
      if (m >= M) continue;
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        const int n = n0 + (wn * NF + i) * 16 + 4 * q;
        if (n >= N) continue;
        const float y[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        store4<type(), vec()>(a, m, n, y);
      }
    }
  });
}

template <int TN, int TM, int S>
hipError_t go_big(const F8Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + TN - 1) / TN, tiles = (int64_t)((a.M + TM - 1) / TM) * tiles_n;
  hipLaunchKernelGGL((gemm_f8_big<TN, TM, S>),
                     dim3((unsigned)((tiles + kXcds - 1) / kXcds * kXcds)), dim3(512), 0, stream, a,
                     (int)tiles_n);
  return hipGetLastError();
}

template <int TN, int TM, int WN, int WM, int S, bool GU, bool W32>
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
  hipLaunchKernelGGL((gemm_f8_tile<TN, TM, WN, WM, S, GU, W32>), dim3(grid),
                     dim3(64 * WN * WM), lds, stream, a, (int)tiles_n);
  return hipGetLastError();
}

}  // namespace

// The finest tiles any of the kernels takes for a large call (small ones are few), times
// its threads.
bool gemm_f8_fits(const F8Args& a) {
  const int64_t limit = ((int64_t)1 << 32) - 512 * kXcds;
  if (a.slots) {
    const int64_t cap = a.n_rows < a.M ? a.n_rows : a.M;
    return (cap + a.M / 64) * ((a.N + 63) / 64) * 512 < limit;
  }
  return ((a.M + 63) / 64) * (int64_t)((a.N + 31) / 32) * 256 < limit;
}

hipError_t launch_gemm_f8(const F8Args& a, hipStream_t s) {
  // All times here: us, calls in a row by events. Small tiles and a buffer more where experts
  // have few rows, the FFN, 128 x 64 / 64 x 32: 384 experts, H 4096, I 2880, 1 token 70 / 53, 16
  // 592 / 518, 256 (4 rows each) 2608 / 2292, 1024 (16) 2778 / 2642, 1536 (24) 2858 / 2897, 2048
  // (32) 2931 / 3461, 4096 (64) 3998 / 5088; 32 experts, H 2048, I 1408, 12 rows each 74 / 67, 24
  // 79 / 70, 32 81 / 82; 8 experts, H 4096, I 2880, 24 rows 79 / 65, 48 83 / 101. M counts the
  // picks of both banks of a step, so that a bank with a small share is taken for a fuller one:
  // 89 rows with 230 of 24576 slots 671 / 656, 720 slots 681 / 708.
  if (a.slots) {
    const int64_t cap = a.n_rows < a.M ? a.n_rows : a.M;
    const bool few = a.M <= 24 * cap;
    if (a.gate_up)
      return few ? go<64, 32, 2, 2, 4, true, true>(a, s) : go<128, 64, 2, 2, 3, true, true>(a, s);
    return few ? go<64, 32, 2, 2, 4, false, false>(a, s) : go<128, 64, 2, 2, 3, false, false>(a, s);
  }
  const int64_t cus = device_cus();
  auto tiles = [&](int tn, int tm) {
    return (int64_t)((a.N + tn - 1) / tn) * ((a.M + tm - 1) / tm);
  };
  const bool wide = a.dtype == MOE_DTYPE_F32;
  // Wide tiles where they fill the card, or where small ones, twice as many, would start a
  // second round over the CUs with a long sum, wide / small: 1024 x 4096 x 4096 40 / 47, 640 x
  // 4096 x 4096 (160 tiles) 38 / 43, 512 x 4096 x 4096 (128 tiles) 37 / 30, 1030 x 2047 x 4096
  // (144) 40 / 43, x 2064 26 / 28, x 1040 18 / 18. Of them the one whose rounds over the CUs
  // cost least; a round's cost is its time per step, 3.6, 2.6, 1.9 and 1.15 us (4096 x 5760 x
  // 4096: 238, 171, 184, 217 us; 4096 x 4096 x 2880: 98, 122, 96, 113; 8192 x 8192 x 8192: 890,
  // 924, 926, 1082; 8192 x 1024 x 4096: 116, 84, 64, 77). 32-bit outputs have no such kernel:
  // 4096 x 5760 x 4096 252.
  const int64_t small = tiles(128, 128);
  if (!wide && a.lda <= 1 << 22 && (small >= cus || (2 * small > cus && a.K >= 2048))) {
    auto cost = [&](int tn, int tm, int us) { return (tiles(tn, tm) + cus - 1) / cus * us; };
    const int64_t c[4] = {cost(256, 256, 360), cost(256, 192, 260), cost(256, 128, 190),
                          cost(128, 128, 115)};
    const int64_t least = std::min(std::min(c[0], c[1]), std::min(c[2], c[3]));
    if (least == c[0]) return go_big<256, 256, 2>(a, s);
    if (least == c[1]) return go_big<256, 192, 2>(a, s);
    if (least == c[2]) return go_big<256, 128, 3>(a, s);
    return go_big<128, 128, 3>(a, s);
  }
  // Tiles of 64 rows / 32, 5760 x 4096: 1 row 13.8 / 11.3, 32 15.0 / 11.4, 33 15.2 / 16.0
  if (a.M <= 32)
    return wide ? go<32, 32, 2, 2, 4, false, true>(a, s) : go<32, 32, 2, 2, 4, false, false>(a, s);
  if (tiles(128, 64) >= cus)
    return wide ? go<128, 64, 2, 2, 3, false, true>(a, s) : go<128, 64, 2, 2, 3, false, false>(a, s);
  if (tiles(64, 64) >= cus)
    return wide ? go<64, 64, 2, 2, 3, false, true>(a, s) : go<64, 64, 2, 2, 3, false, false>(a, s);
  return wide ? go<32, 64, 2, 2, 4, false, true>(a, s) : go<32, 64, 2, 2, 4, false, false>(a, s);
}

}  // namespace moe
