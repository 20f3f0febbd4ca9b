// Products of 8-bit rows with a scale per activation row and per weight row, in
// tiles: the grouped products of the expert FFN, and dense ones but for those of
// gemm_i8_use_stream.
//
//   y[r][n] = sa[r] * sw[n] * sum_k a[r][k] w[n][k]
//
// v_mfma_i32_16x16x64_i8 with the weights as A operand (result rows) and the
// activations as B operand (result columns), so that a lane ends with 4
// consecutive outputs of one activation row. The integer sums are exact, so no
// tile shape, split or order changes a bit of the result; the epilogue scales
// in fp32 and rounds once.
//
// Both operands are K-contiguous rows. A step takes 128 bytes of each row of the
// tile: global-to-LDS copies of 16 bytes per lane, a wavefront's copy covering 8
// rows x one whole line, into one of S static buffers (distinct objects, named
// at compile time, so that the compiler need not wait for the copies into one
// before reading another), S - 1 steps ahead, with one barrier per step.
// Granule g of row r lies at g ^ (r & 7) (applied to the source address, as the
// copy writes LDS in lane order), which spreads an operand read over all banks.
// Granules past the end of K are copied from 16 zero bytes instead.
//
// Grouped steps (4096 tokens of top-6 over 384 experts, H 4096, I 2880): gate/up
// 2.11 ms for 9.06 GB of weights, down 1.26 ms for 4.53 GB. The copies bound
// them: without the products 2.12 and 1.24 ms, with every weight from one
// expert, so on chip, 1.46 and 0.86, without the activations' copies 1.98 and
// 1.13. Two or three buffers and two or three workgroups per CU are equal; one
// workgroup with four buffers takes 2.5 ms; tiles of 32 slots 2.5, of 128 slots
// 2.18, of 256 weight rows 2.6; weights straight into registers, six steps
// ahead, 2.6. At 16 tokens (65-73 experts, bound by HBM reads) 276 and 148 us, 6.0
// and 5.6 TB/s.
#include "gemm_i8.h"
#include "mxfp4_common.h"
#include "tile_items.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// TN x TM tile (weight rows x activation rows), WN x WM wavefronts, S buffers.
template <int TN, int TM, int WN, int WM, int S, bool GU>
__global__ __launch_bounds__(64 * WN * WM, WN * WM / 2) void gemm_i8_tile(I8Args a, int tiles_n) {
  constexpr int kW = WN * WM, kRows = TN + TM, kCopies = kRows / 8 / kW;
  static_assert(kRows % (8 * kW) == 0 && TN % (8 * kW) == 0 && (S == 3 || S == 4),
                "whole copies per wavefront");
  constexpr int NF = TN / WN / 16, MF = TM / WM / 16;  // MFMA tiles per wavefront
  static_assert(!GU || NF % 2 == 0, "gate and up tiles in pairs");
  __shared__ __align__(128) uint8_t buf0[kRows * 128];
  __shared__ __align__(128) uint8_t buf1[kRows * 128];
  __shared__ __align__(128) uint8_t buf2[kRows * 128];
  __shared__ __align__(128) uint8_t buf3[S > 3 ? kRows * 128 : 16];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K;

  // which tile: [m0, m1) of the group's slots, weight rows from n0
  int m0, m1, n0;
  const int8_t* w = a.w;
  const float* sw = a.sw;
  const int wrows = GU ? 2 * N : N;
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
    w += row * wrows * (int64_t)K;
    sw += row * wrows;
  } else {
    const int item = xcd_item((a.M + TM - 1) / TM * tiles_n);
    if (item < 0) return;
    const int mt = item / tiles_n, nb = item - mt * tiles_n;
    m0 = mt * TM;
    m1 = min(m0 + TM, a.M);
    n0 = nb * TN;
  }
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
    const int8_t* p = r < TN ? w + (int64_t)wrow(r) * K
                             : a.a + arow(min(m0 + (r - TN), m1 - 1)) * a.lda;
    src[i] = reinterpret_cast<const uint8_t*>(p) + 16 * gran;
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

  i32x4 acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  const int wn = wv % WN, wm = wv / WN, r = lane & 15, q = lane >> 4;
  auto frag = [&](const uint8_t* buf, int row, int half) {
    return *reinterpret_cast<const i32x4*>(buf + row * 128 + 16 * ((4 * half + q) ^ (row & 7)));
  };
  auto compute = [&](const uint8_t* buf) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      i32x4 bf[MF], af[NF];
#pragma unroll
      for (int j = 0; j < MF; ++j) bf[j] = frag(buf, TN + (wm * MF + j) * 16 + r, half);
#pragma unroll
      for (int i = 0; i < NF; ++i) af[i] = frag(buf, (wn * NF + i) * 16 + r, half);
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < MF; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[i], bf[j], acc[i][j], 0, 0, 0);
    }
  };

  const int steps = (K + 127) / 128;
  // past the end of K a copy brings zeros, which the products ignore
  copy(buf0, 0);
  copy(buf1, 128);
  if constexpr (S > 3) copy(buf2, 256);
  for (int s = 0; s < steps; s += S) {
    // each step: its copies (the oldest) have arrived for every wavefront, and
    // the buffer the last step read is free for the copies S - 1 steps ahead
    tile_barrier(vm_lds((S - 2) * kCopies));
    copy(S == 3 ? buf2 : buf3, (s + S - 1) * 128);
    compute(buf0);
    tile_barrier(vm_lds((S - 2) * kCopies));
    copy(buf0, (s + S) * 128);
    compute(buf1);
    tile_barrier(vm_lds((S - 2) * kCopies));
    copy(buf1, (s + S + 1) * 128);
    compute(buf2);
    if constexpr (S > 3) {
      tile_barrier(vm_lds((S - 2) * kCopies));
      copy(buf2, (s + S + 2) * 128);
      compute(buf3);
    }
  }

  __builtin_amdgcn_s_waitcnt(vm_lds(0));  // no copy outlives the workgroup's LDS

  // lane (r, q): outputs 16 i + 4 q + v of activation row 16 j + r
  auto rows = [&](auto f) {
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int m = m0 + (wm * MF + j) * 16 + r;
      if (m >= m1) continue;
      f(j, a.sa[arow(m)], a.slots ? (int64_t)a.slots[m] : (int64_t)m);
    }
  };
  if constexpr (GU) {
    rows([&](int j, float sa, int64_t orow) {
#pragma unroll
      for (int i = 0; i < NF; i += 2) {
        const int n = n0 + (wn * NF + i) * 8 + 4 * q;
        if (n >= N) continue;  // N is a multiple of 64
        const float4 sg = *reinterpret_cast<const float4*>(sw + n);
        const float4 su = *reinterpret_cast<const float4*>(sw + N + n);
        float h[4];
        const float g4[4] = {sg.x, sg.y, sg.z, sg.w}, u4[4] = {su.x, su.y, su.z, su.w};
#pragma unroll
        for (int v = 0; v < 4; ++v)
          h[v] = mx::silu_f32((float)acc[i][j][v] * sa * g4[v]) *
                 ((float)acc[i + 1][j][v] * sa * u4[v]);
        *reinterpret_cast<float4*>(static_cast<float*>(a.y) + orow * a.ldy + n) =
            make_float4(h[0], h[1], h[2], h[3]);
      }
    });
  } else {
    with_output(a, [&](auto type, auto vec) {
      rows([&](int j, float sa, int64_t orow) {
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          const int n = n0 + (wn * NF + i) * 16 + 4 * q;
          if (n >= N) continue;
          float y[4];
#pragma unroll
          for (int v = 0; v < 4; ++v)
            y[v] = (float)acc[i][j][v] * sa * sw[min(n + v, N - 1)];
          store4<type(), vec()>(a, orow, n, y);
        }
      });
    });
  }
}

// Dense products large enough to fill the card with wide tiles: MFMA-bound, 8
// wavefronts (2 x 4) of TN/2 x TM/4 outputs, S buffers of 128 bytes per row.
// The operands of the next half step are read from LDS, spread between the
// products of this one; the one barrier per step sits between its halves, after
// the last read of the step's buffer, which then takes the copies for the step
// S steps on.
template <int TN, int TM, int S>
__global__ __launch_bounds__(512, 2) void gemm_i8_big(I8Args a, int tiles_n) {
  constexpr int WN = 2, WM = 4, kW = 8;
  constexpr int kRows = TN + TM, kCopies = kRows / 8 / kW;
  static_assert(kRows % (8 * kW) == 0 && (S == 2 || S == 3), "whole copies per wavefront");
  constexpr int NF = TN / WN / 16, MF = TM / WM / 16;
  __shared__ __align__(128) uint8_t buf0[kRows * 128];
  __shared__ __align__(128) uint8_t buf1[kRows * 128];
  __shared__ __align__(128) uint8_t buf2[S > 2 ? kRows * 128 : 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K, M = a.M;
  // items in groups of 8 rows of tiles, column by column, so that an XCD's
  // share is about square and its L2 meets few rows of either operand
  const int tiles_m = (M + TM - 1) / TM;
  const int item = xcd_item(tiles_m * tiles_n);
  if (item < 0) return;
  const int group = item / (8 * tiles_n), local = item - group * 8 * tiles_n;
  const int gm = min(8, tiles_m - 8 * group);
  const int m0 = (8 * group + local % gm) * TM, n0 = local / gm * TN;

  const int gran = (lane & 7) ^ (lane >> 3);
  const uint8_t* src[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int r = 8 * (wv + kW * i) + (lane >> 3);
    const int8_t* p = r < TN ? a.w + (int64_t)min(n0 + r, N - 1) * K
                             : a.a + (int64_t)min(m0 + (r - TN), M - 1) * a.lda;
    src[i] = reinterpret_cast<const uint8_t*>(p) + 16 * gran;
  }
  auto copy = [&](uint8_t* buf, int k0) {
    const bool in = k0 + 16 * gran < K;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const uint8_t* p = in ? src[i] + k0 : kZeros;
      asm volatile("" : "+v"(p));  // a select, not a branch around two copies
      __builtin_amdgcn_global_load_lds(p, buf + 1024 * (wv + kW * i), 16, 0, 0);
    }
  };
  i32x4 acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  const int wn = wv % WN, wm = wv / WN, r = lane & 15, q = lane >> 4;
  struct Frags {
    i32x4 b[MF], a[NF];
  };
  // rows 16 apart keep r & 7, so one swizzled offset per half serves all
  const int off0 = r * 128 + 16 * (q ^ (r & 7)), off1 = r * 128 + 16 * ((4 + q) ^ (r & 7));
  auto read = [&](const uint8_t* buf, int half, Frags& f) {
    const uint8_t* p = buf + (half ? off1 : off0);
#pragma unroll
    for (int j = 0; j < MF; ++j)
      f.b[j] = *reinterpret_cast<const i32x4*>(p + (TN + (wm * MF + j) * 16) * 128);
#pragma unroll
    for (int i = 0; i < NF; ++i)
      f.a[i] = *reinterpret_cast<const i32x4*>(p + (wn * NF + i) * 16 * 128);
  };
  auto mul = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < MF; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
  };
  Frags f0, f1;
  auto spread = [&](bool copies) {
    constexpr int kOps = NF + MF, kMul = NF * MF;
#pragma unroll
    for (int i = 0; i < kOps; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (copies && i < kCopies) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kMul / kOps, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kMul % kOps, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // the step out of `here`, f0 its first half's operands
  auto step = [&](int k0, uint8_t* here, const uint8_t* next) {
    read(here, 1, f1);
    mul(f0);
    spread(false);
    tile_barrier(vm_lds((S - 2) * kCopies));  // the next step's copies have arrived
    copy(here, k0 + 128 * S);
    read(next, 0, f0);
    mul(f1);
    spread(true);
  };
  copy(buf0, 0);
  copy(buf1, 128);
  if constexpr (S > 2) copy(buf2, 256);
  tile_barrier(vm_lds((S - 1) * kCopies));
  read(buf0, 0, f0);
  for (int k0 = 0; k0 < K; k0 += 128 * S) {
    step(k0, buf0, buf1);
    if constexpr (S == 2) {
      step(k0 + 128, buf1, buf0);
    } else {
      step(k0 + 128, buf1, buf2);
      step(k0 + 256, buf2, buf0);
    }
  }
  __builtin_amdgcn_s_waitcnt(vm_lds(0));  // no copy outlives the workgroup's LDS
  float sw[NF][4];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) sw[i][v] = a.sw[min(n0 + (wn * NF + i) * 16 + 4 * q + v, N - 1)];
  with_output(a, [&](auto type, auto vec) {
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int m = m0 + (wm * MF + j) * 16 + r;
      if (m >= M) continue;
      const float sa = a.sa[m];
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        const int n = n0 + (wn * NF + i) * 16 + 4 * q;
        if (n >= N) continue;
        float y[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] = (float)acc[i][j][v] * sa * sw[i][v];
        store4<type(), vec()>(a, m, n, y);
      }
    }
  });
}

template <int TN, int TM, int S>
hipError_t go_big(const I8Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + TN - 1) / TN, tiles = (int64_t)((a.M + TM - 1) / TM) * tiles_n;
  hipLaunchKernelGGL((gemm_i8_big<TN, TM, S>),
                     dim3((unsigned)((tiles + kXcds - 1) / kXcds * kXcds)), dim3(512), 0, stream, a,
                     (int)tiles_n);
  return hipGetLastError();
}

template <int TN, int TM, int WN, int WM, int S, bool GU>
hipError_t go(const I8Args& a, hipStream_t stream) {
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
  hipLaunchKernelGGL((gemm_i8_tile<TN, TM, WN, WM, S, GU>), dim3(grid), dim3(64 * WN * WM), lds,
                     stream, a, (int)tiles_n);
  return hipGetLastError();
}

}  // namespace

// The finest tiles any of the kernels takes for such a call, times its threads.
bool gemm_i8_tile_fits(const I8Args& a) {
  const int64_t limit = ((int64_t)1 << 32) - 512 * kXcds;
  if (a.slots) {
    const int64_t cap = a.n_rows < a.M ? a.n_rows : a.M;
    return (cap + a.M / 64) * ((a.N + 63) / 64) * 512 < limit;
  }
  return ((a.M + 63) / 64) * (int64_t)((a.N + 31) / 32) * 256 < limit;
}

hipError_t launch_gemm_i8_tile(const I8Args& a, hipStream_t s) {
  if (a.gate_up) return go<128, 64, 4, 2, 3, true>(a, s);
  if (a.slots) return go<128, 64, 4, 2, 3, false>(a, s);
  // Wide tiles once they fill the card: the width whose rounds over the CUs cost
  // least (4096 x 5760 x 4096: 192 wide 102 us, 256 wide 119; 4096 x 4096 x 2880:
  // 256 wide 60 us, 128 wide 63, 192 wide 81; 8192 x 8192 x 4096: 261, 312, 308).
  const int cus = device_cus();
  const int64_t tiles_m = (a.M + 255) / 256;
  // Products of at most 64 rows take one row of tiles of 64 (a 128- or 256-row
  // tile of the same width multiplies as many rows of padding: 17 x 65536 x 2880
  // 57.1 us at 256 x 256, 38.5 at 128 x 64; 64 x 16384 x 4096 25.0 us at 128 x 128,
  // 19.9).
  if (a.M > 64 && tiles_m * ((a.N + 255) / 256) >= cus) {
    auto cost = [&](int tn) {
      return (tiles_m * ((a.N + tn - 1) / tn) + cus - 1) / cus * tn;
    };
    const int64_t c256 = cost(256), c192 = cost(192), c128 = cost(128);
    if (c256 <= c192 && c256 <= c128) return go_big<256, 256, 2>(a, s);
    return c192 <= c128 ? go_big<192, 256, 2>(a, s) : go_big<128, 256, 3>(a, s);
  }
  // Smaller ones, us (each with about 6 of launch): 500 x 4096 x 4096 at 128 x
  // 128 with the operands read ahead 19.9, at 128 x 64 23.2, 64 x 64 23.3; 1001 x
  // 2048 x 1040 10.9, 9.7, 10.7; 112 x 4096 x 2880 at 64 x 64 10.7, at 32 x 64 8.3
  // (5, 6 or 8 buffers instead of 4: 8.6, 8.5, 8.8).
  auto tiles = [&](int tn, int tm) {
    return (int64_t)((a.N + tn - 1) / tn) * ((a.M + tm - 1) / tm);
  };
  if (a.M > 64 && a.K >= 2048 && tiles(128, 128) >= cus / 2) return go_big<128, 128, 3>(a, s);
  if (tiles(128, 64) >= cus) return go<128, 64, 4, 2, 3, false>(a, s);
  if (tiles(64, 64) >= cus) return go<64, 64, 2, 2, 3, false>(a, s);
  return go<32, 64, 2, 2, 4, false>(a, s);
}

}  // namespace moe
