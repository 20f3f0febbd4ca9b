// Matrix products grouped by expert, in bf16 or fp16 with fp32 sums, over the rows
// that a step's split gives each expert, and their two gradients:
//
//   forward  y[s][n]    = sum over k of w[e][n][k] x[s][k]     (slots s of expert e)
//   input    dx[s][k]   = sum over n of w[e][n][k] dy[s][n]
//   weights  dw[e][n][k] = sum over the slots s of e of dy[s][n] x[s][k]
//
// One kernel, with two operands of MFMA tiles (v_mfma_f32_16x16x32): A gives the
// result's rows, 4 consecutive ones a lane, so the axis that is contiguous in the
// output (n, k, k); B its columns (slots, slots, n). A step takes 64 elements of the
// sum's axis, 128 bytes of LDS for each row of either operand, by global-to-LDS
// copies of 16 bytes per lane into one of S static buffers, S - 1 steps ahead, one
// barrier per step (as in gemm_i8_tile).
//
// Where an operand is contiguous along the sum (w and x forward, dy for dx) a copy
// brings 8 of its rows and a lane's 8 elements are one 16-byte read. Where it is
// contiguous across the sum (w for dx, x and dy for dw) the buffer holds 64 rows of
// the sum's axis as they lie in memory, and ds_read_b64_tr_b16 turns them: 16 lanes
// that read 4 rows of 16 elements get 4 rows' elements of one column each. Either
// way lane (r, q) has elements 8 q .. 8 q + 7 of a half step's 32, and both layouts
// are swizzled over the banks (by the source address, as a copy writes LDS in lane
// order).
#include "gemm_tile.h"
#include "tile_items.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <int DT>
__device__ __forceinline__ f32x4 mfma(i32x4 a, i32x4 b, f32x4 c) {
  if constexpr (DT == MOE_DTYPE_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint64_t read_turned(const uint8_t* p) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  return __builtin_bit_cast(uint64_t,
                            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p));
}

// An operand of ROWS result rows (or columns) that is contiguous along the sum.
template <int ROWS>
struct Along {
  // copy c of a step (of ROWS / 8): rows 8 c .. + 7, lane l granule l % 8 of row l /
  // 8 from where the swizzle has it
  static __device__ __forceinline__ int row(int c, int lane) { return 8 * c + (lane >> 3); }
  static __device__ __forceinline__ int gran(int, int lane) { return (lane & 7) ^ (lane >> 3); }
  // a lane's 8 elements of half `half` for result row `at` + r
  static __device__ __forceinline__ i32x4 frag(const uint8_t* buf, int at, int half, int r, int q) {
    const int row = at + r;
    return *reinterpret_cast<const i32x4*>(buf + row * 128 + 16 * ((4 * half + q) ^ (row & 7)));
  }
};

// An operand of COLS result rows (or columns) that is contiguous across the sum: 64
// rows of COLS elements.
template <int COLS>
struct Across {
  static constexpr int kGran = COLS / 8;  // granules of a row
  static_assert(COLS == 64 || COLS == 128 || COLS == 256, "whole rows per copy");
  // chunks of 32 bytes are swapped: the 4 rows of a turned read lie in different banks
  static __device__ __forceinline__ int swizzle(int row) {
    return COLS == 64 ? row & 3 : (row & 3) | ((row >> 3 & 1) << 2);
  }
  static __device__ __forceinline__ int row(int c, int lane) {
    return (64 / kGran) * c + lane / kGran;
  }
  static __device__ __forceinline__ int gran(int c, int lane) {
    return (lane % kGran) ^ (2 * swizzle(row(c, lane)));
  }
  static __device__ __forceinline__ i32x4 frag(const uint8_t* buf, int at, int half, int r, int q) {
    const int row = 32 * half + 8 * q + (r >> 2);
    uint64_t v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = read_turned(buf + (row + 4 * i) * (2 * COLS) +
                         32 * ((at / 16) ^ swizzle(row + 4 * i)) + 8 * (r & 3));
    return i32x4{(int)v[0], (int)(v[0] >> 32), (int)v[1], (int)(v[1] >> 32)};
  }
};

enum { kForward, kInput, kWeights };

// TA x TB result tile, WA x WB wavefronts, S buffers.
template <int OP, int DT, int TA, int TB, int WA, int WB, int S>
__global__ __launch_bounds__(64 * WA * WB,
                                  (TA + TB) * 128 * S > 80 << 10 ? WA * WB / 4
                                                                 : WA * WB / 2) void grouped(GroupedArgs a, int tiles_a,
                                                                    int tiles_b) {
  constexpr int kW = WA * WB, kRows = TA + TB, kCopies = kRows / 8 / kW, kCopiesA = TA / 8 / kW;
  static_assert(TA % (8 * kW) == 0 && TB % (8 * kW) == 0 && (S == 3 || S == 4),
                "whole copies per wavefront");
  constexpr int NF = TA / WA / 16, MF = TB / WB / 16;  // MFMA tiles per wavefront
  constexpr bool kTurnA = OP != kForward, kTurnB = OP == kWeights;
  using A = std::conditional_t<kTurnA, Across<TA>, Along<TA>>;
  using B = std::conditional_t<kTurnB, Across<TB>, Along<TB>>;
  __shared__ __align__(128) uint8_t buf0[kRows * 128];
  __shared__ __align__(128) uint8_t buf1[kRows * 128];
  __shared__ __align__(128) uint8_t buf2[kRows * 128];
  __shared__ __align__(128) uint8_t buf3[S > 3 ? kRows * 128 : 16];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K;
  const int wn = wv % WA, wm = wv / WA, r = lane & 15, q = lane >> 4;

  // the tile: result rows of A from a0 (of na_), of B from b0, of expert `row`; its
  // slots [m0, m1), all of the expert's (kWeights) or those of the tile
  int a0, b0 = 0, m0, m1;
  int64_t row;
  if constexpr (OP == kWeights) {
    const int per = tiles_a * tiles_b;
    const int item = xcd_item(a.n_rows * per);
    if (item < 0) return;
    const int e = item / per, local = item - e * per;
    const int active = a.n_active ? *a.n_active : 0;
    a0 = local % tiles_a * TA;
    b0 = local / tiles_a * TB;
    if (e < active) {
      m0 = a.row_off[e];
      m1 = a.row_off[e + 1];
      row = a.active_rows[e];
    } else {
      // the (e - active)-th row of the bank that has no slot: its gradient is zero
      __shared__ uint32_t seen[MOE_MAX_ROWS / 32];
      for (int i = tid; i < MOE_MAX_ROWS / 32; i += 64 * kW) seen[i] = 0;
      __syncthreads();
      for (int i = tid; i < active; i += 64 * kW)
        atomicOr(&seen[a.active_rows[i] >> 5], 1u << (a.active_rows[i] & 31));
      __syncthreads();
      int left = e - active, word = 0;
      uint32_t free = ~seen[0];
      while (left >= __popc(free)) {
        left -= __popc(free);
        free = ~seen[++word];
      }
      for (; left > 0; --left) free &= free - 1;
      row = 32 * word + __ffs(free) - 1;
      m0 = m1 = 0;
    }
  } else {
    extern __shared__ int tpre[];  // [n_active + 1]
    __shared__ int wsum[kW];
    const int active = *a.n_active;
    tiles::build_tile_prefix<TB, kW>(a.row_off, active, tpre, wsum);
    const int item = xcd_item(tpre[active] * tiles_a);
    if (item < 0) return;  // the whole workgroup
    // items of one expert: weight rows outermost, so that its tiles meet a block of
    // weights together
    const int e = tiles::row_of_tile(tpre, active, item / tiles_a);
    const int local = item - tpre[e] * tiles_a, nt = tpre[e + 1] - tpre[e];
    a0 = local / nt * TA;
    m0 = a.row_off[e] + (local - local / nt * nt) * TB;
    m1 = min(m0 + TB, a.row_off[e + 1]);
    row = a.active_rows[e];
  }
  const int width = OP == kForward ? N : K;                              // of A's rows
  const int sum = OP == kForward ? K : OP == kInput ? N : m1 - m0;      // length of the sum
  const uint8_t* w = OP == kWeights ? nullptr : a.w + row * N * (int64_t)K * 2;

  // copies: wavefront wv takes copies wv + kW i of each operand. Per copy, where its
  // granule lies at element 0 of the sum (Along) or in row 0 (Across), and which byte
  // of the sum's axis (Along) or row (Across) it is in a step
  constexpr int kCopiesB = kCopies - kCopiesA;
  const uint8_t *sa[kCopiesA], *sb[kCopiesB];
  int fa[kCopiesA], fb[kCopiesB];
  bool ina[kCopiesA], inb[kCopiesB];  // Across: the granule lies inside the row
#pragma unroll
  for (int i = 0; i < kCopiesA; ++i) {
    const int c = wv + kW * i;
    if constexpr (OP == kForward) {
      sa[i] = w + (int64_t)min(a0 + A::row(c, lane), N - 1) * K * 2 + 16 * A::gran(c, lane);
      fa[i] = 16 * A::gran(c, lane);
    } else {
      const int col = a0 + 8 * A::gran(c, lane);
      sa[i] = (OP == kInput ? w : a.x) + col * 2;
      fa[i] = A::row(c, lane);
      ina[i] = col < K;
    }
  }
#pragma unroll
  for (int i = 0; i < kCopiesB; ++i) {
    const int c = wv + kW * i;
    if constexpr (OP == kWeights) {
      const int col = b0 + 8 * B::gran(c, lane);
      sb[i] = a.dy + col * 2;
      fb[i] = B::row(c, lane);
      inb[i] = col < N;
    } else {
      const int s = a.slots[min(m0 + B::row(c, lane), m1 - 1)];
      const int64_t at = OP == kForward && a.by_token ? s / a.k : s;
      sb[i] = (OP == kForward ? a.x + at * K * 2 : a.dy + at * N * 2) + 16 * B::gran(c, lane);
      fb[i] = 16 * B::gran(c, lane);
    }
  }
  auto copy1 = [&](uint8_t* buf, const uint8_t* p) {
    asm volatile("" : "+v"(p));  // a select, not a branch around two copies
    __builtin_amdgcn_global_load_lds(p, buf, 16, 0, 0);
  };
  auto copy = [&](uint8_t* buf, int step) {
#pragma unroll
    for (int i = 0; i < kCopiesA; ++i) {
      const int at = step * (kTurnA ? 64 : 128) + fa[i];
      const uint8_t* p;
      if constexpr (OP == kForward) {
        p = at < 2 * sum ? sa[i] + step * 128 : kZeros;
      } else {
        int from = at;  // row of w, or of x
        if constexpr (OP == kWeights) {
          from = a.slots[m0 + (at < sum ? at : 0)];
          if (a.by_token) from /= a.k;
        }
        p = at < sum && ina[i] ? sa[i] + (int64_t)from * K * 2 : kZeros;
      }
      copy1(buf + 1024 * (wv + kW * i), p);
    }
#pragma unroll
    for (int i = 0; i < kCopiesB; ++i) {
      const int at = step * (kTurnB ? 64 : 128) + fb[i];
      const uint8_t* p;
      if constexpr (OP == kWeights) {
        const int64_t from = a.slots[m0 + (at < sum ? at : 0)];
        p = at < sum && inb[i] ? sb[i] + from * N * 2 : kZeros;
      } else {
        p = at < 2 * sum ? sb[i] + step * 128 : kZeros;
      }
      copy1(buf + TA * 128 + 1024 * (wv + kW * i), p);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  f32x4 acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  auto compute = [&](const uint8_t* buf) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      i32x4 bf[MF], af[NF];
#pragma unroll
      for (int j = 0; j < MF; ++j) bf[j] = B::frag(buf + TA * 128, (wm * MF + j) * 16, half, r, q);
#pragma unroll
      for (int i = 0; i < NF; ++i) af[i] = A::frag(buf, (wn * NF + i) * 16, half, r, q);
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < MF; ++j) acc[i][j] = mfma<DT>(af[i], bf[j], acc[i][j]);
    }
  };

  const int steps = (sum + 63) / 64;
  if (steps > 0) {  // the whole workgroup
    // past the end of the sum a copy brings zeros, which the products ignore
    copy(buf0, 0);
    copy(buf1, 1);
    if constexpr (S > 3) copy(buf2, 2);
    for (int s = 0; s < steps; s += S) {
      // each step: its copies (the oldest) have arrived for every wavefront, and
      // the buffer the last step read is free for the copies S - 1 steps ahead
      tile_barrier(vm_lds((S - 2) * kCopies));
      copy(S == 3 ? buf2 : buf3, s + S - 1);
      compute(buf0);
      tile_barrier(vm_lds((S - 2) * kCopies));
      copy(buf0, s + S);
      compute(buf1);
      tile_barrier(vm_lds((S - 2) * kCopies));
      copy(buf1, s + S + 1);
      compute(buf2);
      if constexpr (S > 3) {
        tile_barrier(vm_lds((S - 2) * kCopies));
        copy(buf2, s + S + 2);
        compute(buf3);
      }
    }
    __builtin_amdgcn_s_waitcnt(vm_lds(0));  // no copy outlives the workgroup's LDS
  }

  // lane (r, q): result rows 16 i + 4 q + v of column 16 j + r
  auto store = [&](auto type) {
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int at = (wm * MF + j) * 16 + r;
      int64_t out;
      if constexpr (OP == kWeights) {
        if (b0 + at >= N) continue;
        out = row * N + b0 + at;
      } else {
        if (m0 + at >= m1) continue;
        out = a.slots[m0 + at];
      }
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        const int n = a0 + (wn * NF + i) * 16 + 4 * q;
        if (n >= width) continue;  // a multiple of 8
        const float y[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        store4<type(), true>(a, out, n, y);
      }
    }
  };
  if (a.dtype == MOE_DTYPE_BF16) store(std::integral_constant<int, MOE_DTYPE_BF16>());
  else if (a.dtype == MOE_DTYPE_F16) store(std::integral_constant<int, MOE_DTYPE_F16>());
  else store(std::integral_constant<int, MOE_DTYPE_F32>());
}

template <int OP, int DT, int TA, int TB, int WA, int WB, int S>
hipError_t go(const GroupedArgs& a, hipStream_t stream) {
  const int64_t tiles_a = ((OP == kForward ? a.N : a.K) + TA - 1) / TA;
  int64_t tiles, tiles_b = 0, lds = 0;
  if (OP == kWeights) {
    tiles_b = (a.N + TB - 1) / TB;
    tiles = a.n_rows * tiles_a * tiles_b;
  } else {
    // at most one part-filled tile per active row
    const int64_t cap = a.n_rows < a.M ? a.n_rows : a.M;
    tiles = (cap + a.M / TB) * tiles_a;
    lds = (cap + 1) * sizeof(int);
  }
  hipLaunchKernelGGL((grouped<OP, DT, TA, TB, WA, WB, S>),
                     dim3((unsigned)((tiles + kXcds - 1) / kXcds * kXcds)), dim3(64 * WA * WB), lds,
                     stream, a, (int)tiles_a, (int)tiles_b);
  return hipGetLastError();
}

template <int DT>
hipError_t pick(const GroupedArgs& a, hipStream_t s) {
  if (a.op == kForward) return go<kForward, DT, 128, 64, 4, 2, 3>(a, s);
  if (a.op == kInput) return go<kInput, DT, 128, 64, 4, 2, 3>(a, s);
  return go<kWeights, DT, 128, 128, 4, 2, 3>(a, s);
}

}  // namespace

// The finest tiles any of the kernels takes for such a call, times its threads.
bool grouped_fits(const GroupedArgs& a) {
  const int64_t limit = ((int64_t)1 << 32) - 512 * kXcds;
  if (a.op == kWeights)
    return (int64_t)((a.N + 63) / 64) * ((a.K + 63) / 64) < limit / 512 / a.n_rows;
  const int64_t cap = a.n_rows < a.M ? a.n_rows : a.M;
  return (cap + a.M / 64) * (((a.op == kForward ? a.N : a.K) + 63) / 64) * 512 < limit;
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t s) {
  return a.elem == MOE_DTYPE_BF16 ? pick<MOE_DTYPE_BF16>(a, s) : pick<MOE_DTYPE_F16>(a, s);
}

}  // namespace moe
