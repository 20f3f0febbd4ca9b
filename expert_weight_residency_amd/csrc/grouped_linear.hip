// Matrix products grouped by expert, in bf16 or fp16 with fp32 sums, over the rows
// that a step's split gives each expert, and their two gradients:
//
//   forward  y[s][n]    = sum over k of w[e][n][k] x[s][k]     (slots s of expert e)
//   input    dx[s][k]   = sum over n of w[e][n][k] dy[s][n]
//   weights  dw[e][n][k] = sum over the slots s of e of dy[s][n] x[s][k]
//
// One kernel (grouped; the others below are forms of it for many rows, short sums and few
// outputs), with two operands of MFMA tiles (v_mfma_f32_16x16x32): A gives the
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
//
// Bounds, at 384 experts of 5760 x 4096, 64 rows each (18.4 GB, 2.87 ms at the read rate):
// 3.76 ms, 4.9 TB/s. Few rows: the weights' bytes; one token's 6 experts of 4096 x 2880 25
// us (5.7 TB/s). Many rows (64 experts, 2880 x 4096, 384 rows: 580 GFLOP, 391 us at the rate
// of a large library product): forward 800 us, input 700, weights 1190 (3.0 GB written;
// 1078 with the operands in the caches). Of the CUs' busy cycles the matrix cores are busy for
// 0.47, 0.49 and 0.25, operand reads from LDS for 0.30, 0.19 and 0.14 (no bank conflicts);
// HBM gives 2.5, 2.3 and 0.6 GB. So none of the three is full. The wavefronts wait for 0.45,
// 0.21 and 0.27 of their cycles: forward at the barrier of each step, with one workgroup per CU
// and nothing beside it. With one expert's weights for all 690 and 610 us (forward, input):
// what HBM's latency adds.
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

// Row of x for a slot (at most 2^23): its token, by the multiple of 2^32 / k rounded up,
// off by less than 32 / 2^32 of the slot, or itself.
__device__ __forceinline__ int token(const GroupedArgs& a, int slot) {
  return a.by_token ? (int)__umulhi((uint32_t)slot, a.by_token) : slot;
}

// The value of another lane of the same 16: lane r ^ 8, or 7 - r of the same 8.
constexpr int kRor8 = 0x128, kHalfMirror = 0x141;
template <int CTRL>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
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
  static_assert(COLS == 64 || COLS == 128, "whole rows per copy");
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

// The slots of a long group, for the weights' gradient: a ring of two halves of
// kHalf slots (x row and dy row of each), one read while the other is filled.
constexpr int kHalf = 256;
struct SlotRing {
  int x[2 * kHalf], dy[2 * kHalf];
};
struct NoRing {};

// The result tile of a workgroup and where its operands come from.
template <int OP, int TA, int TB, int kW>
struct Tile {
  static constexpr bool kTurnA = OP != kForward, kTurnB = OP == kWeights;
  using A = std::conditional_t<kTurnA, Across<TA>, Along<TA>>;
  using B = std::conditional_t<kTurnB, Across<TB>, Along<TB>>;
  using Ring = std::conditional_t<OP == kWeights, SlotRing, NoRing>;
  static constexpr int kCopiesA = TA / 8 / kW, kCopiesB = TB / 8 / kW;
  static constexpr int kCopies = kCopiesA + kCopiesB;
  static_assert(TA % (8 * kW) == 0 && TB % (8 * kW) == 0, "whole copies per wavefront");

  int a0, b0, m0, m1;  // first result row and column; slots of the tile, or of the group
  int sum, steps;      // length of the sum, 64-element steps of it
  int64_t row;         // of the bank
  // Along: where each copy's granule lies at element 0 of the sum. Across: where it
  // lies in row 0 (the same in all copies of a wavefront: rows that they are apart
  // swizzle alike), and whether inside the row
  const uint8_t *sa[kTurnA ? 1 : kCopiesA], *sb[kTurnB ? 1 : kCopiesB];
  bool ina, inb;

  // false: no tile is left for this workgroup
  __device__ __forceinline__ bool init(const GroupedArgs& a, int tiles_a, int tiles_b, int* tpre,
                                       int* wsum, uint32_t* seen) {
    const int tid = threadIdx.x;
    if constexpr (OP == kWeights) {
      const int per = tiles_a * tiles_b;
      const int item = xcd_item(a.n_rows * per);
      if (item < 0) return false;
      const int e = item / per, local = item - e * per;
      // in groups of 6 columns of tiles, row by row: the tiles that an XCD runs at one time
      // are about a square, whose rows its L2 holds (64 experts, 2880 x 4096, 384 rows,
      // operands not in the caches: 1195 us, by all 16 columns 1265; by 8 1210)
      constexpr int kGroup = 6;
      const int group = local / (kGroup * tiles_b), rest = local - group * kGroup * tiles_b;
      const int wide = min(kGroup, tiles_a - kGroup * group);
      a0 = (kGroup * group + rest % wide) * TA;
      b0 = rest / wide * TB;
      // asked for at once with their count: entries past it are not used
      const int at = min(e, min(a.n_rows, a.M) - 1);
      const int active = a.n_active ? *a.n_active : 0;
      m0 = a.n_active ? a.row_off[at] : 0;
      m1 = a.n_active ? a.row_off[at + 1] : 0;
      row = a.n_active ? a.active_rows[at] : 0;
      if (e >= active) {
        // the (e - active)-th row of the bank that has no slot: its gradient is zero
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
      const int active = *a.n_active;
      tiles::build_tile_prefix<TB, kW>(a.row_off, active, tpre, wsum);
      const int item = xcd_item(tpre[active] * tiles_a);
      if (item < 0) return false;
      // items of one expert: weight rows outermost, so that its tiles meet a block of
      // weights together
      const int e = tiles::row_of_tile(tpre, active, item / tiles_a);
      const int local = item - tpre[e] * tiles_a, nt = tpre[e + 1] - tpre[e];
      a0 = local / nt * TA;
      b0 = 0;
      m0 = a.row_off[e] + (local - local / nt * nt) * TB;
      m1 = min(m0 + TB, a.row_off[e + 1]);
      row = a.active_rows[e];
    }
    sum = OP == kForward ? a.K : OP == kInput ? a.N : m1 - m0;
    steps = (sum + 63) / 64;
    return true;
  }

  __device__ __forceinline__ void sources(const GroupedArgs& a) {
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int N = a.N, K = a.K;
    const uint8_t* w = OP == kWeights ? nullptr : a.w + row * N * (int64_t)K * 2;
    if constexpr (kTurnA) {
      const int col = a0 + 8 * A::gran(wv, lane);
      sa[0] = (OP == kInput ? w : a.x) + col * 2;
      ina = col < K;
    } else {
#pragma unroll
      for (int i = 0; i < kCopiesA; ++i)
        sa[i] = w + (int64_t)min(a0 + A::row(wv + kW * i, lane), N - 1) * K * 2 +
                16 * A::gran(0, lane);
    }
    if constexpr (kTurnB) {
      const int col = b0 + 8 * B::gran(wv, lane);
      sb[0] = a.dy + col * 2;
      inb = col < N;
    } else {
#pragma unroll
      for (int i = 0; i < kCopiesB; ++i) {
        const int s = a.slots[min(m0 + B::row(wv + kW * i, lane), m1 - 1)];
        const int64_t at = OP == kForward ? token(a, s) : s;
        sb[i] = (OP == kForward ? a.x + at * K * 2 : a.dy + at * N * 2) + 16 * B::gran(0, lane);
      }
    }
  }

  // Half h of the ring: each thread's share of its slots, asked for and then kept.
  struct Slots {
    int v[(kHalf + 64 * kW - 1) / (64 * kW)];
  };
  __device__ __forceinline__ Slots ask(const GroupedArgs& a, int h) const {
    Slots s;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(s.v) / 4); ++i)
      s.v[i] = a.slots[m0 + min(h * kHalf + (int)threadIdx.x + 64 * kW * i, sum - 1)];
    return s;
  }
  __device__ __forceinline__ void keep(const GroupedArgs& a, Ring& ring, int h,
                                       const Slots& s) const {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(s.v) / 4); ++i) {
      const int at = threadIdx.x + 64 * kW * i;
      if (at < kHalf) {
        ring.dy[(h & 1) * kHalf + at] = s.v[i];
        ring.x[(h & 1) * kHalf + at] = token(a, s.v[i]);
      }
    }
  }

  // The copies of a step into buf, A's rows first; past the end of the sum zeros,
  // which the products ignore.
  __device__ __forceinline__ void copy(const GroupedArgs& a, const Ring& ring, uint8_t* buf,
                                       int step) const {
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint8_t* p[kCopies];
#pragma unroll
    for (int i = 0; i < kCopiesA; ++i) {
      if constexpr (kTurnA) {
        const int at = step * 64 + A::row(wv + kW * i, lane);
        int from = at;
        if constexpr (OP == kWeights) from = ring.x[at & (2 * kHalf - 1)];
        p[i] = at < sum && ina ? sa[0] + (int64_t)from * a.K * 2 : kZeros;
      } else {
        p[i] = step * 128 + 16 * A::gran(0, lane) < 2 * sum ? sa[i] + (int64_t)step * 128 : kZeros;
      }
    }
#pragma unroll
    for (int i = 0; i < kCopiesB; ++i) {
      if constexpr (kTurnB) {
        const int at = step * 64 + B::row(wv + kW * i, lane);
        const int from = ring.dy[at & (2 * kHalf - 1)];
        p[kCopiesA + i] = at < sum && inb ? sb[0] + (int64_t)from * a.N * 2 : kZeros;
      } else {
        p[kCopiesA + i] =
            step * 128 + 16 * B::gran(0, lane) < 2 * sum ? sb[i] + (int64_t)step * 128 : kZeros;
      }
    }
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      copy16(buf + (i < kCopiesA ? 0 : TA * 128) +
                 1024 * (wv + kW * (i < kCopiesA ? i : i - kCopiesA)),
             p[i]);
    }
  }

  // Lane (r, q) of wavefront tile (wn, wm) holds result rows 16 i + 4 q + v of column
  // 16 j + r.
  template <int NF, int MF>
  __device__ __forceinline__ void store(const GroupedArgs& a, const f32x4 (&acc)[NF][MF], int wn,
                                        int wm) const {
    const int r = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
    const int width = OP == kForward ? a.N : a.K;
    auto as = [&](auto type) {
#pragma unroll
      for (int j = 0; j < MF; ++j) {
        const int at = (wm * MF + j) * 16 + r;
        int64_t out;
        if constexpr (OP == kWeights) {
          if (b0 + at >= a.N) continue;
          out = row * a.N + b0 + at;
        } else {
          if (m0 + at >= m1) continue;
          out = a.slots[m0 + at];
        }
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          const int n = a0 + (wn * NF + i) * 16 + 4 * q;
          if (n >= width) continue;  // a multiple of 8
          const f32x4 y = acc[i][j];
          if constexpr (type() == MOE_DTYPE_F32)
            *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + out * a.ldy + n) = y;
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + out * a.ldy + n) =
                make_uint2(pack2<type()>(y[0], y[1]), pack2<type()>(y[2], y[3]));
        }
      }
    };
    if (a.dtype == MOE_DTYPE_BF16) as(std::integral_constant<int, MOE_DTYPE_BF16>());
    else if (a.dtype == MOE_DTYPE_F16) as(std::integral_constant<int, MOE_DTYPE_F16>());
    else as(std::integral_constant<int, MOE_DTYPE_F32>());
  }

  // The weights' gradients, which are many: whole lines with the streaming policy, so
  // that they do not push the operands out of the L2 (64 experts, 2880 x 4096 in 32 bits,
  // 384 rows each: 1318 us with ordinary stores, 1192 so). Lanes trade tiles until a store
  // takes 128 bytes of a row: 64, as the tiles lie, are written at 3.8 TB/s with that
  // policy instead of 6.6. Lanes r and r + 8 swap a tile of each pair; for 16-bit types,
  // whose rows are half as long, lanes r and 7 - r then swap a pair of each two.
  template <int DT, int NF, int MF>
  __device__ __forceinline__ void store_lines(const GroupedArgs& a, const f32x4 (&acc)[NF][MF],
                                              int wn, int wm) const {
    constexpr bool kWide = DT == MOE_DTYPE_F32;
    constexpr int kWords = kWide ? 4 : 2;  // of 4 outputs
    typedef uint32_t words __attribute__((ext_vector_type(kWords)));
    const int r = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
    const bool low = r < 8, left = !(r & 4);
    auto pack = [](const f32x4& v) {
      words w;
      if constexpr (kWide) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
      } else {
        w[0] = pack2<DT>(v[0], v[1]);
        w[1] = pack2<DT>(v[2], v[3]);
      }
      return w;
    };
    // x where mine, else the other lane's y; every lane takes part in the exchange
    auto swap = [](auto ctrl, bool mine, const words& x, const words& y) {
      words w;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t other = from_lane<ctrl()>(y[i]);
        w[i] = mine ? x[i] : other;
      }
      return w;
    };
    auto put = [&](int at, int n, const words& w) {
      if (at < a.N && n < a.K)  // K is a multiple of 8
        __builtin_nontemporal_store(
            w, reinterpret_cast<words*>(static_cast<uint8_t*>(a.y) +
                                        ((row * a.N + at) * a.ldy + n) * (kWide ? 4 : 2)));
    };
    constexpr std::integral_constant<int, kRor8> ror8;
    constexpr std::integral_constant<int, kHalfMirror> mirror;
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int at = b0 + (wm * MF + j) * 16;
#pragma unroll
      for (int i = 0; i < NF; i += kWide ? 2 : 4) {
        words two[2][2];  // [pair][rows r & 7, and 8 on] of tile 2 pair + r / 8
#pragma unroll
        for (int p = 0; p < (kWide ? 1 : 2); ++p) {
          const words x = pack(acc[i + 2 * p][j]), y = pack(acc[i + 2 * p + 1][j]);
          two[p][0] = swap(ror8, low, x, y);
          two[p][1] = swap(ror8, !low, y, x);
        }
        if constexpr (kWide) {
          const int n = a0 + (wn * NF + i + r / 8) * 16 + 4 * q;
          put(at + (r & 7), n, two[0][0]);
          put(at + (r & 7) + 8, n, two[0][1]);
        } else {
          const int n = a0 + (wn * NF + i + (left ? 0 : 2) + r / 8) * 16 + 4 * q;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // rows 0 .. 3, then 4 .. 7 of the 8
            put(at + 8 * h + (left ? r & 3 : 7 - (r & 7)), n,
                swap(mirror, left, two[0][h], two[1][h]));
            put(at + 8 * h + (left ? 7 - (r & 7) : r & 7), n,
                swap(mirror, !left, two[1][h], two[0][h]));
          }
        }
      }
    }
  }
};

// Tiles of the kernels for groups of many rows.
constexpr int kWideA = 256, kWideB = 128;

// TA x TB result tile, WA x WB wavefronts, S buffers.
template <int OP, int DT, int TA, int TB, int WA, int WB, int S>
__global__ __launch_bounds__(64 * WA * WB,
                             (TA + TB) * 128 * S > 80 << 10 ? WA * WB / 4 : WA * WB / 2)
void grouped(GroupedArgs a, int tiles_a, int tiles_b) {
  constexpr int kW = WA * WB, kRows = TA + TB;
  constexpr int NF = TA / WA / 16, MF = TB / WB / 16;  // MFMA tiles per wavefront
  using T = Tile<OP, TA, TB, kW>;
  __shared__ __align__(128) uint8_t buf0[kRows * 128];
  __shared__ __align__(128) uint8_t buf1[kRows * 128];
  __shared__ __align__(128) uint8_t buf2[kRows * 128];
  __shared__ __align__(128) uint8_t buf3[S > 3 ? kRows * 128 : 16];
  __shared__ __align__(128) uint8_t buf4[S > 3 ? kRows * 128 : 16];
  __shared__ __align__(128) uint8_t buf5[S > 3 ? kRows * 128 : 16];
  static_assert(S == 3 || S == 6, "buffers");
  __shared__ typename T::Ring ring;
  __shared__ uint32_t seen[OP == kWeights ? MOE_MAX_ROWS / 32 : 1];
  __shared__ int wsum[kW];
  extern __shared__ int tpre[];  // [n_active + 1]

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wv % WA, wm = wv / WA, r = lane & 15, q = lane >> 4;
  T t;
  if (!t.init(a, tiles_a, tiles_b, tpre, wsum, seen)) return;  // the whole workgroup
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
      for (int j = 0; j < MF; ++j)
        bf[j] = T::B::frag(buf + TA * 128, (wm * MF + j) * 16, half, r, q);
#pragma unroll
      for (int i = 0; i < NF; ++i) af[i] = T::A::frag(buf, (wn * NF + i) * 16, half, r, q);
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < MF; ++j) acc[i][j] = mfma<DT>(af[i], bf[j], acc[i][j]);
    }
  };

  if (t.steps > 0) {  // the whole workgroup
    t.sources(a);
    typename T::Slots slots;
    if constexpr (OP == kWeights) {
      const typename T::Slots first = t.ask(a, 0), second = t.ask(a, 1);
      t.keep(a, ring, 0, first);
      t.keep(a, ring, 1, second);
      __syncthreads();
    }
    // the copies of step s; where they are the first of a half of the ring, the other
    // half is free for the slots after it, which arrive a step later
    auto copy = [&](uint8_t* buf, int s) {
      t.copy(a, ring, buf, s);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (OP == kWeights) {
        if (s >= kHalf / 64 && s < t.steps) {
          if ((s & (kHalf / 64 - 1)) == 0) slots = t.ask(a, s / (kHalf / 64) + 1);
          if ((s & (kHalf / 64 - 1)) == 1) t.keep(a, ring, s / (kHalf / 64) + 1, slots);
        }
      }
    };
    int s = 0;
    // each step: its copies (the oldest) have arrived for every wavefront, and the
    // buffer the last step read is free for the copies S - 1 steps ahead. False after
    // the last
    auto step = [&](const uint8_t* here, uint8_t* before) __attribute__((always_inline)) {
      tile_barrier(vm_lds((S - 2) * T::kCopies));
      copy(before, s + S - 1);
      compute(here);
      return ++s < t.steps;
    };
    copy(buf0, 0);
    copy(buf1, 1);
    if constexpr (S == 3) {
      while (step(buf0, buf2) && step(buf1, buf0) && step(buf2, buf1)) {
      }
    } else {
      copy(buf2, 2);
      copy(buf3, 3);
      copy(buf4, 4);
      while (step(buf0, buf5) && step(buf1, buf0) && step(buf2, buf1) && step(buf3, buf2) &&
             step(buf4, buf3) && step(buf5, buf4)) {
      }
    }
    __builtin_amdgcn_s_waitcnt(vm_lds(0));  // no copy outlives the workgroup's LDS
  }
  t.store(a, acc, wn, wm);
}

// Operands in steps of 32 elements, for the wide tiles. Along: rows of 64 bytes, 16 to a
// copy, swizzled as above.
template <int ROWS>
struct Along32 {
  static constexpr int kBytes = ROWS * 64;
  static __device__ __forceinline__ int row(int c, int lane) { return 16 * c + (lane >> 2); }
  static __device__ __forceinline__ int gran(int, int lane) { return (lane & 3) ^ (lane >> 3 & 3); }
  // the operand lies `from` bytes into buf (one sum of offsets: past a few additions to
  // a pointer the compiler no longer tells the buffers apart, and waits for every copy)
  static __device__ __forceinline__ i32x4 frag(const uint8_t* buf, int from, int at, int r, int q) {
    const int row = at + r;
    return *reinterpret_cast<const i32x4*>(buf + (from + row * 64 + 16 * (q ^ (row >> 1 & 3))));
  }
};
// Across: 32 rows of the sum's axis. A copy is followed by 32 bytes that nothing uses,
// and brings rows that no read joins, so that the 8 rows that 32 lanes read at once lie
// in different banks and a lane's addresses are one and constants (swizzled chunks
// would take a register or an operation each). Place p of a row: copy p % kCopies,
// part p / kCopies of it. Lane (r, q) reads rows 8 q + r / 4 + 4 i, i = 0, 1, as the
// operand beside it holds them (PAIRED), or 4 q + r / 4 + 16 i where both are across.
template <int COLS, bool PAIRED>
struct Across32 {
  static constexpr int kGran = COLS / 8, kCopies = COLS / 16, kCopy = 1024 + 32;
  static constexpr int kBytes = kCopies * kCopy;
  static_assert(COLS == 256 || (COLS == 128 && !PAIRED), "places of the rows");
  static __device__ __forceinline__ int row(int c, int lane) {
    const int p = c + kCopies * (lane / kGran);
    return PAIRED ? (p & 19) | (p & 4) << 1 | (p & 8) >> 1 : p;
  }
  static __device__ __forceinline__ int gran(int lane) { return lane % kGran; }
  static __device__ __forceinline__ i32x4 frag(const uint8_t* buf, int from, int at, int r, int q) {
    uint64_t v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // PAIRED: row 8 q + r / 4 + 4 i is in place r / 4 + 4 (q & 1) + 8 i + 16 (q / 2)
      const int p = (r >> 2) + (PAIRED ? 4 * (q & 1) + 8 * i + 16 * (q >> 1) : 4 * q + 16 * i);
      v[i] = read_turned(buf + (from + p % kCopies * kCopy + p / kCopies * (2 * COLS) + 2 * at +
                                8 * (r & 3)));
    }
    return i32x4{(int)v[0], (int)(v[0] >> 32), (int)v[1], (int)(v[1] >> 32)};
  }
};

// The same for groups of many rows, in 256 x 128 tiles. Forward: 8 wavefronts (2 x 4) of
// 128 x 32 outputs, 3 buffers of 64 elements. The weights' operand of two tiles on is read
// from LDS while a row of tiles is multiplied; the one barrier per step sits after the last
// read of the step's buffer. The order of
// instructions is fixed, and copies go out one row of tiles at a time: a step's, asked for
// at once by all wavefronts, hold the products up (as in gemm_f8_big).
template <int DT>
__global__ __launch_bounds__(512, 2) void grouped_forward(GroupedArgs a, int tiles_a) {
  constexpr int TA = kWideA, TB = kWideB, S = 3, WN = 2, NF = TA / WN / 16, MF = TB / 4 / 16, kW = 8;
  using T = Tile<kForward, TA, TB, kW>;
  constexpr int kCopies = T::kCopies;
  __shared__ __align__(128) uint8_t buf0[(TA + TB) * 128];
  __shared__ __align__(128) uint8_t buf1[(TA + TB) * 128];
  __shared__ __align__(128) uint8_t buf2[(TA + TB) * 128];
  __shared__ int wsum[kW];
  extern __shared__ int tpre[];  // [n_active + 1]

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wv % WN, wm = wv / WN, r = lane & 15, q = lane >> 4;
  const int N = a.N, K = a.K;
  T t;
  if (!t.init(a, tiles_a, 1, tpre, wsum, nullptr)) return;  // the whole workgroup

  constexpr uint32_t kOutside = 1u << 31;  // above the bytes of any copy
  const int gran = (lane & 7) ^ (lane >> 3);
  const uint8_t* base = a.w + (t.row * N + t.a0) * K * 2;
  uint32_t offa[T::kCopiesA];
  const uint8_t* src[T::kCopiesB];
#pragma unroll
  for (int i = 0; i < T::kCopiesA; ++i)
    offa[i] = min(8 * (wv + kW * i) + (lane >> 3), N - 1 - t.a0) * K * 2 + 16 * gran;
#pragma unroll
  for (int i = 0; i < T::kCopiesB; ++i) {
    const int slot = a.slots[min(t.m0 + 8 * (wv + kW * i) + (lane >> 3), t.m1 - 1)];
    src[i] = a.x + (int64_t)token(a, slot) * K * 2 + 16 * gran;
  }
  // copies [from, to) of step s's: weights first
  auto copy = [&](uint8_t* buf, int s, int from, int to) __attribute__((always_inline)) {
    const bool in = s * 128 + 16 * gran < 2 * K;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      if (i < from || i >= to) continue;
      if (i < T::kCopiesA)
        copy16(buf + 1024 * (wv + kW * i), base + (int64_t)s * 128, kOutside,
               in ? offa[i < T::kCopiesA ? i : 0] : kOutside);
      else
        copy16(buf + TA * 128 + 1024 * (wv + kW * (i - T::kCopiesA)),
               in ? src[i < T::kCopiesA ? 0 : i - T::kCopiesA] + (int64_t)s * 128 : kZeros);
    }
  };
  f32x4 acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  struct Frag {
    i32x4 half[2];
  };
  const int off0 = r * 128 + 16 * (q ^ (r & 7)), off1 = r * 128 + 16 * ((4 + q) ^ (r & 7));
  auto frag = [&](const uint8_t* p) {
    return Frag{{*reinterpret_cast<const i32x4*>(p + off0),
                 *reinterpret_cast<const i32x4*>(p + off1)}};
  };
  auto fa = [&](const uint8_t* buf, int i) { return frag(buf + (wn * NF + i) * 2048); };
  auto fb = [&](const uint8_t* buf, int j) { return frag(buf + (TA / 16 + wm * MF + j) * 2048); };

  // w: operands i .. i + kAhead
  constexpr int kAhead = 2, kRing = 4;
  static_assert(NF % kRing == 0, "the ring starts over with a step");
  Frag b[MF], w[kRing];
  int s = 0;
  // step s out of `here`. False after the last
  auto step = [&](uint8_t* before, uint8_t* here, const uint8_t* next)
                  __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      if (i == NF - kAhead) tile_barrier(vm_lds((S - 2) * kCopies));  // the next step's arrived
      // a share of the copies for the step S on, into the buffer that this step, and
      // before the barrier the one before, has read
      const int at = i + kAhead < NF ? i + kAhead : i + kAhead - NF;
      if (i < NF - kAhead) copy(before, s - 1 + S, at * kCopies / NF, (at + 1) * kCopies / NF);
      else copy(here, s + S, at * kCopies / NF, (at + 1) * kCopies / NF);
      w[at % kRing] = i + kAhead < NF ? fa(here, at) : fa(next, at);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < MF; ++j) {
          acc[i][j] = mfma<DT>(w[i % kRing].half[h], b[j].half[h], acc[i][j]);
          if (h == 1 && i == NF - 1) b[j] = fb(next, j);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
    return ++s < t.steps;
  };
  copy(buf0, 0, 0, kCopies);
  copy(buf1, 1, 0, kCopies);
  copy(buf2, 2, 0, kAhead * kCopies / NF);  // the first step brings the others
  tile_barrier(vm_lds((S - 2) * kCopies + kAhead * kCopies / NF));
#pragma unroll
  for (int j = 0; j < MF; ++j) b[j] = fb(buf0, j);
  w[0] = fa(buf0, 0);
  w[1] = fa(buf0, 1);
  while (step(buf2, buf0, buf1) && step(buf0, buf1, buf2) && step(buf1, buf2, buf0)) {
  }
  __builtin_amdgcn_s_waitcnt(vm_lds(0));  // no copy outlives the workgroup's LDS
  t.store(a, acc, wn, wm);
}

// The gradients: 4 wavefronts (2 x 2) of 128 x 64 outputs and steps of 32 elements, two
// workgroups per CU, so that one's start and end run beside the other's products. The
// operands of the next step are read from LDS between the products of this one, whose
// buffer then takes the copies for the step 3 steps on; one barrier per step.
template <int OP, int DT>
__global__ __launch_bounds__(256, 2) void grouped_gradient(GroupedArgs a, int tiles_a,
                                                             int tiles_b) {
  constexpr int TA = kWideA, TB = kWideB, NF = 8, MF = 4;
  constexpr int kW = 4;
  using T = Tile<OP, TA, TB, kW>;
  using A = Across32<TA, OP == kInput>;
  using B = std::conditional_t<T::kTurnB, Across32<TB, false>, Along32<TB>>;
  constexpr int kBytesA = A::kBytes, kBytesB = B::kBytes;
  constexpr int kCopiesA = TA / 64, kCopiesB = TB / 64, kCopies = kCopiesA + kCopiesB;
  __shared__ __align__(128) uint8_t buf0[kBytesA + kBytesB];
  __shared__ __align__(128) uint8_t buf1[kBytesA + kBytesB];
  __shared__ __align__(128) uint8_t buf2[kBytesA + kBytesB];
  __shared__ typename T::Ring ring;
  __shared__ uint32_t seen[OP == kWeights ? MOE_MAX_ROWS / 32 : 1];
  __shared__ int wsum[kW];
  extern __shared__ int tpre[];  // [n_active + 1]

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wv & 1, wm = wv >> 1, r = lane & 15, q = lane >> 4;
  const int N = a.N, K = a.K;
  T t;
  if (!t.init(a, tiles_a, tiles_b, tpre, wsum, seen)) return;  // the whole workgroup
  f32x4 acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  if (t.sum > 0) {  // the whole workgroup
    const int steps = (t.sum + 31) / 32;
    constexpr uint32_t kOutside = 1u << 31;  // above the bytes of any copy
    uint32_t offa[kCopiesA];
    const uint8_t *base = nullptr, *sa = nullptr, *sb[kCopiesB];
    bool inb = true;
    const int col = t.a0 + 8 * A::gran(lane);
    const bool ina = col < K;
    if constexpr (OP == kInput) {
      base = a.w + t.row * N * (int64_t)K * 2;
#pragma unroll
      for (int i = 0; i < kCopiesA; ++i)
        offa[i] = ina ? A::row(wv + kW * i, lane) * K * 2 + col * 2 : kOutside;
    } else {
      sa = a.x + col * 2;
    }
    if constexpr (OP == kWeights) {
      const int col = t.b0 + 8 * B::gran(lane);
      sb[0] = a.dy + col * 2;
      inb = col < N;
    } else {
#pragma unroll
      for (int i = 0; i < kCopiesB; ++i) {
        const int s = a.slots[min(t.m0 + B::row(wv + kW * i, lane), t.m1 - 1)];
        sb[i] = a.dy + (int64_t)s * N * 2 + 16 * B::gran(0, lane);
      }
    }
    typename T::Slots slots;
    if constexpr (OP == kWeights) {
      const typename T::Slots first = t.ask(a, 0), second = t.ask(a, 1);
      t.keep(a, ring, 0, first);
      t.keep(a, ring, 1, second);
      __syncthreads();
    }
    // weights: rows of x and dy that a step's copies bring, read a step before
    uint32_t rows[kCopies];
    auto look = [&](int s, int i) __attribute__((always_inline)) {
      if constexpr (OP == kWeights) {
        if (i < kCopiesA) rows[i] = ring.x[(s * 32 + A::row(wv + kW * i, lane)) & (2 * kHalf - 1)];
        else rows[i] = ring.dy[(s * 32 + B::row(wv + kW * (i - kCopiesA), lane)) & (2 * kHalf - 1)];
      }
    };
    // copy i of step s's, A's first; then the rows of the next step's
    auto copy = [&](uint8_t* buf, int s, int i) __attribute__((always_inline)) {
      if (i < kCopiesA) {
        uint8_t* const to = buf + A::kCopy * (wv + kW * i);
        if constexpr (OP == kInput) {
          const int left = min(max(N - 32 * s, 0), 32);
          copy16(to, base + (int64_t)s * 32 * K * 2, (uint32_t)left * K * 2,
                 offa[i < kCopiesA ? i : 0]);
        } else {
          const int at = s * 32 + A::row(wv + kW * i, lane);
          copy16(to, at < t.sum && ina ? sa + (uint64_t)rows[i] * (2u * K) : kZeros);
        }
      } else {
        const int c = wv + kW * (i - kCopiesA);
        if constexpr (OP == kWeights) {
          const int at = s * 32 + B::row(c, lane);
          copy16(buf + kBytesA + B::kCopy * c,
                 at < t.sum && inb ? sb[0] + (uint64_t)rows[i] * (2u * N) : kZeros);
        } else {
          const bool in = s * 64 + 16 * B::gran(0, lane) < 2 * t.sum;
          copy16(buf + kBytesA + 1024 * c,
                 in ? sb[i < kCopiesA ? 0 : i - kCopiesA] + (int64_t)s * 64 : kZeros);
        }
      }
    };
    auto copies = [&](uint8_t* buf, int s) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        copy(buf, s, i);
        look(s + 1, i);
      }
    };
    // where the copies of step s are the first of a half of the ring, the other half is
    // free for the slots after it, which arrive a step later
    auto refill = [&](int s) {
      if constexpr (OP == kWeights) {
        if (s >= kHalf / 32 && s < steps) {
          if ((s & (kHalf / 32 - 1)) == 0) slots = t.ask(a, s / (kHalf / 32) + 1);
          if ((s & (kHalf / 32 - 1)) == 1) t.keep(a, ring, s / (kHalf / 32) + 1, slots);
        }
      }
    };
    struct Frags {
      i32x4 b[MF], a[NF];
    };
    auto reada = [&](const uint8_t* buf, int i) {
      return A::frag(buf, 0, (wn * NF + i) * 16, r, q);
    };
    auto readb = [&](const uint8_t* buf, int j) {
      return B::frag(buf, kBytesA, (wm * MF + j) * 16, r, q);
    };
    Frags f0, f1;
    int s = 0;
    // the step whose operands are in f, out of `here`; the next one's go into g. False
    // after the last. The order of instructions is fixed: with each row of products one
    // copy, and reads of the next step's operands
    auto step = [&](uint8_t* here, const uint8_t* next, const Frags& f, Frags& g)
                    __attribute__((always_inline)) {
      tile_barrier(vm_lds(kCopies));  // the next step's copies have arrived
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        if (i < kCopies) {
          copy(here, s + 3, i);
          look(s + 4, i);
        }
        g.a[i] = reada(next, i);
        if (i % (NF / MF) == 0) g.b[i / (NF / MF)] = readb(next, i / (NF / MF));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < MF; ++j) {
          acc[i][j] = mfma<DT>(f.a[i], f.b[j], acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      refill(s + 3);
      return ++s < steps;
    };
#pragma unroll
    for (int i = 0; i < kCopies; ++i) look(0, i);
    copies(buf0, 0);
    copies(buf1, 1);
    copies(buf2, 2);
    tile_barrier(vm_lds(2 * kCopies));
#pragma unroll
    for (int i = 0; i < NF; ++i) f0.a[i] = reada(buf0, i);
#pragma unroll
    for (int j = 0; j < MF; ++j) f0.b[j] = readb(buf0, j);
    while (step(buf0, buf1, f0, f1) && step(buf1, buf2, f1, f0) && step(buf2, buf0, f0, f1) &&
           step(buf0, buf1, f1, f0) && step(buf1, buf2, f0, f1) && step(buf2, buf0, f1, f0)) {
    }
    __builtin_amdgcn_s_waitcnt(vm_lds(0));  // no copy outlives the workgroup's LDS
  }
  if constexpr (OP == kInput) t.store(a, acc, wn, wm);
  else if (a.dtype == MOE_DTYPE_F32) t.template store_lines<MOE_DTYPE_F32>(a, acc, wn, wm);
  else if (a.dtype == MOE_DTYPE_BF16) t.template store_lines<MOE_DTYPE_BF16>(a, acc, wn, wm);
  else t.template store_lines<MOE_DTYPE_F16>(a, acc, wn, wm);
}

// Forward with a sum of at most 64 elements (an adapter's second product), which is bound
// by its output: no buffers. A wavefront holds the 64 x rows of its tile in registers and
// walks over a quarter of the tile's 1024 weight rows, whose elements go from memory to the
// products as they lie, 64 rows at a time, the next 64 asked for before. A product's row
// 4 q + v is weight row 8 q + v of a pair of tiles' 32 for 16-bit outputs, 4 on in the
// pair's other tile: a lane stores 8 consecutive outputs. N = 4096, us, 256 / 512 / 1024 /
// 2048 weight rows per tile: K 16, 64 experts, 6000 slots 21.5 / 19.7 / 18.2 / 19.2 (49 MB
// written); K 32, 24576 slots 60.6 / 48.9 / 46.9 / 52.1.
constexpr int kShortA = 1024, kShortB = 64, kShortK = 64;
template <int DT, int OUT>
__device__ void short_sums(const GroupedArgs& a, const Tile<kForward, kShortA, kShortB, 4>& t) {
  constexpr bool kPairs = OUT != MOE_DTYPE_F32;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int N = a.N, K = a.K;
  const bool in[2] = {8 * q < K, 32 + 8 * q < K};
  const uint8_t* w = a.w + t.row * N * (int64_t)K * 2 + 16 * q;
  auto load = [&](const uint8_t* p, int half) {
    return *reinterpret_cast<const i32x4*>(in[half] ? p + 64 * half : kZeros);
  };
  i32x4 x[4][2];
  int slot[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int at = t.m0 + 16 * j + r;
    slot[j] = a.slots[min(at, t.m1 - 1)];
    const uint8_t* p = a.x + (int64_t)token(a, slot[j]) * K * 2 + 16 * q;
    for (int h = 0; h < 2; ++h) x[j][h] = load(p, h);
    if (at >= t.m1) slot[j] = -1;
  }
  // weight row of a product's row `m` of tile i
  auto row = [](int i, int m) {
    return kPairs ? i / 2 * 32 + m / 4 * 8 + i % 2 * 4 + m % 4 : 16 * i + m;
  };
  auto block = [&](int n0, i32x4 (&f)[4][2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* p = w + (int64_t)min(n0 + row(i, r), N - 1) * K * 2;
      for (int h = 0; h < 2; ++h) f[i][h] = load(p, h);
    }
  };
  const int end = min(t.a0 + kShortA, N);
  i32x4 next[4][2];
  int n0 = t.a0 + 64 * wv;
  if (n0 < end) block(n0, next);
  for (; n0 < end; n0 += 256) {
    i32x4 f[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      for (int h = 0; h < 2; ++h) f[i][h] = next[i][h];
    if (n0 + 256 < end) block(n0 + 256, next);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x4 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = mfma<DT>(f[i][0], x[j][0], f32x4{0, 0, 0, 0});
        y[i] = mfma<DT>(f[i][1], x[j][1], y[i]);
      }
      if (slot[j] < 0) continue;
      const int64_t out = slot[j] * a.ldy;
      if constexpr (kPairs) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const int n = n0 + row(i, 4 * q);
          if (n < N)  // a multiple of 8
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + out + n) =
                make_uint4(pack2<OUT>(y[i][0], y[i][1]), pack2<OUT>(y[i][2], y[i][3]),
                           pack2<OUT>(y[i + 1][0], y[i + 1][1]),
                           pack2<OUT>(y[i + 1][2], y[i + 1][3]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + row(i, 4 * q);
          if (n < N) *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + out + n) = y[i];
        }
      }
    }
  }
}

template <int DT>
__global__ __launch_bounds__(256) void grouped_short(GroupedArgs a, int tiles_a) {
  __shared__ int wsum[4];
  extern __shared__ int tpre[];  // [n_active + 1]
  Tile<kForward, kShortA, kShortB, 4> t;
  if (!t.init(a, tiles_a, 1, tpre, wsum, nullptr)) return;  // the whole workgroup
  if (a.dtype == MOE_DTYPE_F32) short_sums<DT, MOE_DTYPE_F32>(a, t);
  else if (a.dtype == MOE_DTYPE_BF16) short_sums<DT, MOE_DTYPE_BF16>(a, t);
  else short_sums<DT, MOE_DTYPE_F16>(a, t);
}

// Forward with at most 32 outputs and a longer sum (an adapter's first product): few tiles,
// whose steps' latency is what costs. The 4 wavefronts of a workgroup take the sum's chunks
// of 64 elements in turn and add their parts in order at the end; a lane's 16 consecutive
// elements of a chunk, one 32-byte piece of a row, go from memory to the products, D chunks
// ahead, with no barrier.
constexpr int kNarrowA = 32, kNarrowB = 32;
template <int DT, int NF, int D>
__device__ void narrow_sums(const GroupedArgs& a, const Tile<kForward, kNarrowA, kNarrowB, 4>& t,
                            f32x4* parts) {
  constexpr int MF = kNarrowB / 16, kTiles = NF * MF;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int N = a.N, K = a.K, chunks = (K + 63) / 64;
  const uint8_t* p[NF + MF];  // rows of w, then of x
#pragma unroll
  for (int i = 0; i < NF; ++i)
    p[i] = a.w + (t.row * N + min(16 * i + r, N - 1)) * (int64_t)K * 2 + 32 * q;
#pragma unroll
  for (int j = 0; j < MF; ++j) {
    const int slot = a.slots[min(t.m0 + 16 * j + r, t.m1 - 1)];
    p[NF + j] = a.x + (int64_t)token(a, slot) * K * 2 + 32 * q;
  }
  struct Chunk {
    i32x4 v[NF + MF][2];
  };
  // zeros past the end of the sum
  auto load = [&](int c, Chunk& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = 64 * c + 16 * q + 8 * h < K;
#pragma unroll
      for (int i = 0; i < NF + MF; ++i)
        f.v[i][h] =
            *reinterpret_cast<const i32x4*>(in ? p[i] + ((int64_t)128 * c + 16 * h) : kZeros);
    }
  };
  f32x4 acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  Chunk f[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load(wv + 4 * d, f[d]);
  for (int c = wv; c < chunks; c += 4 * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
          for (int j = 0; j < MF; ++j)
            acc[i][j] = mfma<DT>(f[d].v[i][h], f[d].v[NF + j][h], acc[i][j]);
      load(c + 4 * (D + d), f[d]);
    }
  }
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) parts[(wv * kTiles + i * MF + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int tile = wv; tile < kTiles; tile += 4) {
    f32x4 y = parts[tile * 64 + lane];
    for (int k = 1; k < 4; ++k) y += parts[(k * kTiles + tile) * 64 + lane];
    const int n = tile / MF * 16 + 4 * q, at = t.m0 + tile % MF * 16 + r;
    if (n >= N || at >= t.m1) continue;  // N is a multiple of 8
    const int64_t out = a.slots[at] * a.ldy + n;
    if (a.dtype == MOE_DTYPE_F32)
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + out) = y;
    else if (a.dtype == MOE_DTYPE_BF16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + out) =
          make_uint2(pack2<MOE_DTYPE_BF16>(y[0], y[1]), pack2<MOE_DTYPE_BF16>(y[2], y[3]));
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + out) =
          make_uint2(pack2<MOE_DTYPE_F16>(y[0], y[1]), pack2<MOE_DTYPE_F16>(y[2], y[3]));
  }
}

template <int DT, int NF>
__global__ __launch_bounds__(256) void grouped_narrow(GroupedArgs a) {
  __shared__ int wsum[4];
  __shared__ f32x4 parts[4 * NF * (kNarrowB / 16) * 64];
  extern __shared__ int tpre[];  // [n_active + 1]
  Tile<kForward, kNarrowA, kNarrowB, 4> t;
  if (!t.init(a, 1, 1, tpre, wsum, nullptr)) return;  // the whole workgroup
  narrow_sums<DT, NF, NF == 1 ? 4 : 3>(a, t, parts);
}

struct Grid {
  int64_t tiles_a, tiles_b, tiles, lds;
};
// Grouped rows: at most one part-filled tile per active row.
Grid grid_of(const GroupedArgs& a, int ta, int tb) {
  const int64_t tiles_a = ((a.op == kForward ? a.N : a.K) + ta - 1) / ta;
  if (a.op == kWeights) {
    const int64_t tiles_b = (a.N + tb - 1) / tb;
    return {tiles_a, tiles_b, a.n_rows * tiles_a * tiles_b, 0};
  }
  const int64_t cap = a.n_rows < a.M ? a.n_rows : a.M;
  return {tiles_a, 1, (cap + a.M / tb) * tiles_a, (cap + 1) * (int64_t)sizeof(int)};
}

template <int OP, int DT, int TA, int TB, int WA, int WB, int S>
hipError_t go(const GroupedArgs& a, hipStream_t stream) {
  const Grid g = grid_of(a, TA, TB);
  hipLaunchKernelGGL((grouped<OP, DT, TA, TB, WA, WB, S>),
                     dim3((unsigned)((g.tiles + kXcds - 1) / kXcds * kXcds)), dim3(64 * WA * WB),
                     g.lds, stream, a, (int)g.tiles_a, (int)g.tiles_b);
  return hipGetLastError();
}

template <int DT>
hipError_t go_short(const GroupedArgs& a, hipStream_t stream) {
  const Grid g = grid_of(a, kShortA, kShortB);
  hipLaunchKernelGGL((grouped_short<DT>), dim3((unsigned)((g.tiles + kXcds - 1) / kXcds * kXcds)),
                     dim3(256), g.lds, stream, a, (int)g.tiles_a);
  return hipGetLastError();
}

template <int DT, int NF>
hipError_t go_narrow(const GroupedArgs& a, hipStream_t stream) {
  const Grid g = grid_of(a, kNarrowA, kNarrowB);
  hipLaunchKernelGGL((grouped_narrow<DT, NF>),
                     dim3((unsigned)((g.tiles + kXcds - 1) / kXcds * kXcds)), dim3(256), g.lds,
                     stream, a);
  return hipGetLastError();
}

template <int OP, int DT>
hipError_t go_wide(const GroupedArgs& a, hipStream_t stream) {
  const Grid g = grid_of(a, kWideA, kWideB);
  const dim3 blocks((unsigned)((g.tiles + kXcds - 1) / kXcds * kXcds));
  if constexpr (OP == kForward)
    hipLaunchKernelGGL((grouped_forward<DT>), blocks, dim3(512), g.lds, stream, a,
                       (int)g.tiles_a);
  else
    hipLaunchKernelGGL((grouped_gradient<OP, DT>), blocks, dim3(256), g.lds, stream, a,
                       (int)g.tiles_a, (int)g.tiles_b);
  return hipGetLastError();
}

// Times in the rules below: us, calls in a row by events, so with operands in the caches
// where they fit, each kernel launched whatever the rule. Rows are T k / n_rows: with two
// banks both banks' picks count for each, so that one with a small share is taken for a
// fuller one (89 rows of 5760 x 4096 with 230, 720 and 2525 of 24576 slots: 128 x 64 691, 719,
// 751; wide, which it takes, 687, 716, 753).
//
// Wide tiles where they fill the card (forward one workgroup per CU, the gradients two), the
// result is wider than one ordinary tile (for the weights' gradient a small one) and, but
// there, an expert has rows for them. 128 x 64 tiles / wide ones:
// forward 2880 x 4096, 64 experts, 48 rows each 285 / 287, 56 310 / 290, 64 341 / 294, 80 396 /
// 299, 384 1016 / 794; 5760 x 4096, 384 experts, 64 rows 3863 / 3421; 2048 x 1408, 128 experts,
// 64 rows 196 / 174; 4096 x 2880, 8 experts, 96 rows (112 wide tiles) 39 / 43, 192 66 / 52; 4096
// x 256, 16 experts, 2048 rows 265 / 213; 4096 x 512, 125 rows 30 / 34, 512 85 / 74. By width, 64
// experts, K 4096, 384 rows: 40 outputs 45 / 57, 64 48 / 58, 96 49 / 58, 128 66 / 64, 136 102 / 64,
// 256 125 / 87; 128 outputs, 16 experts, K 1024, 4096 rows 45 / 57.
// Input 2880 x 4096, 64 experts, 12 rows 275 / 271, 24 282 / 274, 384 1039 / 735; by width, N 4096,
// 64 experts, 384 rows: 16 columns 48 / 76, 64 51 / 80, 128 67 / 82, 136 112 / 80, 256 131 / 99.
// Above about 510 rows in the bank the prefix of its tiles no longer fits beside two
// workgroups' buffers, and the input's gradient takes 128 x 64 tiles.
// Weights (128 x 128 / wide) 2880 x 4096, 64 experts, 12 rows 766 / 475, 384 1749 / 1078 (1,190
// with operands from HBM); 4096 x 96, 64 experts, 94 rows 42 / 36, 72 x 4096 39 / 26.
bool use_wide(const GroupedArgs& a) {
  const Grid g = grid_of(a, kWideA, kWideB);
  const int64_t cus = device_cus(), cap = a.n_rows < a.M ? a.n_rows : a.M;
  const size_t fixed = a.op == kForward ? 3 * (kWideA + kWideB) * 128 + 256 : 78 << 10;
  if (g.lds + fixed > (a.op == kForward ? device_lds_per_block() : 80 << 10)) return false;
  switch (a.op) {
    case kForward: return a.N > 128 && a.M >= 64 * cap && g.tiles >= cus;
    case kInput: return a.K > 128 && a.M >= 24 * cap && g.tiles >= 2 * cus;
    default: return a.K > 64 && g.tiles >= 2 * cus;
  }
}

// Small tiles (64 x 32, two workgroups per CU), with many buffers, where all that there may
// be are about one round of them: 2 1/4 per CU, as part-filled ones are counted for every
// expert. 128 x 64 / small, with that count: forward 4096 x 2880, one token's 6 experts (384)
// 27 / 24, 12 (768) 41 / 44; 2048 x 1408, 16 slots (512) 15.9 / 14.9, 32 experts, 64 slots (1088)
// 27 / 30; 1024 x 4096, 64 experts, 64 slots (1056) 76 / 78; 264 x 5000, 4 experts, 3000 rows
// (485) 49 / 39, 6000 (955) 68 / 78; 520 x 1032, 8 experts, 1000 rows (351) 12.4 / 10.2, 2048
// (648) 12.7 / 16.5; 64 x 4096, 64 experts, 96 rows each (256) 34 / 23, 384 (832) 48 / 53; 4096 x
// 4096, 256 rows (576) 35 / 24, 400 (832) 36 / 43. Input 4096 x 2880, one token (270) 38 / 28; N
// 4096, K 16, 384 experts, 2 rows each (408) 45 / 30, 16 (571) 48 / 31, 23 (665) 48 / 32, 31 (758)
// 49 / 55; 64 experts, 192 rows (448) 40 / 31, 384 (832) 48 / 57; 1024 x 1024, 16 experts, 32 rows
// (512) 14.5 / 13.2, 100 (1056) 15.8 / 21.5.
// The weights' small tiles (64 x 64, three per CU) for up to 64 columns, and else where
// they start no round more than 128 x 128 ones (one per CU). 128 x 128 / small: 4096 x 16, 64
// experts, 94 rows 33 / 23, 4096 x 64 37 / 28; 1024 x 1024 by experts, 4096 rows each: 2 69 / 57, 3
// (192 tiles of 128 x 128, 768 small) 69 / 65, 4 (256) 73 / 108; 1024 x 1280, 4 (320) 134 / 114,
// 1024 x 1536 (384) 134 / 121, 1024 x 1792 (448) 134 / 159; 520 x 1032, 8 (360), 256 rows 17 / 15;
// 264 x 5000, 4 (480), 750 rows 32 / 37; 2048 x 2048, 1 (256), 2048 rows 39 / 56.
bool use_small(const GroupedArgs& a) {
  const int64_t cus = device_cus();
  if (a.op != kWeights) return 4 * grid_of(a, 64, 32).tiles <= 9 * cus;
  const int64_t tiles = grid_of(a, 128, 128).tiles;
  return a.K <= 64 || 4 * tiles <= 3 * cus || (tiles > cus && tiles < 2 * cus);
}

template <int DT>
hipError_t pick(const GroupedArgs& a, hipStream_t s) {
  const bool wide = use_wide(a), small = use_small(a);
  switch (a.op) {
    case kForward:
      // 128 x 64 tiles / this: N 4096, 64 experts, K 16, 6000 slots 45 / 23, K 64 46 / 29; K 32,
      // 24576 slots 130 / 46; 136 x 64, 16000 slots 10.3 / 10.1
      if (a.K <= kShortK && a.N > 64) return go_short<DT>(a, s);
      // By N and K alone, as the sum's order is another one. 64 x 32 tiles / this: 16 x 4096,
      // 384 experts, 112 tokens 23.7 / 18.3, one token 18.4 / 10.4; 64 experts, 4096 tokens 49.3
      // / 49.6; 32 x 4096, 384 experts, 1000 tokens 28 / 33; a form for 64 outputs, 64 x 4096, 64
      // experts, 4096 tokens, 93 against 48 with 128 x 64 tiles
      if (a.K > kShortK && a.N <= kNarrowA)
        return a.N <= 16 ? go_narrow<DT, 1>(a, s) : go_narrow<DT, 2>(a, s);
      return wide    ? go_wide<kForward, DT>(a, s)
             : small ? go<kForward, DT, 64, 32, 2, 2, 6>(a, s)
                     : go<kForward, DT, 128, 64, 4, 2, 3>(a, s);
    case kInput:
      return wide    ? go_wide<kInput, DT>(a, s)
             : small ? go<kInput, DT, 64, 32, 2, 2, 6>(a, s)
                     : go<kInput, DT, 128, 64, 4, 2, 3>(a, s);
    default:
      return wide    ? go_wide<kWeights, DT>(a, s)
             : small ? go<kWeights, DT, 64, 64, 2, 2, 3>(a, s)
                     : go<kWeights, DT, 128, 128, 4, 2, 3>(a, s);
  }
}

}  // namespace

// The finest tiles any of the kernels takes for a large call (small ones are few), times
// its threads.
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
