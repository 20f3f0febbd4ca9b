// Products of 8-bit rows with a scale per activation row and per weight row,
// for few activation rows per weight matrix (decode): bound by streaming the
// weights once.
//
//   y[r][n] = sa[r] * sw[n] * sum_k a[r][k] w[n][k]
//
// Organised like the few-token layer's gate/up kernel (layer_few.hip): one
// workgroup of 8 wavefronts per CU; the reduction axis is cut over the
// wavefronts; a work item is 8 weight rows (8 gate and 8 up rows for the
// expert FFN); a wavefront holds its slice of the activations in registers as
// MFMA B operands (columns 0-7 the first halves of 8 rows' 128-byte chunks,
// columns 8-15 the second halves; the result's two diagonal 8 x 8 blocks are
// their partial sums) and streams its slice of the weights, a load taking 8
// rows x one 128-byte line, through a register ring. One barrier per step; the
// partial sums are added from LDS by one wavefront per item, in turn. Integer
// sums: no order, slice or pass changes a bit.
//
// The activations of up to 8 (16) rows of one group are a unit; a workgroup's
// run of items is contiguous over (unit, weight rows), so it reloads the
// activations and the scales once or twice. A group with more rows takes
// further units, which stream its weights again.
//
// Measured (H 4096, I 2880, 16 tokens of top-6 over 384 experts, about 69 of them
// met): gate/up 270-278 us, 5.9 TB/s of its 1.63 GB; down, whose 2880-byte rows
// are not whole lines, 139-142 us, 5.8 TB/s. One row times 5760 x 4096: 11.1 us,
// 2.1 TB/s, launch and first round trip being half of it.
#include <algorithm>

#include "gemm_i8.h"
#include "mxfp4_common.h"
#include "tile_items.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

struct Cut {
  int cpw, ks, sub;  // 128-byte chunks per wavefront, wavefronts per row, such groups
};
Cut cut_of(int K) {
  const int nchunk = (K + 127) / 128;
  int cpw = (nchunk + kWaves - 1) / kWaves;
  cpw = cpw <= 4 ? cpw : (cpw <= 6 ? 6 : 8);
  const int ks = (nchunk + cpw - 1) / cpw;
  return {cpw, ks, kWaves / ks};
}
constexpr int kMaxK = kWaves * 8 * 128;  // longest axis: 8 chunks per wavefront

__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
__device__ __forceinline__ i32x4 ld16(const uint8_t* p, bool stream) {
  const i32x4* v = reinterpret_cast<const i32x4*>(p);
  return stream ? __builtin_nontemporal_load(v) : *v;
}

// STREAM: rows are whole 128-byte lines, each read once (streaming policy).
template <int CPW, int SETS, bool GU, bool STREAM>
__global__ __launch_bounds__(kThreads, 2) void gemm_i8_stream(I8Args a, int ks, int nsub,
                                                              int run_items) {
  constexpr int RG = GU ? 2 : 1;  // row groups per item
  constexpr int kCols = 8 * SETS;
  // ring slots: about 128 KB of weights in flight per CU
  constexpr int R = RG * CPW >= 8 ? 2 : (RG * CPW >= 4 ? 4 : (RG * CPW == 3 ? 5 : 6));
  // [2][sub][RG][SETS][2 ks][8 columns][8 rows] partial sums | scales of the
  // run's weight rows in this unit [run_items][RG][8] | units before each
  // active row [n_active + 1]
  extern __shared__ __align__(16) int smem[];
  __shared__ int wsum[kWaves];
  __shared__ float l_sa[kCols];
  __shared__ int l_row[kCols];  // output row of each column, -1: none
  const int per_sub = RG * SETS * 2 * ks * 64;
  int* red = smem;
  float* l_sw = reinterpret_cast<float*>(smem + 2 * nsub * per_sub);
  int* upre = reinterpret_cast<int*>(l_sw + run_items * RG * 8);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slice = wv % ks, sub = wv / ks;
  const bool active = sub < nsub;
  const int r = lane & 15, q = lane >> 4;
  const int N = a.N, K = a.K;
  const int per = (N + 7) / 8;  // items per unit
  int units = 1;
  if (a.slots) {
    const int na = *a.n_active;
    tiles::build_tile_prefix<kCols, kWaves>(a.row_off, na, upre, wsum);
    units = __builtin_amdgcn_readfirstlane(upre[na]);
  }
  const int n = units * per;
  const int qb = (n + gridDim.x - 1) / gridDim.x;  // <= run_items or one unit's items
  const int g0 = blockIdx.x * qb, g1 = min(n, g0 + qb);
  if (g0 >= g1) return;  // the whole workgroup

  // this lane's 16-byte piece of each chunk, within a row; past the end of the
  // axis the row's start instead (the activations there are zero)
  uint32_t koff[CPW];
  bool in[CPW];
#pragma unroll
  for (int j = 0; j < CPW; ++j) {
    const int k = 128 * (slice * CPW + j) + 16 * (q + (r >= 8 ? 4 : 0));
    in[j] = k < K;
    koff[j] = in[j] ? (uint32_t)k : 0u;
  }

  // A place in the run: unit u, items [ib, end) of it left.
  struct Place {
    int u, ib, end;
  };
  auto at = [&](int u, int ib) { return Place{u, ib, min(per, g1 - u * per)}; };
  auto advance = [&](Place& p) {
    p.ib += nsub;
    if (p.ib >= p.end) p = at(p.u + 1, 0);
  };
  const Place start = at(g0 / per, g0 % per);
  int steps = 0;
  for (Place p = start; p.u * per < g1; p = at(p.u + 1, 0)) steps += (p.end - p.ib + nsub - 1) / nsub;

  // the active row and the first column of unit u
  auto group_of = [&](int u, int& first) {
    if (!a.slots) {
      first = 0;
      return 0;
    }
    const int e = tiles::row_of_tile(upre, __builtin_amdgcn_readfirstlane(*a.n_active), u);
    first = (u - __builtin_amdgcn_readfirstlane(upre[e])) * kCols;
    return __builtin_amdgcn_readfirstlane(e);
  };
  const int wrows = GU ? 2 * N : N;
  auto matrix = [&](int e) -> int64_t {  // first weight row of group e
    return a.slots ? (int64_t)__builtin_amdgcn_readfirstlane(a.active_rows[e]) * wrows : 0;
  };

  // prefetch cursor
  Place pp = start;
  int p_unit = -1;
  int64_t p_row = 0;
  i32x4 ring[R][RG][CPW];
  auto issue = [&](i32x4 (&o)[RG][CPW]) {
    const bool more = pp.u * per < g1;
    if (more && pp.u != p_unit) {
      int f;
      p_unit = pp.u;
      p_row = matrix(group_of(p_unit, f));
    }
    // past the run's end (or a part step's): the run's first matrix's first rows
    const int ib = more && active && pp.ib + sub < pp.end ? pp.ib + sub : 0;
    const uint8_t* base = reinterpret_cast<const uint8_t*>(a.w) + (p_row + 8 * ib) * (int64_t)K;
    const uint32_t lrow = (uint32_t)min(r & 7, N - 1 - 8 * ib) * (uint32_t)K;
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
      for (int j = 0; j < CPW; ++j)
        o[g][j] = ld16(base + (int64_t)g * N * K + lrow + koff[j], STREAM);
    __builtin_amdgcn_sched_barrier(0);
    if (more) advance(pp);
  };
#pragma unroll
  for (int u = 0; u < R; ++u) issue(ring[u]);

  i32x4 xb[SETS][CPW];
#pragma unroll
  for (int st = 0; st < SETS; ++st)
#pragma unroll
    for (int j = 0; j < CPW; ++j) xb[st][j] = i32x4{0, 0, 0, 0};
  // The unit at p becomes the current one; every wavefront calls it at the same
  // step.
  int cur = -1, sw0 = 0;
  auto enter = [&](const Place& p) {
    cur = p.u;
    sw0 = p.ib;
    int first;
    const int e = group_of(cur, first);
    const int64_t row0 = matrix(e);
    const int c0 = (a.slots ? a.row_off[e] : 0) + first;
    const int c1 = a.slots ? a.row_off[e + 1] : a.M;
    lds_barrier();  // the last unit's tables have been read
    if (tid < kCols) {
      int arow = 0, orow = -1;
      if (c0 + tid < c1) {
        orow = a.slots ? a.slots[c0 + tid] : c0 + tid;
        arow = a.slots && a.by_token ? orow / a.k : orow;
      }
      l_row[tid] = orow;
      l_sa[tid] = orow >= 0 ? a.sa[arow] : 0.0f;
    }
    for (int i = tid; i < (p.end - p.ib) * 8 * RG; i += kThreads) {
      const int it = i / (8 * RG), g = (i >> 3) % RG, rw = min(8 * (p.ib + it) + (i & 7), N - 1);
      l_sw[i] = a.sw[row0 + (int64_t)g * N + rw];
    }
#pragma unroll
    for (int st = 0; st < SETS; ++st) {
      const int c = c0 + st * 8 + (r & 7);
      const bool has = c < c1;
      int arow = 0;
      if (has) {
        arow = a.slots ? a.slots[c] : c;
        if (a.slots && a.by_token) arow /= a.k;
      }
      const uint8_t* p0 = reinterpret_cast<const uint8_t*>(a.a) + (int64_t)arow * a.lda;
#pragma unroll
      for (int j = 0; j < CPW; ++j) xb[st][j] = *reinterpret_cast<const i32x4*>(p0 + koff[j]);
#pragma unroll
      for (int j = 0; j < CPW; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) xb[st][j][v] = has && in[j] ? xb[st][j][v] : 0;
    }
    lds_barrier();
  };

  const bool diag = (r >= 8) == (q >= 2) && active;
  const int red_off = (2 * slice + (r >= 8)) * 64 + (r & 7) * 8 + (q & 1) * 4;
  Place pc = start;
  // whole turns of the ring: the steps past the run's end store nothing
  for (int s0 = 0; s0 < steps; s0 += R) {
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const int step = s0 + u;
      const bool live = step < steps;
      if (live && pc.u != cur) enter(pc);
      i32x4 acc[RG][SETS];
      if (live) {
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
          for (int st = 0; st < SETS; ++st) {
            acc[g][st] = i32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < CPW; ++j)
              acc[g][st] = __builtin_amdgcn_mfma_i32_16x16x64_i8(ring[u][g][j], xb[st][j],
                                                                 acc[g][st], 0, 0, 0);
          }
      }
      issue(ring[u]);
      if (live) {
        if (diag) {
          int* o = red + ((step & 1) * nsub + sub) * per_sub + red_off;
#pragma unroll
          for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int st = 0; st < SETS; ++st)
              *reinterpret_cast<i32x4*>(o + (g * SETS + st) * 2 * ks * 64) = acc[g][st];
        }
        lds_barrier();
        // see few_gate_up: one wavefront per item, each in turn
        for (int sb = 0; sb < nsub; ++sb) {
          const int ib = pc.ib + sb;
          if (ib >= pc.end || (step * nsub + sb) % kWaves != wv) continue;
          const int* o = red + ((step & 1) * nsub + sb) * per_sub + lane;
          const float* sw = l_sw + (ib - sw0) * 8 * RG + (lane & 7);
          const int nn = 8 * ib + (lane & 7);
#pragma unroll
          for (int st = 0; st < SETS; ++st) {
            int s[RG];
#pragma unroll
            for (int g = 0; g < RG; ++g) s[g] = 0;
            auto add = [&](int p) {
#pragma unroll
              for (int g = 0; g < RG; ++g) s[g] += o[((g * SETS + st) * 2 * ks + p) * 64];
            };
            if (ks == kWaves) {
#pragma unroll
              for (int p = 0; p < 2 * kWaves; ++p) add(p);
            } else {
              for (int p = 0; p < 2 * ks; ++p) add(p);
            }
            const int c = st * 8 + (lane >> 3);
            const int row = l_row[c];
            if (row >= 0 && nn < N) {
              const float sa = l_sa[c];
              if constexpr (GU) {
                static_cast<float*>(a.y)[(int64_t)row * a.ldy + nn] =
                    mx::silu_f32((float)s[0] * sa * sw[0]) * ((float)s[RG - 1] * sa * sw[8]);
              } else {
                store1(a, row, nn, (float)s[0] * sa * sw[0]);
              }
            }
          }
        }
        advance(pc);
      }
    }
  }
}

// Items of the longest run of one unit in one workgroup (the whole unit at most,
// and with the most units the step can have, their even share), and the LDS
// bytes that follow.
struct Plan {
  int grid, run;
  size_t lds;
};
Plan plan_of(const I8Args& a, const Cut& c, int sets) {
  const int rg = a.gate_up ? 2 : 1, per = (a.N + 7) / 8;
  const int grid = a.host ? kHostBankCUs : device_cus();
  const int64_t cap = a.slots ? (a.n_rows < a.M ? a.n_rows : a.M) : 1;
  const int64_t units = a.slots ? cap + a.M / (8 * sets) : 1;
  const int64_t share = (units * per + grid - 1) / grid;
  const int run = (int)std::min<int64_t>(share, per);
  const size_t lds = ((size_t)2 * c.sub * rg * sets * 2 * c.ks * 64 + (size_t)run * rg * 8 +
                      (a.slots ? cap + 1 : 0)) * 4;
  return {grid, run, lds};
}
constexpr size_t kMaxLds = 144 * 1024;

template <int CPW, int SETS, bool GU>
hipError_t go(const I8Args& a, const Cut& c, hipStream_t stream) {
  const Plan p = plan_of(a, c, SETS);
  const bool lines = a.K % 128 == 0 && reinterpret_cast<uintptr_t>(a.w) % 128 == 0;
  auto kern = lines ? gemm_i8_stream<CPW, SETS, GU, true> : gemm_i8_stream<CPW, SETS, GU, false>;
  hipLaunchKernelGGL(kern, dim3(p.grid), dim3(kThreads), p.lds, stream, a, c.ks, c.sub, p.run);
  return hipGetLastError();
}

template <int CPW>
hipError_t pick(const I8Args& a, const Cut& c, hipStream_t s) {
  // grouped: units of 8 slots (an expert rarely has more in such steps); 16
  // columns at once would double the registers and products for most
  if (a.gate_up) return go<CPW, 1, true>(a, c, s);
  if (a.slots || a.M <= 8) return go<CPW, 1, false>(a, c, s);
  return go<CPW, 2, false>(a, c, s);
}

}  // namespace

bool gemm_i8_use_stream(const I8Args& a) {
  if (a.K > kMaxK || plan_of(a, cut_of(a.K), a.slots || a.M <= 8 ? 1 : 2).lds > kMaxLds)
    return false;
  if (!a.slots) return a.M <= 16;
  const int64_t cap = a.n_rows < a.M ? a.n_rows : a.M;
  return a.M <= 4096 && a.M <= 4 * cap;
}

hipError_t launch_gemm_i8_stream(const I8Args& a, hipStream_t s) {
  const Cut c = cut_of(a.K);
  switch (c.cpw) {
    case 1: return pick<1>(a, c, s);
    case 2: return pick<2>(a, c, s);
    case 3: return pick<3>(a, c, s);
    case 4: return pick<4>(a, c, s);
    case 6: return pick<6>(a, c, s);
    default: return pick<8>(a, c, s);
  }
}

bool gemm_i8_fits(const I8Args& a) { return gemm_i8_use_stream(a) || gemm_i8_tile_fits(a); }

hipError_t launch_gemm_i8(const I8Args& a, hipStream_t s) {
  return gemm_i8_use_stream(a) ? launch_gemm_i8_stream(a, s) : launch_gemm_i8_tile(a, s);
}

}  // namespace moe
