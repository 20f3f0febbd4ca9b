// Dense products of 8-bit rows with a scale per activation row and per weight
// row, for at most 16 activation rows and matrices that the tiles stream less
// well (few long rows, many rows of 4096 or 8192): bound by streaming the
// weights once.
//
//   y[m][n] = sa[m] * sw[n] * sum_k a[m][k] w[n][k]
//
// Organised like the few-token layer's gate/up kernel (layer_few.hip): one
// workgroup of 8 wavefronts per CU; the reduction axis is cut over the
// wavefronts; a work item is 8 weight rows; a wavefront holds its slice of the
// activations in registers as MFMA B operands (columns 0-7 the first halves of 8
// rows' 128-byte chunks, columns 8-15 the second halves; the result's two
// diagonal 8 x 8 blocks are their partial sums) and streams its slice of the
// weights, a load taking 8 rows x one 128-byte line, through a register ring.
// One barrier per step; the partial sums are added from LDS by one wavefront per
// item, in turn. Integer sums: no order or slice changes a bit.
//
// Measured (one row, bf16 out, in a graph): N 65536 x K 8192 96.7 us, 5.6 TB/s;
// 4096 x 8192 12.4 us, 2.7 TB/s. gemm_i8_use_stream has the tiles' times.
#include <algorithm>

#include "gemm_i8.h"

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
  const int cpw = nchunk <= 32 ? 4 : 8;  // K is 4096, or above 6144
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
template <int CPW, int SETS, bool STREAM>
__global__ __launch_bounds__(kThreads, 2) void gemm_i8_stream(I8Args a, int ks, int nsub) {
  constexpr int kCols = 8 * SETS;
  // ring slots: about 128 KB of weights in flight per CU
  constexpr int R = CPW >= 8 ? 2 : 4;
  // [2][sub][SETS][2 ks][8 columns][8 rows] partial sums | scales of the run's
  // weight rows
  extern __shared__ __align__(16) int smem[];
  __shared__ float l_sa[kCols];
  const int per_sub = SETS * 2 * ks * 64;
  int* red = smem;
  float* l_sw = reinterpret_cast<float*>(smem + 2 * nsub * per_sub);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slice = wv % ks, sub = wv / ks;
  const bool active = sub < nsub;
  const int r = lane & 15, q = lane >> 4;
  const int N = a.N, K = a.K, M = a.M;
  // this workgroup's run of items: [g0, g1)
  const int items = (N + 7) / 8, share = (items + gridDim.x - 1) / gridDim.x;
  const int g0 = blockIdx.x * share, g1 = min(items, g0 + share);
  if (g0 >= g1) return;  // the whole workgroup
  const int steps = (g1 - g0 + nsub - 1) / nsub;

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

  int next = g0;  // prefetch cursor
  i32x4 ring[R][CPW];
  auto issue = [&](i32x4 (&o)[CPW]) {
    // past the run's end (or a part step's): the matrix's first rows
    const int it = active && next + sub < g1 ? next + sub : 0;
    const uint8_t* base = reinterpret_cast<const uint8_t*>(a.w) + (int64_t)(8 * it) * K;
    const uint32_t row = (uint32_t)min(r & 7, N - 1 - 8 * it) * (uint32_t)K;
#pragma unroll
    for (int j = 0; j < CPW; ++j) o[j] = ld16(base + row + koff[j], STREAM);
    __builtin_amdgcn_sched_barrier(0);
    next += nsub;
  };
#pragma unroll
  for (int u = 0; u < R; ++u) issue(ring[u]);

  if (tid < kCols) l_sa[tid] = tid < M ? a.sa[tid] : 0.0f;
  for (int i = tid; i < (g1 - g0) * 8; i += kThreads) l_sw[i] = a.sw[min(8 * g0 + i, N - 1)];
  i32x4 xb[SETS][CPW];
#pragma unroll
  for (int st = 0; st < SETS; ++st) {
    const int m = st * 8 + (r & 7);
    const uint8_t* p0 = reinterpret_cast<const uint8_t*>(a.a) + (int64_t)(m < M ? m : 0) * a.lda;
#pragma unroll
    for (int j = 0; j < CPW; ++j) xb[st][j] = *reinterpret_cast<const i32x4*>(p0 + koff[j]);
#pragma unroll
    for (int j = 0; j < CPW; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) xb[st][j][v] = m < M && in[j] ? xb[st][j][v] : 0;
  }
  lds_barrier();

  const bool diag = (r >= 8) == (q >= 2) && active;
  const int red_off = (2 * slice + (r >= 8)) * 64 + (r & 7) * 8 + (q & 1) * 4;
  // whole turns of the ring: the steps past the run's end store nothing
  for (int s0 = 0; s0 < steps; s0 += R) {
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const int step = s0 + u;
      const bool live = step < steps;
      i32x4 acc[SETS];
      if (live) {
#pragma unroll
        for (int st = 0; st < SETS; ++st) {
          acc[st] = i32x4{0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < CPW; ++j)
            acc[st] = __builtin_amdgcn_mfma_i32_16x16x64_i8(ring[u][j], xb[st][j], acc[st], 0, 0, 0);
        }
      }
      issue(ring[u]);
      if (live) {
        if (diag) {
          int* o = red + ((step & 1) * nsub + sub) * per_sub + red_off;
#pragma unroll
          for (int st = 0; st < SETS; ++st)
            *reinterpret_cast<i32x4*>(o + st * 2 * ks * 64) = acc[st];
        }
        lds_barrier();
        // see few_gate_up: one wavefront per item, each in turn
        for (int sb = 0; sb < nsub; ++sb) {
          const int it = g0 + step * nsub + sb;
          if (it >= g1 || (step * nsub + sb) % kWaves != wv) continue;
          const int* o = red + ((step & 1) * nsub + sb) * per_sub + lane;
          const float sw = l_sw[(it - g0) * 8 + (lane & 7)];
          const int n = 8 * it + (lane & 7);
#pragma unroll
          for (int st = 0; st < SETS; ++st) {
            int s = 0;
            auto add = [&](int p) { s += o[(st * 2 * ks + p) * 64]; };
            if (ks == kWaves) {
#pragma unroll
              for (int p = 0; p < 2 * kWaves; ++p) add(p);
            } else {
              for (int p = 0; p < 2 * ks; ++p) add(p);
            }
            const int m = st * 8 + (lane >> 3);
            if (m < M && n < N) store1(a, m, n, (float)s * l_sa[m] * sw);
          }
        }
      }
    }
  }
}

size_t lds_bytes(const I8Args& a, const Cut& c, int sets) {
  const int items = (a.N + 7) / 8, run = (items + device_cus() - 1) / device_cus();
  return ((size_t)2 * c.sub * sets * 2 * c.ks * 64 + (size_t)run * 8) * 4;
}
constexpr size_t kMaxLds = 144 * 1024;

template <int CPW, int SETS>
hipError_t go(const I8Args& a, const Cut& c, hipStream_t stream) {
  const bool lines = a.K % 128 == 0 && reinterpret_cast<uintptr_t>(a.w) % 128 == 0;
  auto kern = lines ? gemm_i8_stream<CPW, SETS, true> : gemm_i8_stream<CPW, SETS, false>;
  hipLaunchKernelGGL(kern, dim3(device_cus()), dim3(kThreads), lds_bytes(a, c, SETS), stream, a,
                     c.ks, c.sub);
  return hipGetLastError();
}

template <int CPW>
hipError_t pick(const I8Args& a, const Cut& c, hipStream_t s) {
  return a.M <= 8 ? go<CPW, 1>(a, c, s) : go<CPW, 2>(a, c, s);
}

}  // namespace

// us for 1 row (16 rows), this kernel / the tiles, bf16 out, in a graph over
// weights that are not on chip:
//   K 8192: N 64 9.9 / 13.4 (12.7 / 13.5), 4096 12.4 / 18.0 (15.2 / 18.2),
//           16384 28.9 / 33.8 (32.2 / 33.9), 65536 96.7 / 106 (105 / 107)
//   K 7168: N 4096 11.8 / 16.0 (15.3 / 16.0), 16384 26.5 / 27.5 (31.1 / 27.6),
//           32768 46.5 / 42.7 (54.1 / 42.7)
//   K 6144: N 4096 15.0 / 14.0 (17.0 / 14.1), 16384 25.4 / 23.9 (27.5 / 24.0)
//   K 4096: N 5760 11.4 / 10.7 (12.7 / 10.9), 16384 18.6 / 18.6 (19.5 / 18.7),
//           65536 51.1 / 64.5 (54.1 / 64.5)
//   K 2880: N 5760 8.8 / 8.8 (10.2 / 8.8), 65536 38.6 / 35.8 (47.3 / 37.4)
//   K 2048: N 5760 8.7 / 6.9 (9.9 / 7.0), 65536 29.4 / 26.5 (38.7 / 27.1)
// So: rows past 6144 of matrices that do not fill the tiles, and many rows of
// whole multiples of 4096 bytes, which the tiles' loads of one line of each of
// 128 rows read at a lower rate.
// Grouped products had a form of this kernel too, slower than the tiles at every
// step measured (384 experts, H 4096, I 2880, top-6: 16 tokens 465 / 459 us, 128
// tokens 1439 / 1288, 256 tokens 2262 / 1657; 16 tokens on the same 6 experts
// 93.5 / 50.0; an expert in host memory 865 / 838).
bool gemm_i8_use_stream(const I8Args& a) {
  if (a.slots || a.M > 16 || a.K > kMaxK) return false;
  const bool many = a.N >= 64 * device_cus();
  if (many ? a.K % 4096 != 0 : a.K <= 6144) return false;
  return lds_bytes(a, cut_of(a.K), a.M <= 8 ? 1 : 2) <= kMaxLds;
}

hipError_t launch_gemm_i8_stream(const I8Args& a, hipStream_t s) {
  const Cut c = cut_of(a.K);
  return c.cpw == 4 ? pick<4>(a, c, s) : pick<8>(a, c, s);
}

bool gemm_i8_fits(const I8Args& a) { return gemm_i8_use_stream(a) || gemm_i8_tile_fits(a); }

hipError_t launch_gemm_i8(const I8Args& a, hipStream_t s) {
  return gemm_i8_use_stream(a) ? launch_gemm_i8_stream(a, s) : launch_gemm_i8_tile(a, s);
}

}  // namespace moe
