// The whole routed MXFP4 layer for a few tokens (at most 16) in two launches,
// against six for the split, the two banks' gate/up and down, and the finalize.
//
//   out[t] = sum over the distinct experts e of token t of
//            Wdown[e] . bf16(w[t][e] * silu(Wgate[e] . x[t]) * (Wup[e] . x[t]))
//
// The router weight multiplies h before its one rounding to bf16 (the MFMA
// operand type; an error of at most 2^-8 of each h, as the split path has), so
// that the down products of a token's experts add up in one fp32 accumulator
// and no row per pick is written: the second kernel ends in `out`.
//
// A step of one token touches 6 of 384 experts, 113 MB: it is bound by how
// soon every CU has its share of those bytes in flight. Hence, in both kernels:
//  - The reduction axis is cut over the wavefronts of a workgroup (512 of 4096
//    elements each), and a work item is only 8 rows of the product (8 gate and
//    8 up rows; 16 down rows), so that one expert already spreads over all CUs.
//  - Each wavefront holds its slice of the activations in registers (gate/up)
//    or in LDS (down) and streams weights through a register ring
//    some items ahead, with one barrier per two gate/up items for the sum of
//    the wavefronts' partial results (the step at 16 tokens: 247 us, 260 with
//    one barrier per item; at 1 and 7 tokens no difference) and none but the
//    staging's in the down kernel.
//  - A weight load takes 8 rows x one whole 128-byte line (256 elements). Lanes
//    r < 8 of the MFMA operand hold the first half of row r's line, lanes r >= 8
//    the second half of row r - 8's; the B operand holds the tokens' first
//    halves in columns 0-7 and their second halves in columns 8-15. The result
//    tile's two diagonal 8 x 8 blocks are then the two halves' partial sums
//    (the other two are discarded), and no lane exchange is needed. More than 8
//    tokens take a second set of columns (which 8 and fewer could do without
//    harm to the result, but not for nothing: the step at 1, 7 and 8 tokens 34.3,
//    129.5 and 144.4 us with two sets, 32.7, 127.5 and 140.6 with one).
// The order of every sum is fixed by the shapes and the picks' order alone, not
// by the banks: a step gives the same bits wherever its experts are.
#include <algorithm>
#include <type_traits>

#include "layer_ops.h"
#include "mxfp4_common.h"

namespace moe {
namespace {

using namespace mx;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxPicks = MOE_FEW_MAX_TOKENS * MOE_MAX_TOPK;  // 512
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
static_assert(kThreads >= kMaxPicks, "one thread per pick");
constexpr int kMaxH = 8192, kMaxI = 4096;

// What the gate/up kernel leaves for the down kernel, at the workspace's start;
// the h rows follow it.
struct Tables {
  int32_t n_u;               // distinct experts, in the order of their first picks
  int32_t pad[15];
  int32_t row[kMaxPicks];    // row map entry of each: >= 0 hot, < 0 cold
  int32_t mask[kMaxPicks];   // its tokens, one bit each
  int32_t base[kMaxPicks];   // its first h row; one row per token, ascending
};
constexpr size_t kTableBytes = (sizeof(Tables) + 255) / 256 * 256;

// How a reduction axis of K elements is cut: chunks of 256 elements, CPW
// consecutive chunks per wavefront, KS wavefronts per row, SUB such groups.
struct Cut {
  int nchunk, cpw, ks, sub;
};
// Gate/up: as many wavefronts per row as there are (its partial sums go through
// LDS for every item anyway, and short slices keep the x operands few): the step
// at 1, 7 and 16 tokens and H = 4096 32.7, 127.5 and 247 us with 8 wavefronts of
// 2 chunks, 37.2, 132.4 and 248 with 2 x 4 of 4. Above 4096 a wavefront takes 4
// chunks, so H just past it leaves some idle (16 tokens: 2.9 TB/s at H = 4160, 4.6
// at 8128, 4.95 at 8192, 4.5 at 4096; the ragged form for two sets also spills 16
// registers).
__host__ __device__ inline Cut gate_up_cut(int H) {
  Cut c;
  c.nchunk = (H + kChunkElems - 1) / kChunkElems;
  c.cpw = c.nchunk <= 8 ? 1 : (c.nchunk <= 16 ? 2 : 4);
  c.ks = (c.nchunk + c.cpw - 1) / c.cpw;
  c.sub = kWaves / c.ks;
  return c;
}
// Down: at most 4 wavefronts per row and the rest on other experts, so that the
// SIMDs have equal shares and an expert's fixed cost is paid by few wavefronts
// (7 tokens at I = 2880: 6 wavefronts of 2 chunks 56 us, 2 x 4 of 3 chunks
// 47.7 us).
__host__ __device__ inline Cut down_cut(int I) {
  Cut c;
  c.nchunk = (I + kChunkElems - 1) / kChunkElems;
  c.cpw = (c.nchunk + 3) / 4;
  c.ks = (c.nchunk + c.cpw - 1) / c.cpw;
  c.sub = kWaves / c.ks;
  return c;
}

// Orders LDS between the wavefronts of the workgroup and leaves global loads in
// flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// One ring slot: the weights of 16 rows (two groups of 8) over the wavefront's
// chunks and their scale bytes, as loaded (nothing looks at a loaded value
// before its step: widening a half word at the load would wait for it). Lane l
// loads scale bytes of row l / 4. WIDE (gate/up, whole slices): 2 CPW
// consecutive bytes of the slice; otherwise the 8 bytes of one chunk (chunk l % 4
// of the slice), with CPW = 1 the two bytes l % 4 of the one chunk.
template <int CPW, bool WIDE>
struct Slot {
  static constexpr bool kPairs = !WIDE && CPW == 1;
  uint4 w[2][CPW];
  std::conditional_t<kPairs, uint16_t, uint32_t> s[kPairs ? 1 : (WIDE ? CPW / 2 : 2)];
};

// The lane's place in the weight rows of a slice: rows of K/2 bytes, K/32
// scale bytes. Pieces (32 elements, 16 bytes, 1 scale byte) past the end of the
// axis are read at the row's start instead; their scale becomes 1 and their
// activations are zero.
template <int CPW, bool WIDE>
struct Lane {
  uint32_t woff[CPW];              // weight bytes, within a group of 8 rows
  uint32_t soff;                   // scale bytes, within this lane's row
  int sfirst[CPW];                 // a chunk's first scale byte, within the 8 loaded
  bool in[CPW];
  int r, q, srow, piece;

  __device__ __forceinline__ void init(int lane, int slice, int K) {
    r = lane & 15;
    q = lane >> 4;
    srow = lane >> 2;
    piece = q + (r >= 8 ? 4 : 0);
    const int nblk = K / 32;  // even
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      const int b = (slice * CPW + j) * 8 + piece;
      in[j] = WIDE || b < nblk;
      woff[j] = (uint32_t)(r & 7) * (uint32_t)(K / 2) + 16u * (uint32_t)(in[j] ? b : 0);
    }
    if constexpr (WIDE) {
      soff = slice * CPW * 8 + (lane & 3) * 2 * CPW;
    } else if constexpr (CPW == 1) {
      const int b = slice * 8 + 2 * (lane & 3);
      soff = b < nblk ? b : 0;
    } else {
      // 8 bytes end at the row's end at the latest (rows are longer than 8)
      auto start = [&](int c) { return min(8 * c, nblk - 8); };
      soff = start(slice * CPW + min(lane & 3, CPW - 1));
#pragma unroll
      for (int j = 0; j < CPW; ++j) sfirst[j] = 8 * (slice * CPW + j) - start(slice * CPW + j);
    }
  }

  // g0, g1: the two groups' first weight rows; sb: the item's scale rows, of
  // which this lane's starts at so.
  template <bool STREAM>
  __device__ __forceinline__ void load(Slot<CPW, WIDE>& o, const uint8_t* g0, const uint8_t* g1,
                                       const uint8_t* sb, uint32_t so) const {
    const uint8_t* sp = sb + so;
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      if constexpr (STREAM) {
        o.w[0][j] = ld_stream16(g0 + woff[j]);
        o.w[1][j] = ld_stream16(g1 + woff[j]);
      } else {
        o.w[0][j] = *reinterpret_cast<const uint4*>(g0 + woff[j]);
        o.w[1][j] = *reinterpret_cast<const uint4*>(g1 + woff[j]);
      }
    }
    load_scales(o, sp);
  }
  __device__ __forceinline__ void load_scales(Slot<CPW, WIDE>& o, const uint8_t* sp) const {
    if constexpr (Slot<CPW, WIDE>::kPairs)
      o.s[0] = *reinterpret_cast<const uint16_t*>(sp + soff);
    else
      __builtin_memcpy(o.s, sp + soff, sizeof o.s);  // even addresses; one load
  }

  // This lane's scales of group g: the E8M0 byte of its piece of chunk j, of row
  // (r & 7) + 8g, turned into the exponent field of the conversion's fp32 scale
  // operand. The instruction reads that field only (the tests run bytes 0 .. 254
  // through both products with other bytes beside them, and NaN's), so a rotation
  // replaces e8m0_to_f32's selects.
  __device__ __forceinline__ void scales(const Slot<CPW, WIDE>& o, int g, float (&sc)[CPW]) const {
    const int row = 32 * g + 4 * (r & 7);
    auto fetch = [&](int src, uint32_t v) {
      return (uint32_t)__builtin_amdgcn_ds_bpermute(src * 4, (int)v);
    };
    auto expo = [&](uint32_t v, int byte, bool ok) {
      const uint32_t e = __builtin_rotateright32(v, (uint32_t)(8 * byte + 9) & 31u);
      return __uint_as_float(ok ? e : 0x3f800000u);
    };
    if constexpr (Slot<CPW, WIDE>::kPairs) {
      sc[0] = expo(fetch(row + (piece >> 1), o.s[0]), piece & 1, in[0]);
    } else {
#pragma unroll
      for (int j = 0; j < CPW; ++j) {
        // WIDE: byte 8j + piece of the slice; else byte sfirst + piece of lane j's 8
        constexpr int kPer = WIDE ? 2 * CPW : 8;
        const int b = WIDE ? 8 * j + piece : sfirst[j] + piece;
        const int src = row + (WIDE ? b / kPer : j), byte = b % kPer;
        uint32_t v = fetch(src, o.s[0]);
        if constexpr (kPer == 8) {
          const uint32_t hi = fetch(src, o.s[1]);
          v = byte >= 4 ? hi : v;
        }
        sc[j] = expo(v, byte & 3, in[j]);
      }
    }
  }
};

__device__ __forceinline__ uint32_t word4(const uint4& v, int m) {
  return m == 0 ? v.x : (m == 1 ? v.y : (m == 2 ? v.z : v.w));
}

// ---- gate/up ----------------------------------------------------------------

struct Shared {
  int key[kMaxPicks];     // expert id of a pick that has a row, else -1
  float w[kMaxPicks];
  int upos[kMaxPicks];    // of a first pick: its expert's place among the distinct ones
  int row[kMaxPicks], mask[kMaxPicks], base[kMaxPicks];
  float wsum[kMaxPicks];  // per h row: the token's router weight for the expert
  int list[kMaxPicks];    // experts in device banks, then the ones in host banks
  int part[kWaves];
  int n_u, n_dev;
};

// Exclusive prefix over the workgroup's threads of v; all threads call it.
__device__ __forceinline__ int block_prefix(int v, int* part, int& total) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d, 64);
    if (lane >= d) s += o;
  }
  __syncthreads();  // part may still be read from an earlier call
  if (lane == 63) part[wv] = s;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    before += i < wv ? part[i] : 0;
    total += part[i];
  }
  return before + s - v;
}

// The step's distinct experts, their tokens and their h rows. Thread s is pick
// s. Returns whether this thread's pick has no row in a bank.
__device__ void build_tables(const FewArgs& a, Shared& L) {
  const int n = a.T * a.k, s = threadIdx.x;
  int id = -1, m = 0;
  bool ok = false;
  if (s < n) {
    id = a.ids[s];
    L.w[s] = a.w[s];
    if ((uint32_t)id < (uint32_t)a.E) {
      m = a.row_map[id];
      ok = m >= 0 ? m < a.hot.n_rows : -1 - m < a.cold.n_rows;
    }
  }
  L.key[s] = ok ? id : -1;
  const int bad = __syncthreads_count(s < n && !ok);
  if (blockIdx.x == 0) {
    if (s == 0) *a.n_invalid = bad;
    if (a.counts && (uint32_t)id < (uint32_t)a.E && s < n)
      __hip_atomic_fetch_add(&a.counts[id], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  int first = s;  // earliest pick of the same expert
  if (ok) {
    for (int p = (s & ~3) - 4; p >= 0; p -= 4) {
      const int4 v = *reinterpret_cast<const int4*>(&L.key[p]);
      first = v.w == id ? p + 3 : first;
      first = v.z == id ? p + 2 : first;
      first = v.y == id ? p + 1 : first;
      first = v.x == id ? p : first;
    }
    for (int p = s - 1; p >= (s & ~3); --p)
      if (first >= (s & ~3) && L.key[p] == id) first = p;
  }
  const bool lead = ok && first == s;
  int n_u;
  const int u0 = block_prefix(lead ? 1 : 0, L.part, n_u);
  if (lead) {
    L.row[u0] = m;
    L.mask[u0] = 0;
    L.upos[s] = u0;
  }
  __syncthreads();
  int u = 0;
  const int t = s / a.k;
  if (ok) {
    u = L.upos[first];
    atomicOr(&L.mask[u], 1 << t);
  }
  __syncthreads();
  int rows;
  const int mk = s < n_u ? L.mask[s] : 0;
  const int b0 = block_prefix(__popc(mk), L.part, rows);
  if (s < n_u) L.base[s] = b0;
  // device-bank experts first, each kind in order
  const int code = s < n_u ? L.row[s] : 0;
  const bool host = s < n_u && (code >= 0 ? a.hot.host : a.cold.host);
  int n_host;
  const int h0 = block_prefix(host ? 1 : 0, L.part, n_host);
  if (s < n_u) L.list[host ? n_u - n_host + h0 : s - h0] = s;
  if (s == 0) {
    L.n_u = n_u;
    L.n_dev = n_u - n_host;
  }
  __syncthreads();
  if (ok) {
    // the token's weight for this expert: its picks of it, in order
    bool mine = true;
    float sum = 0.0f;
    for (int p = t * a.k; p < (t + 1) * a.k; ++p)
      if (L.key[p] == id) {
        if (p < s) mine = false;
        sum += L.w[p];
      }
    if (mine) L.wsum[L.base[u] + __popc(L.mask[u] & ((1 << t) - 1))] = sum;
  }
  __syncthreads();
}

// Adds the partial sums of item `it` (o: this lane's, 64 apart; in their order)
// and writes its 8 values of h for each token that picked the expert. One
// wavefront.
template <int SETS>
__device__ __forceinline__ void write_h(const FewArgs& a, const Shared& L, int it, int ks,
                                        const float* o, uint16_t* h) {
  const int lane = threadIdx.x & 63, per = a.I / 8;
  const int li = it / per, i0 = (it - li * per) * 8;
  const int u = L.list[li];
  const int mask = L.mask[u], base = L.base[u];
#pragma unroll
  for (int st = 0; st < SETS; ++st) {
    float g = 0.0f, up = 0.0f;
    auto add = [&](int p) {
      g += o[(st * 2 * ks + p) * 64];
      up += o[((SETS + st) * 2 * ks + p) * 64];
    };
    if (ks == kWaves) {
#pragma unroll
      for (int p = 0; p < 2 * kWaves; ++p) add(p);
    } else {
      for (int p = 0; p < 2 * ks; ++p) add(p);
    }
    const int t = st * 8 + (lane >> 3);
    if ((mask >> t) & 1) {
      const int rw = base + __popc(mask & ((1 << t) - 1));
      h[(size_t)rw * a.I + i0 + (lane & 7)] =
          (uint16_t)f32_to_bf16_bits(silu_f32(g) * up * L.wsum[rw]);
    }
  }
}

// Experts in pinned host memory are read by kHostBlocks workgroups, the others
// stream the device banks beside them. The host link wants long contiguous
// reads (see ffn_host.hip): an item's 8 gate and 8 up rows are two contiguous
// blocks, copied in linear order through registers into LDS while the last item
// is multiplied out of it, instead of 8 rows x 128 bytes per load (one expert
// of 12.5 MB beside 35 in HBM: 315 us in place, 230 us so; the step with 4, 8, 16
// and 32 workgroups for it 423, 396, 403 and 396 us).
constexpr int kHostBlocks = 8;
constexpr int kHostVecs = kMaxH / 2 / 512;  // 16-byte pieces per thread and item

// Multiplies items [g0, g1) (list entries from n_dev on) of host experts; every
// product and sum as in the device path below, so the bits are the same.
template <int CPW, int SETS, bool WIDE>
__device__ void host_gate_up(const FewArgs& a, const Shared& L, int g0, int g1,
                             const Lane<CPW, WIDE>& ln, const bf16x8 (&xb)[SETS][CPW][4],
                             int slice, bool active, int ks, float* red, unsigned char* wl,
                             uint16_t* h) {
  const int H = a.H, I = a.I, tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int per = I / 8, wrb = H / 2, srb = H / 32;
  const int half = wrb / 2, shalf = srb / 2;  // pieces of 8 rows of weights, of scales
  unsigned char* sl = wl + 16 * wrb;          // the 16 rows' scale bytes
  u32x4 v[kHostVecs], sv;
  auto issue = [&](int it) {
    const int li = it / per, i0 = (it - li * per) * 8;
    const int code = __builtin_amdgcn_readfirstlane(L.row[L.list[li]]);
    const FewBank& b = code >= 0 ? a.hot : a.cold;
    const size_t r0 = (size_t)(uint32_t)(code >= 0 ? code : -1 - code) * 2 * I + i0, r1 = r0 + I;
    const u32x4* wg = reinterpret_cast<const u32x4*>(b.w13 + r0 * wrb);
    const u32x4* wu = reinterpret_cast<const u32x4*>(b.w13 + r1 * wrb);
#pragma unroll
    for (int n = 0; n < kHostVecs; ++n) {
      const int p = n * kThreads + tid;
      if (n * kThreads < 2 * half) {  // uniform
        const int c = min(p, 2 * half - 1);
        v[n] = c < half ? wg[c] : wu[c - half];
      }
    }
    const int c = min(tid, 2 * shalf - 1);
    sv = c < shalf ? reinterpret_cast<const u32x4*>(b.s13 + r0 * srb)[c]
                   : reinterpret_cast<const u32x4*>(b.s13 + r1 * srb)[c - shalf];
  };
  issue(g0);
  for (int it = g0; it < g1; ++it) {
#pragma unroll
    for (int n = 0; n < kHostVecs; ++n)
      if (n * kThreads < 2 * half)
        *reinterpret_cast<u32x4*>(wl + 16 * min(n * kThreads + tid, 2 * half - 1)) = v[n];
    *reinterpret_cast<u32x4*>(sl + 16 * min(tid, 2 * shalf - 1)) = sv;
    if (it + 1 < g1) issue(it + 1);
    lds_barrier();
    f32x4 acc[2][SETS];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int st = 0; st < SETS; ++st) acc[g][st] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      uint4 w[2];
      float sc[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        w[g] = *reinterpret_cast<const uint4*>(wl + 8 * g * wrb + ln.woff[j]);
        const int row = (ln.r & 7) + 8 * g, b = (slice * CPW + j) * 8 + ln.piece;
        const uint32_t e = sl[row * srb + (ln.in[j] ? b : 0)];
        sc[g] = __uint_as_float((ln.in[j] ? e : 127u) << 23);  // see Lane::scales
      }
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const bf16x8 av = dequant8(word4(w[g], m), sc[g]);
#pragma unroll
          for (int st = 0; st < SETS; ++st)
            acc[g][st] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, xb[st][j][m], acc[g][st], 0,
                                                                 0, 0);
        }
    }
    if (active && (ln.r >= 8) == (ln.q >= 2)) {
      float* o = red + (2 * slice + (ln.r >= 8)) * 64 + (ln.r & 7) * 8 + (ln.q & 1) * 4;
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int st = 0; st < SETS; ++st)
          *reinterpret_cast<f32x4*>(o + (g * SETS + st) * 2 * ks * 64) = acc[g][st];
    }
    lds_barrier();  // the item's weights have been read, its partial sums written
    if (wv == it % kWaves) write_h<SETS>(a, L, it, ks, red + lane, h);
  }
}

template <int CPW, int SETS, int R, bool WIDE>
__global__ __launch_bounds__(kThreads, 2) void few_gate_up(FewArgs a) {
  extern __shared__ __align__(16) float red[];  // [4][SUB][2 groups][SETS][2 KS][8][8]
  __shared__ __align__(16) Shared L;
  const int H = a.H, I = a.I, T = a.T;
  const Cut cut = gate_up_cut(H);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ks = cut.ks, nsub = cut.sub;
  const int slice = wv % ks, sub = wv / ks;
  const bool active = sub < nsub;
  Lane<CPW, WIDE> ln;
  ln.init(lane, slice, H);

  // this wavefront's slice of x as B operands: column c holds token c (first
  // halves) or c - 8 (second halves) of its set
  bf16x8 xb[SETS][CPW][4];
#pragma unroll
  for (int st = 0; st < SETS; ++st) {
    const int t = st * 8 + (ln.r & 7);
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      const int e0 = (slice * CPW + j) * kChunkElems + (ln.r >= 8 ? 128 : 0) + 32 * ln.q;
      const bool in = t < T && e0 < H;  // H is a multiple of 64: 32 elements at once
      const uint4* p = reinterpret_cast<const uint4*>(a.x + (size_t)(t < T ? t : 0) * H +
                                                      (e0 < H ? e0 : 0));
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint4 v = p[m];
        xb[st][j][m] = __builtin_bit_cast(
            bf16x8, make_uint4(in ? v.x : 0u, in ? v.y : 0u, in ? v.z : 0u, in ? v.w : 0u));
      }
    }
  }

  build_tables(a, L);
  const int n_u = __builtin_amdgcn_readfirstlane(L.n_u);
  const int n_dev = __builtin_amdgcn_readfirstlane(L.n_dev);
  Tables* tab = static_cast<Tables*>(a.workspace);
  uint16_t* h = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.workspace) + kTableBytes);
  if (blockIdx.x == 0) {
    if (tid == 0) tab->n_u = n_u;
    if (tid < n_u) {
      tab->row[tid] = L.row[tid];
      tab->mask[tid] = L.mask[tid];
      tab->base[tid] = L.base[tid];
    }
  }

  // this workgroup's run of items (list entry, 8 rows of I): [g0, g1)
  const int per = I / 8;
  const int hb = n_dev < n_u ? min(kHostBlocks, (int)gridDim.x - 1) : 0;
  const bool on_host = (int)blockIdx.x < hb;
  const uint32_t n = (uint32_t)(on_host ? n_u - n_dev : n_dev) * per;  // < 2^19
  const uint32_t blocks = on_host ? hb : gridDim.x - hb;
  const uint32_t blk = on_host ? blockIdx.x : blockIdx.x - hb;
  const int first = on_host ? n_dev * per : 0;
  const int g0 = first + (int)(n * blk / blocks), g1 = first + (int)(n * (blk + 1) / blocks);
  if (g0 >= g1) return;  // the whole workgroup
  if (on_host) {
    unsigned char* wl = reinterpret_cast<unsigned char*>(red) +
                        (size_t)4 * nsub * 2 * SETS * 2 * ks * 64 * sizeof(float);
    host_gate_up<CPW, SETS, WIDE>(a, L, g0, g1, ln, xb, slice, active && sub == 0, ks, red, wl, h);
    return;
  }
  const int steps = (g1 - g0 + nsub - 1) / nsub;

  const size_t wrb = H / 2, srb = H / 32;
  // this lane's scale row of an item, from its first gate row
  const uint32_t srow_off = ((ln.srow & 7) + (ln.srow >= 8 ? (uint32_t)I : 0u)) * (uint32_t)srb;
  // The prefetch cursor: this wavefront's next item, its place in its expert
  // and its first gate row. Past the run's end it stays on the first rows of a
  // device bank (the same for every wavefront, so they stay in the L2), which
  // keeps the stream unconditional.
  const uint8_t *cw, *cs;
  int c_it = g0 + sub, c_li, c_ib;
  auto enter = [&]() {  // expert c_li, rows 8 c_ib
    const int code = __builtin_amdgcn_readfirstlane(L.row[L.list[c_li]]);
    const FewBank& b = code >= 0 ? a.hot : a.cold;
    const size_t r0 = (size_t)(uint32_t)(code >= 0 ? code : -1 - code) * 2 * I + 8 * c_ib;
    cw = b.w13 + r0 * wrb;
    cs = b.s13 + r0 * srb;
  };
  auto park = [&]() {
    const bool hot = (a.hot.n_rows > 0 && !a.hot.host) || a.cold.n_rows == 0;
    cw = hot ? a.hot.w13 : a.cold.w13;
    cs = hot ? a.hot.s13 : a.cold.s13;
  };
  c_li = c_it / per;
  c_ib = c_it - c_li * per;
  if (c_it < g1 && active)
    enter();
  else
    park();
  auto advance = [&]() {
    c_it += nsub;
    c_ib += nsub;
    if (c_it >= g1 || !active) {
      park();
    } else if (c_ib >= per) {
      do {
        c_ib -= per;
        ++c_li;
      } while (c_ib >= per);
      enter();
    } else {
      cw += (size_t)(8 * nsub) * wrb;
      cs += (size_t)(8 * nsub) * srb;
    }
  };
  Slot<CPW, WIDE> ring[R];
  auto issue = [&](Slot<CPW, WIDE>& o) {
    ln.template load<WIDE>(o, cw, cw + (size_t)I * wrb, cs, srow_off);
    __builtin_amdgcn_sched_barrier(0);
    advance();
  };
  // floats of one (buffer, sub): [group][set][partial][token][row]
  const int per_sub = 2 * SETS * 2 * ks * 64;
  const bool diag = (ln.r >= 8) == (ln.q >= 2) && active;
  const int red_off = (2 * slice + (ln.r >= 8)) * 64 + (ln.r & 7) * 8 + (ln.q & 1) * 4;

#pragma unroll
  for (int u = 0; u < R; ++u) issue(ring[u]);

  // Whole turns of the ring: leaving the loop inside a turn made the compiler
  // wait for nearly every load in flight once per turn.
  static_assert(R % 2 == 0, "steps in pairs");
  for (int s0 = 0; s0 < steps; s0 += R) {
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const int step = s0 + u;
      const bool live = step < steps;
      f32x4 acc[2][SETS];
      if (live) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int st = 0; st < SETS; ++st) acc[g][st] = f32x4{0.f, 0.f, 0.f, 0.f};
        float sc[2][CPW];
        ln.scales(ring[u], 0, sc[0]);
        ln.scales(ring[u], 1, sc[1]);
#pragma unroll
        for (int j = 0; j < CPW; ++j) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const bf16x8 av = dequant8(word4(ring[u].w[g][j], m), sc[g][j]);
#pragma unroll
              for (int st = 0; st < SETS; ++st)
                acc[g][st] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, xb[st][j][m],
                                                                     acc[g][st], 0, 0, 0);
            }
        }
      }
      issue(ring[u]);
      // lane (c, q) holds rows 4q .. 4q+3 of column c: keep the diagonal blocks
      if (live && diag) {
        float* o = red + (size_t)((step & 3) * nsub + sub) * per_sub + red_off;
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int st = 0; st < SETS; ++st)
            *reinterpret_cast<f32x4*>(o + (g * SETS + st) * 2 * ks * 64) = acc[g][st];
      }
      if ((u & 1) == 0 || step - 1 >= steps) continue;
      // Every second step: one wavefront per item, each in turn, adds the
      // partial sums (in their order) and writes h; the others go on. A buffer is
      // written again four steps later, past the next barrier, which that
      // wavefront reaches only after its reads.
      lds_barrier();
      for (int n = 0; n < 2 * nsub; ++n) {
        const int st = step - 1 + (n >= nsub), sb = n >= nsub ? n - nsub : n;
        const int it = g0 + st * nsub + sb;
        if (st >= steps || it >= g1 || (it - g0) % kWaves != wv) continue;
        write_h<SETS>(a, L, it, ks, red + (size_t)((st & 3) * nsub + sb) * per_sub + lane, h);
      }
    }
  }
}

// ---- down -------------------------------------------------------------------
//
// Workgroup b owns 16 columns of out and walks every distinct expert, so the
// sum over a token's experts stays in its accumulators. The wavefronts of a row
// take every SUB-th expert. The h rows are staged in LDS in phases of as many
// whole experts as fit, 16-byte granule g of staged row s at g ^ (s & 7); the
// columns of tokens that did not pick the expert read a row of zeros, and their
// results are left out of the sum (an expert with infinite or NaN weights
// reaches its own tokens only). An expert's weights are
// requested as soon as those of the wavefront's last one are multiplied; more in
// flight was no faster (two experts 50.2 us, three 51.8 against 47.7 at 7
// tokens): rows of 1440 bytes share lines, which the L2 then drops between
// their two reads. B operands straight from memory instead of staged rows cost
// 16 more loads per expert and wavefront (49.4 us at 7 tokens, 112 against 96 at
// 16).
//
// An expert in host memory: a wavefront's slice of 16 rows x CPW lines is loaded
// in linear order, so that a load reads CPW consecutive lines of a row, and
// brought into operand order through LDS of the wavefront's own (one such expert
// beside 35 in HBM: 181 us with the operand order's loads of 8 rows x one line,
// 163 us so).

constexpr size_t kDownLds = 150 * 1024;  // staged rows and the row of zeros

// LINEAR: host experts through LDS, as above.
template <int CPW, int SETS, bool LINEAR>
__global__ __launch_bounds__(kThreads, 2) void few_down(FewArgs a, int max_rows) {
  // [max_rows + 1][512 CPW KS bytes], then if LINEAR per wavefront [16][128 CPW]
  extern __shared__ __align__(16) unsigned char hs[];
  __shared__ int l_row[kMaxPicks], l_mask[kMaxPicks], l_base[kMaxPicks + 1];
  const int H = a.H, I = a.I, T = a.T;
  const Cut cut = down_cut(I);
  const int tid = threadIdx.x, lane = tid & 63, threads = blockDim.x;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ks = cut.ks, nsub = cut.sub;
  const int slice = wv % ks, sub = wv / ks;
  Lane<CPW, false> ln;
  ln.init(lane, slice, I);
  const Tables* tab = static_cast<const Tables*>(a.workspace);
  const uint16_t* h =
      reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(a.workspace) + kTableBytes);
  const int n_u = __builtin_amdgcn_readfirstlane(tab->n_u);
  for (int i = tid; i < T * a.k; i += threads) {
    const int row = tab->row[i], mask = tab->mask[i], base = tab->base[i];
    if (i < n_u) {
      l_row[i] = row;
      l_mask[i] = mask;
      l_base[i] = base;
      if (i == n_u - 1) l_base[n_u] = base + __popc(mask);
    }
  }
  const int row_bytes = 512 * CPW * ks;  // of a staged row
  for (int i = tid; i < row_bytes / 16; i += threads)
    *reinterpret_cast<uint4*>(hs + (size_t)max_rows * row_bytes + 16 * i) = make_uint4(0, 0, 0, 0);
  __syncthreads();

  const int o0 = blockIdx.x * 16;
  const size_t wrb = I / 2, srb = I / 32;
  const uint32_t srow_off = (uint32_t)ln.srow * (uint32_t)srb;
  // the slice's pieces in linear order: piece i = 64 n + lane of 16 rows x 8 CPW
  unsigned char* own = hs + (size_t)(max_rows + 1) * row_bytes + wv * 2048 * CPW;
  uint32_t loff[2][CPW];
#pragma unroll
  for (int n = 0; n < 2 * CPW; ++n) {
    const int i = 64 * n + lane, row = i / (8 * CPW);
    const uint32_t b = 16u * (uint32_t)(slice * CPW * 8 + i % (8 * CPW));
    loff[n / CPW][n % CPW] = (uint32_t)row * (uint32_t)wrb + (b < wrb ? b : 0u);
  }
  Slot<CPW, false> next;
  // the expert u's; past the last expert the first rows of a device bank (see
  // few_gate_up)
  auto issue = [&](Slot<CPW, false>& o, int u) {
    const bool live = u < n_u;
    const int code = __builtin_amdgcn_readfirstlane(l_row[live ? u : 0]);
    const bool hot = live ? code >= 0 : (a.hot.n_rows > 0 && !a.hot.host) || a.cold.n_rows == 0;
    const uint8_t* w2 = hot ? a.hot.w2 : a.cold.w2;
    const uint8_t* s2 = hot ? a.hot.s2 : a.cold.s2;
    const uint32_t row = live ? (uint32_t)(code >= 0 ? code : -1 - code) : 0u;
    const size_t r0 = (size_t)row * H + (live ? o0 : 0);
    const bool lin = LINEAR && live && (hot ? a.hot.host : a.cold.host);
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int j = 0; j < CPW; ++j)
        o.w[g][j] = *reinterpret_cast<const uint4*>(w2 + (r0 + (lin ? 0 : 8 * g)) * wrb +
                                                    (lin ? loff[g][j] : ln.woff[j]));
    ln.load_scales(o, s2 + r0 * srb + srow_off);
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x4 acc[2][SETS];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int st = 0; st < SETS; ++st) acc[g][st] = f32x4{0.f, 0.f, 0.f, 0.f};

  int ph0 = 0, ph_end = 0;  // first staged h row; first expert past the phase
  // The next phase: every wavefront calls it once per phase, in order.
  auto next_phase = [&]() {
    lds_barrier();  // the last phase's rows have been read
    const int u0 = ph_end;
    ph0 = __builtin_amdgcn_readfirstlane(l_base[u0]);
    while (ph_end < n_u && __builtin_amdgcn_readfirstlane(l_base[ph_end + 1]) - ph0 <= max_rows)
      ++ph_end;
    const int nr = __builtin_amdgcn_readfirstlane(l_base[ph_end]) - ph0;
    const uint32_t per = 32 * CPW * ks, n = nr * per;  // granules
    constexpr int kB = 8;                              // per thread per batch
    for (uint32_t i0 = 0; i0 < n; i0 += kB * threads) {
      u32x4 v[kB];
      uint32_t off[kB];
      int dst[kB];
      uint32_t past = 0;  // bit b: granule b lies past the end of the axis
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const uint32_t i = min(i0 + b * threads + tid, n - 1);
        const uint32_t s = i / per, g = i - s * per;
        const bool in = g * 8 < (uint32_t)I;
        past |= (in ? 0u : 1u) << b;
        off[b] = ((ph0 + s) * (uint32_t)I + (in ? g * 8 : 0u)) * 2u;
        dst[b] = (int)(s * row_bytes + 16 * (g ^ (s & 7)));
      }
      // Loads and their wait in one block: as ordinary loads under this branch
      // they made the compiler wait for every weight in flight at each expert.
      asm volatile(
          "global_load_dwordx4 %0, %8, %16\n\tglobal_load_dwordx4 %1, %9, %16\n\t"
          "global_load_dwordx4 %2, %10, %16\n\tglobal_load_dwordx4 %3, %11, %16\n\t"
          "global_load_dwordx4 %4, %12, %16\n\tglobal_load_dwordx4 %5, %13, %16\n\t"
          "global_load_dwordx4 %6, %14, %16\n\tglobal_load_dwordx4 %7, %15, %16\n\t"
          "s_waitcnt vmcnt(0)"
          : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]),
            "=&v"(v[6]), "=&v"(v[7])
          : "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "v"(off[4]), "v"(off[5]),
            "v"(off[6]), "v"(off[7]), "s"(h)
          : "memory");
#pragma unroll
      for (int b = 0; b < kB; ++b)
        *reinterpret_cast<u32x4*>(hs + dst[b]) = (past >> b) & 1u ? u32x4{0, 0, 0, 0} : v[b];
    }
    lds_barrier();
  };

  if (sub < n_u) issue(next, sub);
  for (int u = sub; u < n_u; u += nsub) {
    while (u >= ph_end) next_phase();
    const int mask = l_mask[u], base = l_base[u] - ph0;
    f32x4 d[2][SETS];
    const unsigned char* hp[SETS];  // this column's staged row
    int sw[SETS];
    bool has[SETS];
#pragma unroll
    for (int st = 0; st < SETS; ++st) {
      const int t = st * 8 + (ln.r & 7);
      has[st] = (mask >> t) & 1;
      const int s = has[st] ? base + __popc(mask & ((1 << t) - 1)) : max_rows;
      hp[st] = hs + s * row_bytes + 512 * CPW * slice;
      sw[st] = 16 * ((ln.r >= 8 ? 16 : 0) + ((4 * ln.q) ^ (has[st] ? s & 7 : 0)));
#pragma unroll
      for (int g = 0; g < 2; ++g) d[g][st] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if constexpr (LINEAR) {
      const int code = __builtin_amdgcn_readfirstlane(l_row[u]);
      if (code >= 0 ? a.hot.host : a.cold.host) {
#pragma unroll
        for (int n = 0; n < 2 * CPW; ++n)
          *reinterpret_cast<uint4*>(own + 16 * (64 * n + lane)) = next.w[n / CPW][n % CPW];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int j = 0; j < CPW; ++j)
            next.w[g][j] = *reinterpret_cast<const uint4*>(
                own + 16 * (((ln.r & 7) + 8 * g) * 8 * CPW + 8 * j + ln.piece));
      }
    }
    float sc[2][CPW];
    ln.scales(next, 0, sc[0]);
    ln.scales(next, 1, sc[1]);
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        bf16x8 bv[SETS];
#pragma unroll
        for (int st = 0; st < SETS; ++st)  // granule 32j + half + (4q + m ^ s & 7)
          bv[st] = *reinterpret_cast<const bf16x8*>(hp[st] + 512 * j + (sw[st] ^ (16 * m)));
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const bf16x8 av = dequant8(word4(next.w[g][j], m), sc[g][j]);
#pragma unroll
          for (int st = 0; st < SETS; ++st)
            d[g][st] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bv[st], d[g][st], 0, 0, 0);
        }
      }
    }
    issue(next, u + nsub);
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int st = 0; st < SETS; ++st)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[g][st][e] += has[st] ? d[g][st][e] : 0.0f;
  }
  while (ph_end < n_u) next_phase();

  // sum of the wavefronts' partial sums, in their order, and the one rounding
  __syncthreads();
  float* red = reinterpret_cast<float*>(hs);  // [wave][half][set][token][16]
  if ((ln.r >= 8) == (ln.q >= 2)) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int st = 0; st < SETS; ++st)
        *reinterpret_cast<f32x4*>(red + (((wv * 2 + (ln.r >= 8)) * SETS + st) * 8 + (ln.r & 7)) * 16 +
                                  8 * g + 4 * (ln.q & 1)) = acc[g][st];
  }
  __syncthreads();
  const int waves = threads >> 6;
  for (int i = tid; i < T * 16; i += threads) {
    const int t = i / 16, o = i % 16;
    float s = 0.0f;
    for (int p = 0; p < 2 * waves; ++p) s += red[((p * SETS + t / 8) * 8 + (t & 7)) * 16 + o];
    a.out[(size_t)t * H + o0 + o] = (uint16_t)f32_to_bf16_bits(s);
  }
}

template <int CPW, int SETS, int R, bool WIDE>
hipError_t go_gate_up(const FewArgs& a, hipStream_t stream) {
  const Cut c = gate_up_cut(a.H);
  size_t lds = (size_t)4 * c.sub * 2 * SETS * 2 * c.ks * 64 * sizeof(float);
  if (a.hot.host || a.cold.host) lds += (size_t)16 * (a.H / 2 + a.H / 32);  // an item's weights
  hipLaunchKernelGGL((few_gate_up<CPW, SETS, R, WIDE>), dim3(device_cus()), dim3(kThreads), lds,
                     stream, a);
  return hipGetLastError();
}

template <int CPW, int SETS>
hipError_t go_down(const FewArgs& a, hipStream_t stream) {
  const Cut c = down_cut(a.I);
  const int waves = c.ks * c.sub;
  const size_t row = (size_t)512 * CPW * c.ks;
  // host experts: room for the wavefronts' linear slices, where the h rows of
  // one expert still fit beside them
  const size_t own = (size_t)waves * 2048 * CPW;
  const bool linear = (a.hot.host || a.cold.host) &&
                      (size_t)(std::min(a.T, MOE_FEW_MAX_TOKENS) + 1) * row + own <= kDownLds;
  const size_t room = kDownLds - (linear ? own : 0);
  const int max_rows = (int)std::min<size_t>(room / row - 1, (size_t)a.T * a.k);
  const size_t lds = std::max((size_t)(max_rows + 1) * row + (linear ? own : 0),
                              (size_t)waves * 2 * SETS * 8 * 16 * sizeof(float));
  auto kern = linear ? few_down<CPW, SETS, true> : few_down<CPW, SETS, false>;
  hipLaunchKernelGGL(kern, dim3(a.H / 16), dim3(64 * waves), lds, stream, a, max_rows);
  return hipGetLastError();
}

// R ring slots, 32 CPW KB of weights each and CU. At H = 4096 (CPW = 2), 2 slots
// take 21.3, 78.4 and 158 us for 1, 7 and 16 tokens, 4 slots 24.2, 83.1 and 154
// (traces of one build range over 154-174 us at 16 tokens).
template <int CPW, int R, bool WIDE>
hipError_t gate_up_sets(const FewArgs& a, hipStream_t s) {
  return a.T <= 8 ? go_gate_up<CPW, 1, R, WIDE>(a, s) : go_gate_up<CPW, 2, R, WIDE>(a, s);
}
template <int CPW>
hipError_t down_sets(const FewArgs& a, hipStream_t s) {
  return a.T <= 8 ? go_down<CPW, 1>(a, s) : go_down<CPW, 2>(a, s);
}

}  // namespace

bool layer_few_fits(int T, int k, int H, int I) {
  return T <= MOE_FEW_MAX_TOKENS && k <= MOE_MAX_TOPK && H <= kMaxH && I <= kMaxI;
}

size_t layer_few_workspace_bytes(int T, int k, int I) {
  return kTableBytes + (size_t)T * k * I * sizeof(uint16_t);
}

hipError_t launch_layer_few(const FewArgs& a, hipStream_t s) {
  const Cut cg = gate_up_cut(a.H), cd = down_cut(a.I);
  const bool wide = a.H % (kChunkElems * cg.cpw * cg.ks) == 0;  // no slice ends past the axis
  hipError_t e;
  if (cg.cpw == 1)
    e = gate_up_sets<1, 4, false>(a, s);
  else if (cg.cpw == 2)
    e = wide ? gate_up_sets<2, 2, true>(a, s) : gate_up_sets<2, 2, false>(a, s);
  else
    e = wide ? gate_up_sets<4, 2, true>(a, s) : gate_up_sets<4, 2, false>(a, s);
  if (e != hipSuccess) return e;
  switch (cd.cpw) {
    case 1: return down_sets<1>(a, s);
    case 2: return down_sets<2>(a, s);
    case 3: return down_sets<3>(a, s);
    default: return down_sets<4>(a, s);
  }
}

}  // namespace moe
