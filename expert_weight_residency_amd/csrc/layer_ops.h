// Declarations of the operators around the residency split: the router's top-k
// gate, the whole layer for a few tokens, and the 8-bit integer products.
#pragma once

#include "internal.h"

namespace moe {

// Element types of the entry points that take more than bf16 (MOE_DTYPE_*).
__host__ __device__ inline int dtype_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
inline bool dtype_known(int dtype) {
  return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F16 || dtype == MOE_DTYPE_F32;
}

// Device-visible addresses of a bank's four tensors; `align` holds each
// tensor's required alignment. MOE_OK, or an error with its message set.
int bank_ptrs(const moe_bank* b, const size_t align[4], const uint8_t* out[4]);

inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

inline int succeed() { return set_error(MOE_OK, "%s", ""); }

// Router logits -> top-k ids and weights (gate_topk.hip).
hipError_t launch_topk_gate(const void* logits, int dtype, int64_t ld, int T, int E, int k,
                            int norm, int32_t* ids, float* w, hipStream_t stream);

// The whole layer for at most MOE_FEW_MAX_TOKENS tokens (layer_few.hip).
struct FewBank {
  const uint8_t *w13, *s13, *w2, *s2;
  int n_rows;
  int host;  // the weights are in pinned host memory
};
struct FewArgs {
  FewBank hot, cold;
  const int32_t* row_map;
  const uint16_t* x;
  const int32_t* ids;
  const float* w;
  int T, k, E, H, I;
  int32_t* counts;  // null: this step does not count
  int32_t* n_invalid;
  void* workspace;
  uint16_t* out;
};
bool layer_few_fits(int T, int k, int H, int I);
size_t layer_few_workspace_bytes(int T, int k, int I);
hipError_t launch_layer_few(const FewArgs& a, hipStream_t stream);

// Rows to 8-bit integers with a scale each (quantize_i8.hip): rows 0 .. rows-1
// of x, or with a split the slots it lists (rows = T*k then bounds the launch).
hipError_t launch_quantize_rows(const void* x, int dtype, int64_t ld, int rows, int K,
                                const moe_split* split, int8_t* q, float* scale,
                                hipStream_t stream);

// Products of 8-bit rows: y[r][n] = sa[r] * sw[n] * sum_k a[r][k] w[n][k].
// Dense (split null): rows 0 .. M-1 and one weight matrix. Grouped: the slots
// of each active row of the split against that row's matrix; activation row
// slot / k (by_token) or slot, output row slot. With `gate_up` the matrix has 2N
// rows, gate then up, and y is fp32 silu(gate) * up.
struct I8Args {
  const int8_t* a;
  int64_t lda;
  const float* sa;
  const int8_t* w;
  const float* sw;
  int M, N, K;  // grouped: M = T * k, a bound on the slots
  const int32_t *n_active, *active_rows, *row_off, *slots;  // null: dense
  int n_rows;   // grouped: rows of the bank
  int k, by_token, gate_up;
  void* y;
  int dtype;
  int64_t ldy;
};
// Whether the launch stays below 2^32 work items (checked before anything of a
// call is enqueued).
bool gemm_i8_fits(const I8Args& a);
hipError_t launch_gemm_i8(const I8Args& a, hipStream_t stream);

// Rows to E4M3 with a scale per 128 elements (quantize_f8.hip); rows and split as
// in launch_quantize_rows.
hipError_t launch_quantize_f8(const void* x, int dtype, int64_t ld, int rows, int K,
                              const moe_split* split, uint8_t* q, float* scale,
                              hipStream_t stream);

// Products of E4M3 rows (gemm_f8.hip): y[r][n] = sum over 128-blocks b of
// sa[r][b] * sw[n / 128][b] * sum over k in b of a[r][k] w[n][k]. Dense, grouped
// and gate_up as in I8Args; with gate_up the scales of up's blocks follow gate's.
struct F8Args {
  const uint8_t* a;
  int64_t lda;
  const float* sa;
  const uint8_t* w;
  const float* sw;
  int M, N, K;  // grouped: M = T * k, a bound on the slots
  const int32_t *n_active, *active_rows, *row_off, *slots;  // null: dense
  int n_rows;   // grouped: rows of the bank
  int k, by_token, gate_up;
  void* y;
  int dtype;
  int64_t ldy;
};
bool gemm_f8_fits(const F8Args& a);
hipError_t launch_gemm_f8(const F8Args& a, hipStream_t stream);

inline int f8_blocks(int n) { return (n + MOE_F8_BLOCK - 1) / MOE_F8_BLOCK; }

// Products grouped by expert (grouped_linear.hip): op 0 forward, 1 the input's
// gradient, 2 the weights' gradient. Rows of one expert are the slots that the split
// lists for it; x holds a row per token (by_token = ceil(2^32 / k)) or per slot
// (by_token = 0, also for k = 1), dy, y and dx a row per slot.
struct GroupedArgs {
  int op, elem;  // elem: type of w, x and dy (bf16 or fp16)
  const uint8_t *w, *x, *dy;
  int M, N, K;  // M = T * k, a bound on the slots
  const int32_t *n_active, *active_rows, *row_off, *slots;  // n_active null: no slots
  int n_rows;
  uint32_t by_token;
  void* y;  // y, dx or dw
  int dtype;
  int64_t ldy;
};
bool grouped_fits(const GroupedArgs& a);
hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream);

}  // namespace moe
