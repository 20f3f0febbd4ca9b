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

}  // namespace moe
