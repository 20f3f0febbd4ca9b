// C ABI of the operators around the residency split: argument checks, then
// launches on the caller's stream (see abi.hip).
#include "layer_ops.h"

namespace moe {

int bank_ptrs(const moe_bank* b, const size_t align[4], const uint8_t* out[4]) {
  if (b->on_host != MOE_BANK_DEVICE && b->on_host != MOE_BANK_HOST &&
      b->on_host != MOE_BANK_HOST_WEIGHTS)
    return set_error(MOE_EINVAL, "bank on_host=%d is not MOE_BANK_DEVICE, _HOST or _HOST_WEIGHTS",
                     b->on_host);
  void* const src[4] = {b->w13, b->s13, b->w2, b->s2};
  for (int i = 0; i < 4; ++i) {
    if (!src[i]) return set_error(MOE_EINVAL, "bank tensor %d is NULL", i);
    if (reinterpret_cast<uintptr_t>(src[i]) % align[i])
      return set_error(MOE_EINVAL, "bank tensor %d must be %zu-byte aligned", i, align[i]);
    out[i] = static_cast<const uint8_t*>(src[i]);
    // tensors 0 and 2 are the weights, 1 and 3 the scales
    if (b->on_host == MOE_BANK_HOST || (b->on_host == MOE_BANK_HOST_WEIGHTS && !(i & 1))) {
      void* d = nullptr;
      if (hipHostGetDevicePointer(&d, src[i], 0) != hipSuccess || !d) {
        (void)hipGetLastError();
        return set_error(MOE_EINVAL, "bank tensor %d is not pinned host memory (on_host=%d)", i,
                         b->on_host);
      }
      out[i] = static_cast<const uint8_t*>(d);
    }
  }
  return MOE_OK;
}

}  // namespace moe

namespace {

using moe::set_error;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

extern "C" {

int moe_topk_gate(const void* logits, int dtype, int64_t ld, int T, int E, int k, int norm,
                  int32_t* topk_ids, float* topk_w, void* stream) {
  if (!moe::dtype_known(dtype)) return set_error(MOE_EINVAL, "dtype=%d unknown", dtype);
  if (norm != MOE_GATE_NORM_PICKS && norm != MOE_GATE_NORM_ALL)
    return set_error(MOE_EINVAL, "norm=%d unknown", norm);
  if (T < 0) return set_error(MOE_EINVAL, "T=%d must be >= 0", T);
  if (E < 1 || E > MOE_MAX_EXPERTS)
    return set_error(MOE_EINVAL, "E=%d outside [1, %d]", E, MOE_MAX_EXPERTS);
  if (k < 1 || k > MOE_MAX_TOPK || k > E)
    return set_error(MOE_EINVAL, "k=%d outside [1, min(E=%d, %d)]", k, E, MOE_MAX_TOPK);
  if ((int64_t)T * k >= (int64_t)1 << 31) return set_error(MOE_EINVAL, "T*k too large");
  if (ld < E || ld > (int64_t)1 << 31)
    return set_error(MOE_EINVAL, "ld=%lld must be in [E=%d, 2^31]", (long long)ld, E);
  if (T == 0) return moe::succeed();
  if (!logits || !topk_ids || !topk_w)
    return set_error(MOE_EINVAL, "logits, topk_ids and topk_w must not be NULL");
  if (!aligned(logits, moe::dtype_bytes(dtype)) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
    return set_error(MOE_EINVAL, "logits, topk_ids and topk_w must be aligned to their elements");
  const hipError_t e = moe::launch_topk_gate(logits, dtype, ld, T, E, k, norm, topk_ids, topk_w,
                                             static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return set_error(MOE_EHIP, "gate launch: %s", hipGetErrorString(e));
  return moe::succeed();
}

size_t moe_layer_few_workspace_bytes(int T, int k, int H, int I) {
  if (T <= 0 || k <= 0 || H <= 0 || I <= 0 || !moe::layer_few_fits(T, k, H, I)) return 0;
  return moe::layer_few_workspace_bytes(T, k, I);
}

int moe_layer_few_mxfp4(const moe_bank* hot, const moe_bank* cold, const int32_t* row_map, int E,
                        const uint16_t* x, const int32_t* topk_ids, const float* topk_w, int T,
                        int k, int H, int I, int32_t* counts_layer, int count_tmax,
                        int32_t* n_invalid, void* workspace, uint16_t* out, void* stream) {
  if (T < 0) return set_error(MOE_EINVAL, "T=%d must be >= 0", T);
  if (k < 1 || k > MOE_MAX_TOPK)
    return set_error(MOE_EINVAL, "k=%d outside [1, %d]", k, MOE_MAX_TOPK);
  if (E < 1 || E > MOE_MAX_EXPERTS)
    return set_error(MOE_EINVAL, "E=%d outside [1, %d]", E, MOE_MAX_EXPERTS);
  if (H <= 0 || H % 64 || I <= 0 || I % 64)
    return set_error(MOE_EINVAL, "H=%d, I=%d must be positive multiples of 64", H, I);
  if (!moe::layer_few_fits(T, k, H, I))
    return set_error(MOE_ENOTSUP, "T=%d, H=%d, I=%d: at most %d, %d and %d supported", T, H, I,
                     MOE_FEW_MAX_TOKENS, MOE_FEW_MAX_H, MOE_FEW_MAX_I);
  if (!hot || !cold) return set_error(MOE_EINVAL, "hot and cold must not be NULL");
  for (const moe_bank* b : {hot, cold})
    if (b->n_rows < 0 || b->n_rows > MOE_MAX_ROWS)
      return set_error(MOE_EINVAL, "bank rows %d outside [0, %d]", b->n_rows, MOE_MAX_ROWS);
  if (T == 0) return moe::succeed();
  if (!row_map || !x || !topk_ids || !topk_w || !n_invalid || !workspace || !out)
    return set_error(MOE_EINVAL, "row_map, x, topk_ids, topk_w, n_invalid, workspace and out must "
                                 "not be NULL");
  if (!aligned(x, 16) || !aligned(workspace, 16) || !aligned(out, 16))
    return set_error(MOE_EINVAL, "x, workspace and out must be 16-byte aligned");
  const uintptr_t xb = reinterpret_cast<uintptr_t>(x), ob = reinterpret_cast<uintptr_t>(out);
  const size_t nb = (size_t)T * H * 2;
  if (xb < ob + nb && ob < xb + nb) return set_error(MOE_EINVAL, "out must not overlap x");
  moe::FewArgs a = {};
  const size_t align[4] = {16, 16, 16, 16};
  const moe_bank* const src[2] = {hot, cold};
  moe::FewBank* const dst[2] = {&a.hot, &a.cold};
  for (int i = 0; i < 2; ++i) {
    if (src[i]->n_rows == 0) continue;
    const uint8_t* p[4];
    const int rc = moe::bank_ptrs(src[i], align, p);
    if (rc != MOE_OK) return rc;
    *dst[i] = {p[0], p[1], p[2], p[3], src[i]->n_rows, src[i]->on_host != MOE_BANK_DEVICE};
  }
  a.row_map = row_map;
  a.x = x;
  a.ids = topk_ids;
  a.w = topk_w;
  a.T = T;
  a.k = k;
  a.E = E;
  a.H = H;
  a.I = I;
  a.counts = counts_layer && T <= count_tmax ? counts_layer : nullptr;
  a.n_invalid = n_invalid;
  a.workspace = workspace;
  a.out = out;
  const hipError_t e = moe::launch_layer_few(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return set_error(MOE_EHIP, "few-token layer: %s", hipGetErrorString(e));
  return moe::succeed();
}

}  // extern "C"
