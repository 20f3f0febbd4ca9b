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

using moe::aligned;
using moe::overlap;
using moe::set_error;

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
  if (T > 1 << 25) return set_error(MOE_EINVAL, "T=%d above 2^25", T);
  if (ld < E || ld > (int64_t)1 << 31)
    return set_error(MOE_EINVAL, "ld=%lld must be in [E=%d, 2^31]", (long long)ld, E);
  if (T == 0) return moe::succeed();
  if (!logits || !topk_ids || !topk_w)
    return set_error(MOE_EINVAL, "logits, topk_ids and topk_w must not be NULL");
  if (!aligned(logits, moe::dtype_bytes(dtype)) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
    return set_error(MOE_EINVAL, "logits, topk_ids and topk_w must be aligned to their elements");
  const size_t in = ((size_t)(T - 1) * ld + E) * moe::dtype_bytes(dtype), ob = (size_t)T * k * 4;
  if (overlap(topk_ids, ob, logits, in) || overlap(topk_w, ob, logits, in) ||
      overlap(topk_ids, ob, topk_w, ob))
    return set_error(MOE_EINVAL, "topk_ids and topk_w must not overlap logits or each other");
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
  const size_t nb = (size_t)T * H * 2;
  const size_t wb = moe::layer_few_workspace_bytes(T, k, I);
  if (overlap(x, nb, out, nb) || overlap(x, nb, workspace, wb) || overlap(out, nb, workspace, wb))
    return set_error(MOE_EINVAL, "x, workspace and out must not overlap");
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
  // every workgroup reads the step's tables while another may write already
  if (!aligned(row_map, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) ||
      !aligned(n_invalid, 4) || !aligned(counts_layer, 4))
    return set_error(MOE_EINVAL, "row_map, topk_ids, topk_w, counts_layer and n_invalid must be "
                                 "aligned to their elements");
  const size_t pb = (size_t)T * k * 4, eb = (size_t)E * 4;
  const struct {
    const void* p;
    size_t n;
  } read[] = {{row_map, eb}, {topk_ids, pb}, {topk_w, pb}, {x, nb}},
    written[] = {{workspace, wb}, {out, nb}, {n_invalid, 4}, {counts_layer, counts_layer ? eb : 0}};
  for (const auto& w : written) {
    if (w.n == 0) continue;
    for (const auto& r : read)
      if (overlap(w.p, w.n, r.p, r.n))
        return set_error(MOE_EINVAL, "workspace, out, n_invalid and counts_layer must not overlap "
                                     "row_map, topk_ids, topk_w or x");
    for (const auto& v : written)
      if (&v < &w && v.n != 0 && overlap(w.p, w.n, v.p, v.n))
        return set_error(MOE_EINVAL, "workspace, out, n_invalid and counts_layer must not overlap "
                                     "each other");
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

int moe_quantize_rows_i8(const void* x, int dtype, int64_t ld, int rows, int K, int8_t* q,
                         float* scale, void* stream) {
  if (!moe::dtype_known(dtype)) return set_error(MOE_EINVAL, "dtype=%d unknown", dtype);
  if (rows < 0 || rows > MOE_I8_MAX_ROWS)
    return set_error(MOE_EINVAL, "rows=%d outside [0, %d]", rows, MOE_I8_MAX_ROWS);
  if (K < 1 || K > MOE_I8_MAX_K)
    return set_error(MOE_EINVAL, "K=%d outside [1, %d]", K, MOE_I8_MAX_K);
  if (ld < K || ld > (int64_t)1 << 31)
    return set_error(MOE_EINVAL, "ld=%lld must be in [K=%d, 2^31]", (long long)ld, K);
  if (rows == 0) return moe::succeed();
  if (!x || !q || !scale) return set_error(MOE_EINVAL, "x, q and scale must not be NULL");
  if (!aligned(x, moe::dtype_bytes(dtype)) || !aligned(scale, 4))
    return set_error(MOE_EINVAL, "x and scale must be aligned to their elements");
  const size_t xb = ((size_t)(rows - 1) * ld + K) * moe::dtype_bytes(dtype), qb = (size_t)rows * K;
  if (overlap(x, xb, q, qb) || overlap(x, xb, scale, (size_t)rows * 4) ||
      overlap(q, qb, scale, (size_t)rows * 4))
    return set_error(MOE_EINVAL, "x, q and scale must not overlap");
  const hipError_t e = moe::launch_quantize_rows(x, dtype, ld, rows, K, nullptr, q, scale,
                                                 static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return set_error(MOE_EHIP, "quantize launch: %s", hipGetErrorString(e));
  return moe::succeed();
}

int moe_linear_i8(const int8_t* xq, int64_t ldx, const float* xs, int M, const int8_t* w,
                  const float* ws, int N, int K, void* y, int dtype, int64_t ldy, void* stream) {
  if (!moe::dtype_known(dtype)) return set_error(MOE_EINVAL, "dtype=%d unknown", dtype);
  if (M < 0 || N < 0 || M > MOE_I8_MAX_ROWS || N > MOE_I8_MAX_ROWS)
    return set_error(MOE_EINVAL, "M=%d, N=%d outside [0, %d]", M, N, MOE_I8_MAX_ROWS);
  if (K < 16 || K % 16 || K > MOE_I8_MAX_K)
    return set_error(MOE_EINVAL, "K=%d must be a multiple of 16 in [16, %d]", K, MOE_I8_MAX_K);
  if (ldx < K || ldx % 16 || ldx > (int64_t)1 << 31)
    return set_error(MOE_EINVAL, "ldx=%lld must be a multiple of 16 in [K=%d, 2^31]",
                     (long long)ldx, K);
  if (ldy < N || ldy > (int64_t)1 << 31)
    return set_error(MOE_EINVAL, "ldy=%lld must be in [N=%d, 2^31]", (long long)ldy, N);
  if (M == 0 || N == 0) return moe::succeed();
  if (!xq || !xs || !w || !ws || !y)
    return set_error(MOE_EINVAL, "xq, xs, w, ws and y must not be NULL");
  const size_t es = moe::dtype_bytes(dtype);
  if (!aligned(xq, 16) || !aligned(w, 16) || !aligned(xs, 4) || !aligned(ws, 4) || !aligned(y, es))
    return set_error(MOE_EINVAL, "xq and w must be 16-byte aligned, xs, ws and y to their elements");
  const size_t yb = ((size_t)(M - 1) * ldy + N) * es;
  if (overlap(y, yb, xq, (size_t)(M - 1) * ldx + K) || overlap(y, yb, w, (size_t)N * K) ||
      overlap(y, yb, xs, (size_t)M * 4) || overlap(y, yb, ws, (size_t)N * 4))
    return set_error(MOE_EINVAL, "y must not overlap the inputs");
  moe::I8Args a = {};
  a.a = xq;
  a.lda = ldx;
  a.sa = xs;
  a.w = w;
  a.sw = ws;
  a.M = M;
  a.N = N;
  a.K = K;
  a.y = y;
  a.dtype = dtype;
  a.ldy = ldy;
  if (!moe::gemm_i8_fits(a))
    return set_error(MOE_ENOTSUP, "M=%d, N=%d: more tiles than one launch takes", M, N);
  const hipError_t e = moe::launch_gemm_i8(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return set_error(MOE_EHIP, "8-bit product: %s", hipGetErrorString(e));
  return moe::succeed();
}

size_t moe_ffn_i8_workspace_bytes(int T, int k, int H, int I) {
  if (T <= 0 || k <= 0 || H <= 0 || I <= 0) return 0;
  return (size_t)T * k * ((size_t)I * 5 + 4);  // h fp32, h in 8 bits, its scale
}

int moe_expert_ffn_i8(const moe_bank* bank, moe_split split, const int8_t* xq, const float* xs,
                      int T, int k, int H, int I, void* workspace, uint16_t* Y, void* stream) {
  if (T < 0) return set_error(MOE_EINVAL, "T=%d must be >= 0", T);
  if (k < 1 || k > MOE_MAX_TOPK)
    return set_error(MOE_EINVAL, "k=%d outside [1, %d]", k, MOE_MAX_TOPK);
  if ((int64_t)T * k > MOE_I8_MAX_ROWS)
    return set_error(MOE_EINVAL, "T*k above %d", MOE_I8_MAX_ROWS);
  if (H <= 0 || H % 64 || I <= 0 || I % 64)
    return set_error(MOE_EINVAL, "H=%d, I=%d must be positive multiples of 64", H, I);
  if (H > 32768 || I > 32768)
    return set_error(MOE_ENOTSUP, "H=%d, I=%d: at most 32768 supported", H, I);
  if (!bank) return set_error(MOE_EINVAL, "bank is NULL");
  if (bank->n_rows < 0 || bank->n_rows > MOE_MAX_ROWS)
    return set_error(MOE_EINVAL, "bank rows %d outside [0, %d]", bank->n_rows, MOE_MAX_ROWS);
  if (T == 0 || bank->n_rows == 0) return moe::succeed();
  if (!split.n_active || !split.active_rows || !split.row_off || !split.slots)
    return set_error(MOE_EINVAL, "split has a NULL buffer");
  if (!xq || !xs || !workspace || !Y)
    return set_error(MOE_EINVAL, "xq, xs, workspace and Y must not be NULL");
  if (!aligned(xq, 16) || !aligned(workspace, 16) || !aligned(Y, 16) || !aligned(xs, 4))
    return set_error(MOE_EINVAL, "xq, workspace and Y must be 16-byte aligned, xs 4-byte");
  const size_t align[4] = {16, 16, 16, 16};
  const uint8_t* p[4];
  int rc = moe::bank_ptrs(bank, align, p);
  if (rc != MOE_OK) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t slots = (size_t)T * k;
  float* h = static_cast<float*>(workspace);
  int8_t* hq = reinterpret_cast<int8_t*>(h + slots * I);
  float* hs = reinterpret_cast<float*>(hq + slots * I);
  moe::I8Args a = {};
  a.a = xq;
  a.lda = H;
  a.sa = xs;
  a.w = reinterpret_cast<const int8_t*>(p[0]);
  a.sw = reinterpret_cast<const float*>(p[1]);
  a.M = (int)slots;
  a.N = I;
  a.K = H;
  a.n_active = split.n_active;
  a.active_rows = split.active_rows;
  a.row_off = split.row_off;
  a.slots = split.slots;
  a.n_rows = bank->n_rows;
  a.k = k;
  a.by_token = 1;
  a.gate_up = 1;
  a.y = h;
  a.dtype = MOE_DTYPE_F32;
  a.ldy = I;
  moe::I8Args d = a;  // the down product
  d.a = hq;
  d.lda = I;
  d.sa = hs;
  d.w = reinterpret_cast<const int8_t*>(p[2]);
  d.sw = reinterpret_cast<const float*>(p[3]);
  d.N = H;
  d.K = I;
  d.by_token = 0;
  d.gate_up = 0;
  d.y = Y;
  d.dtype = MOE_DTYPE_BF16;
  d.ldy = H;
  if (!moe::gemm_i8_fits(a) || !moe::gemm_i8_fits(d))
    return set_error(MOE_ENOTSUP, "T*k=%zu at H=%d, I=%d: more tiles than one launch takes", slots,
                     H, I);
  const size_t wb = moe_ffn_i8_workspace_bytes(T, k, H, I), yb = slots * H * 2;
  if (overlap(Y, yb, workspace, wb) || overlap(Y, yb, xq, (size_t)T * H) ||
      overlap(Y, yb, xs, (size_t)T * 4) || overlap(workspace, wb, xq, (size_t)T * H) ||
      overlap(workspace, wb, xs, (size_t)T * 4))
    return set_error(MOE_EINVAL, "workspace and Y must not overlap xq, xs or each other");
  hipError_t e = moe::launch_gemm_i8(a, s);
  if (e == hipSuccess)
    e = moe::launch_quantize_rows(h, MOE_DTYPE_F32, I, (int)slots, I, &split, hq, hs, s);
  if (e == hipSuccess) e = moe::launch_gemm_i8(d, s);
  if (e != hipSuccess) return set_error(MOE_EHIP, "8-bit expert FFN: %s", hipGetErrorString(e));
  return moe::succeed();
}

}  // extern "C"
