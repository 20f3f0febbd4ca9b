// C ABI of the 8-bit floating point products: argument checks, then launches on the
// caller's stream (see abi.hip).
#include "layer_ops.h"

using moe::aligned;
using moe::overlap;
using moe::set_error;

extern "C" {

int moe_quantize_rows_f8(const void* x, int dtype, int64_t ld, int rows, int K, uint8_t* q,
                         float* scale, void* stream) {
  if (!moe::dtype_known(dtype)) return set_error(MOE_EINVAL, "dtype=%d unknown", dtype);
  if (rows < 0 || rows > MOE_F8_MAX_ROWS)
    return set_error(MOE_EINVAL, "rows=%d outside [0, %d]", rows, MOE_F8_MAX_ROWS);
  if (K < 1 || K > MOE_F8_MAX_K)
    return set_error(MOE_EINVAL, "K=%d outside [1, %d]", K, MOE_F8_MAX_K);
  if (ld < K || ld > (int64_t)1 << 31)
    return set_error(MOE_EINVAL, "ld=%lld must be in [K=%d, 2^31]", (long long)ld, K);
  if (rows == 0) return moe::succeed();
  if (!x || !q || !scale) return set_error(MOE_EINVAL, "x, q and scale must not be NULL");
  if (!aligned(x, moe::dtype_bytes(dtype)) || !aligned(scale, 4))
    return set_error(MOE_EINVAL, "x and scale must be aligned to their elements");
  const size_t xb = ((size_t)(rows - 1) * ld + K) * moe::dtype_bytes(dtype);
  const size_t qb = (size_t)rows * K, sb = (size_t)rows * moe::f8_blocks(K) * 4;
  if (overlap(x, xb, q, qb) || overlap(x, xb, scale, sb) || overlap(q, qb, scale, sb))
    return set_error(MOE_EINVAL, "x, q and scale must not overlap");
  const hipError_t e = moe::launch_quantize_f8(x, dtype, ld, rows, K, nullptr, q, scale,
                                               static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return set_error(MOE_EHIP, "quantize launch: %s", hipGetErrorString(e));
  return moe::succeed();
}

int moe_linear_f8(const uint8_t* xq, int64_t ldx, const float* xs, int M, const uint8_t* w,
                  const float* ws, int N, int K, void* y, int dtype, int64_t ldy, void* stream) {
  if (!moe::dtype_known(dtype)) return set_error(MOE_EINVAL, "dtype=%d unknown", dtype);
  if (M < 0 || N < 0 || M > MOE_F8_MAX_ROWS || N > MOE_F8_MAX_ROWS)
    return set_error(MOE_EINVAL, "M=%d, N=%d outside [0, %d]", M, N, MOE_F8_MAX_ROWS);
  if (K < 16 || K % 16 || K > MOE_F8_MAX_K)
    return set_error(MOE_EINVAL, "K=%d must be a multiple of 16 in [16, %d]", K, MOE_F8_MAX_K);
  if (ldx < K || ldx % 16 || ldx > (int64_t)1 << 31)
    return set_error(MOE_EINVAL, "ldx=%lld must be a multiple of 16 in [K=%d, 2^31]",
                     (long long)ldx, K);
  if (ldy < N || ldy > (int64_t)1 << 31)
    return set_error(MOE_EINVAL, "ldy=%lld must be in [N=%d, 2^31]", (long long)ldy, N);
  if (M == 0 || N == 0) return moe::succeed();
  if (!xq || !xs || !w || !ws || !y)
    return set_error(MOE_EINVAL, "xq, xs, w, ws and y must not be NULL");
  const size_t es = moe::dtype_bytes(dtype), blocks = moe::f8_blocks(K);
  if (!aligned(xq, 16) || !aligned(w, 16) || !aligned(xs, 4) || !aligned(ws, 4) || !aligned(y, es))
    return set_error(MOE_EINVAL, "xq and w must be 16-byte aligned, xs, ws and y to their elements");
  const size_t yb = ((size_t)(M - 1) * ldy + N) * es;
  if (overlap(y, yb, xq, (size_t)(M - 1) * ldx + K) || overlap(y, yb, w, (size_t)N * K) ||
      overlap(y, yb, xs, M * blocks * 4) || overlap(y, yb, ws, moe::f8_blocks(N) * blocks * 4))
    return set_error(MOE_EINVAL, "y must not overlap the inputs");
  moe::F8Args a = {};
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
  if (!moe::gemm_f8_fits(a))
    return set_error(MOE_ENOTSUP, "M=%d, N=%d: more tiles than one launch takes", M, N);
  const hipError_t e = moe::launch_gemm_f8(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return set_error(MOE_EHIP, "FP8 product: %s", hipGetErrorString(e));
  return moe::succeed();
}

size_t moe_ffn_f8_workspace_bytes(int T, int k, int H, int I) {
  if (T <= 0 || k <= 0 || H <= 0 || I <= 0) return 0;
  // h fp32, its scales, h in 8 bits
  return (size_t)T * k * ((size_t)I * 5 + (size_t)moe::f8_blocks(I) * 4);
}

int moe_expert_ffn_f8(const moe_bank* bank, moe_split split, const uint8_t* xq, const float* xs,
                      int T, int k, int H, int I, void* workspace, uint16_t* Y, void* stream) {
  if (T < 0) return set_error(MOE_EINVAL, "T=%d must be >= 0", T);
  if (k < 1 || k > MOE_MAX_TOPK)
    return set_error(MOE_EINVAL, "k=%d outside [1, %d]", k, MOE_MAX_TOPK);
  if ((int64_t)T * k > MOE_F8_MAX_ROWS)
    return set_error(MOE_EINVAL, "T*k above %d", MOE_F8_MAX_ROWS);
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
  const size_t slots = (size_t)T * k, hblocks = moe::f8_blocks(I);
  float* h = static_cast<float*>(workspace);
  uint8_t* hq = reinterpret_cast<uint8_t*>(h + slots * I);
  float* hs = reinterpret_cast<float*>(hq + slots * I);
  moe::F8Args a = {};
  a.a = xq;
  a.lda = H;
  a.sa = xs;
  a.w = p[0];
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
  moe::F8Args d = a;  // the down product
  d.a = hq;
  d.lda = I;
  d.sa = hs;
  d.w = p[2];
  d.sw = reinterpret_cast<const float*>(p[3]);
  d.N = H;
  d.K = I;
  d.by_token = 0;
  d.gate_up = 0;
  // a pick's row is rounded to bf16, as in the other layers: what moe_finalize reads, half the
  // bytes (0.0024 of the layer's output instead of 0.0017 in all)
  d.y = Y;
  d.dtype = MOE_DTYPE_BF16;
  d.ldy = H;
  if (!moe::gemm_f8_fits(a) || !moe::gemm_f8_fits(d))
    return set_error(MOE_ENOTSUP, "T*k=%zu at H=%d, I=%d: more tiles than one launch takes", slots,
                     H, I);
  const size_t wb = slots * (I * 5 + hblocks * 4), yb = slots * H * 2;
  const size_t xqb = (size_t)T * H, xsb = (size_t)T * moe::f8_blocks(H) * 4;
  if (overlap(Y, yb, workspace, wb) || overlap(Y, yb, xq, xqb) || overlap(Y, yb, xs, xsb) ||
      overlap(workspace, wb, xq, xqb) || overlap(workspace, wb, xs, xsb))
    return set_error(MOE_EINVAL, "workspace and Y must not overlap xq, xs or each other");
  hipError_t e = moe::launch_gemm_f8(a, s);
  if (e == hipSuccess)
    e = moe::launch_quantize_f8(h, MOE_DTYPE_F32, I, (int)slots, I, &split, hq, hs, s);
  if (e == hipSuccess) e = moe::launch_gemm_f8(d, s);
  if (e != hipSuccess) return set_error(MOE_EHIP, "FP8 expert FFN: %s", hipGetErrorString(e));
  return moe::succeed();
}

}  // extern "C"
