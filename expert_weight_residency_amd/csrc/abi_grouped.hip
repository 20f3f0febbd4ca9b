// C ABI of the products grouped by expert: argument checks, then launches on the
// caller's stream (see abi.hip).
#include "layer_ops.h"

using moe::aligned;
using moe::overlap;
using moe::set_error;

namespace {

struct Part {
  const void* p;
  size_t n;
  const char* name;
};

// The checks that the three calls share, and the launch. in: two inputs; out: the
// output with its dtype.
int grouped(moe::GroupedArgs& a, int T, int k, int by_token, int on_host, const moe_split& split,
            const Part (&in)[2], const Part& out, void* stream) {
  if (a.elem != MOE_DTYPE_BF16 && a.elem != MOE_DTYPE_F16)
    return set_error(MOE_EINVAL, "dtype=%d is not MOE_DTYPE_BF16 or MOE_DTYPE_F16", a.elem);
  if (!moe::dtype_known(a.dtype))
    return set_error(MOE_EINVAL, "dtype=%d of %s unknown", a.dtype, out.name);
  if (T < 0) return set_error(MOE_EINVAL, "T=%d must be >= 0", T);
  if (k < 1 || k > MOE_MAX_TOPK)
    return set_error(MOE_EINVAL, "k=%d outside [1, %d]", k, MOE_MAX_TOPK);
  if ((int64_t)T * k > MOE_GROUPED_MAX_SLOTS)
    return set_error(MOE_EINVAL, "T*k above %d", MOE_GROUPED_MAX_SLOTS);
  if (a.n_rows < 0 || a.n_rows > MOE_MAX_ROWS)
    return set_error(MOE_EINVAL, "rows %d outside [0, %d]", a.n_rows, MOE_MAX_ROWS);
  if (a.N < 8 || a.N % 8 || a.N > MOE_GROUPED_MAX_DIM || a.K < 8 || a.K % 8 ||
      a.K > MOE_GROUPED_MAX_DIM)
    return set_error(MOE_EINVAL, "N=%d, K=%d must be multiples of 8 in [8, %d]", a.N, a.K,
                     MOE_GROUPED_MAX_DIM);
  if (on_host != MOE_BANK_DEVICE && on_host != MOE_BANK_HOST)
    return set_error(MOE_EINVAL, "on_host=%d is not MOE_BANK_DEVICE or MOE_BANK_HOST", on_host);
  if (a.n_rows == 0 || (T == 0 && a.op != 2)) return moe::succeed();
  if (!out.p) return set_error(MOE_EINVAL, "%s must not be NULL", out.name);
  if (!aligned(out.p, 16)) return set_error(MOE_EINVAL, "%s must be 16-byte aligned", out.name);
  if (T > 0) {
    if (!split.n_active || !split.active_rows || !split.row_off || !split.slots)
      return set_error(MOE_EINVAL, "split has a NULL buffer");
    for (const Part& i : in) {
      if (!i.p) return set_error(MOE_EINVAL, "%s must not be NULL", i.name);
      if (!aligned(i.p, 16)) return set_error(MOE_EINVAL, "%s must be 16-byte aligned", i.name);
      if (overlap(i.p, i.n, out.p, out.n))
        return set_error(MOE_EINVAL, "%s must not overlap %s", out.name, i.name);
    }
    a.n_active = split.n_active;
    a.active_rows = split.active_rows;
    a.row_off = split.row_off;
    a.slots = split.slots;
    if (on_host == MOE_BANK_HOST) {
      void* d = nullptr;
      if (hipHostGetDevicePointer(&d, const_cast<uint8_t*>(a.w), 0) != hipSuccess || !d) {
        (void)hipGetLastError();
        return set_error(MOE_EINVAL, "w is not pinned host memory");
      }
      a.w = static_cast<const uint8_t*>(d);
    }
  }
  a.M = T * k;
  a.by_token = by_token && k > 1 ? (uint32_t)((((uint64_t)1 << 32) + k - 1) / k) : 0;
  a.y = const_cast<void*>(out.p);
  if (!moe::grouped_fits(a))
    return set_error(MOE_ENOTSUP, "T*k=%d, %d rows at N=%d, K=%d: more tiles than one launch takes",
                     a.M, a.n_rows, a.N, a.K);
  const hipError_t e = moe::launch_grouped(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return set_error(MOE_EHIP, "grouped product: %s", hipGetErrorString(e));
  return moe::succeed();
}

size_t bytes(int64_t rows, int64_t cols, int dtype) {
  return (size_t)rows * cols * moe::dtype_bytes(dtype);
}

}  // namespace

extern "C" {

int moe_grouped_linear(const void* x, int dtype, int by_token, const void* w, int n_rows,
                       int on_host, moe_split split, int T, int k, int N, int K, void* y,
                       int ydtype, void* stream) {
  moe::GroupedArgs a = {};
  a.op = 0;
  a.elem = dtype;
  a.w = static_cast<const uint8_t*>(w);
  a.x = static_cast<const uint8_t*>(x);
  a.N = N;
  a.K = K;
  a.n_rows = n_rows;
  a.dtype = ydtype;
  a.ldy = N;
  const int64_t slots = (int64_t)T * k;
  return grouped(a, T, k, by_token, on_host, split,
                 {{x, bytes(by_token ? T : slots, K, dtype), "x"},
                  {w, bytes((int64_t)n_rows * N, K, dtype), "w"}},
                 {y, bytes(slots, N, ydtype), "y"}, stream);
}

int moe_grouped_linear_dx(const void* dy, int dtype, const void* w, int n_rows, int on_host,
                          moe_split split, int T, int k, int N, int K, void* dx, int xdtype,
                          void* stream) {
  moe::GroupedArgs a = {};
  a.op = 1;
  a.elem = dtype;
  a.w = static_cast<const uint8_t*>(w);
  a.dy = static_cast<const uint8_t*>(dy);
  a.N = N;
  a.K = K;
  a.n_rows = n_rows;
  a.dtype = xdtype;
  a.ldy = K;
  const int64_t slots = (int64_t)T * k;
  return grouped(a, T, k, 0, on_host, split,
                 {{dy, bytes(slots, N, dtype), "dy"},
                  {w, bytes((int64_t)n_rows * N, K, dtype), "w"}},
                 {dx, bytes(slots, K, xdtype), "dx"}, stream);
}

int moe_grouped_linear_dw(const void* dy, const void* x, int dtype, int by_token, int n_rows,
                          moe_split split, int T, int k, int N, int K, void* dw, int wdtype,
                          void* stream) {
  moe::GroupedArgs a = {};
  a.op = 2;
  a.elem = dtype;
  a.x = static_cast<const uint8_t*>(x);
  a.dy = static_cast<const uint8_t*>(dy);
  a.N = N;
  a.K = K;
  a.n_rows = n_rows;
  a.dtype = wdtype;
  a.ldy = K;
  const int64_t slots = (int64_t)T * k;
  return grouped(a, T, k, by_token, MOE_BANK_DEVICE, split,
                 {{dy, bytes(slots, N, dtype), "dy"},
                  {x, bytes(by_token ? T : slots, K, dtype), "x"}},
                 {dw, bytes((int64_t)n_rows * N, K, wdtype), "dw"}, stream);
}

}  // extern "C"
