// Host-side argument checks (see validate.hpp).  No HIP headers here.
#include "validate.hpp"

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "../../include/sparse_act.h"

namespace sa {
namespace {

thread_local char g_msg[512] = {0};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return status;
}

}  // namespace

void clear_error() { g_msg[0] = 0; }

void set_error(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
}

const char* last_error() { return g_msg; }

#define REQUIRE(cond, status, ...) \
  do {                             \
    if (!(cond)) return fail(status, __VA_ARGS__); \
  } while (0)

static int check_rows_d(int64_t rows, int64_t d, const char* fn) {
  REQUIRE(rows >= 0, SA_ERR_INVALID_ARG, "%s: rows must be >= 0 (got %lld)", fn, (long long)rows);
  REQUIRE(d >= 1, SA_ERR_INVALID_ARG, "%s: d must be >= 1 (got %lld)", fn, (long long)d);
  REQUIRE(d <= kMaxD, SA_ERR_UNSUPPORTED, "%s: d = %lld exceeds %lld", fn, (long long)d,
          (long long)kMaxD);
  REQUIRE(rows <= 0x7fffffffLL, SA_ERR_UNSUPPORTED, "%s: rows too large", fn);
  return SA_OK;
}

static int check_list_outputs(const void* x, const void* mask, const void* idx, const void* val,
                              const void* nnz, const char* fn) {
  REQUIRE(x != nullptr, SA_ERR_INVALID_ARG, "%s: x is NULL", fn);
  REQUIRE(idx != nullptr && val != nullptr && nnz != nullptr, SA_ERR_INVALID_ARG,
          "%s: idx, val and nnz must not be NULL", fn);
  REQUIRE(aligned(x, 2) && aligned(val, 2), SA_ERR_INVALID_ARG,
          "%s: x and val must be 2-byte aligned", fn);
  REQUIRE(aligned(idx, 4) && aligned(nnz, 4) && aligned(mask, 4), SA_ERR_INVALID_ARG,
          "%s: idx, nnz and mask must be 4-byte aligned", fn);
  return SA_OK;
}

int check_threshold(const void* x, int64_t rows, int64_t d, float t, const void* mask,
                    const void* idx, const void* val, const void* nnz, int64_t cap) {
  const char* fn = "act_sparsify_threshold";
  int st = check_rows_d(rows, d, fn);
  if (st) return st;
  st = check_list_outputs(x, mask, idx, val, nnz, fn);
  if (st) return st;
  REQUIRE(cap >= d, SA_ERR_INVALID_ARG, "%s: cap (%lld) must be >= d (%lld)", fn,
          (long long)cap, (long long)d);
  REQUIRE(isfinite(t) && t >= 0.f, SA_ERR_INVALID_ARG, "%s: t must be finite and >= 0", fn);
  return SA_OK;
}

int check_scored(const void* x, int64_t rows, int64_t d, const void* mu, const void* colnorm,
                 int n, int m, double t, const void* mask, const void* idx, const void* val,
                 const void* nnz, int64_t cap, const void* alpha) {
  const char* fn = "act_sparsify_scored";
  int st = check_rows_d(rows, d, fn);
  if (st) return st;
  st = check_list_outputs(x, mask, idx, val, nnz, fn);
  if (st) return st;
  REQUIRE(aligned(mu, 2) && aligned(colnorm, 8) && aligned(alpha, 4), SA_ERR_INVALID_ARG,
          "%s: misaligned mu, colnorm or alpha", fn);
  if (m == 0) {
    REQUIRE(isfinite(t) && t >= 0.0, SA_ERR_INVALID_ARG, "%s: t must be finite and >= 0", fn);
    REQUIRE(cap >= d, SA_ERR_INVALID_ARG, "%s: cap (%lld) must be >= d (%lld)", fn,
            (long long)cap, (long long)d);
  } else {
    REQUIRE(m == 4 || m == 8 || m == 16 || m == 32, SA_ERR_INVALID_ARG,
            "%s: m must be 0 (threshold), 4, 8, 16 or 32 (got %d)", fn, m);
    REQUIRE(n >= 1 && n <= m, SA_ERR_INVALID_ARG, "%s: n must be in [1, m] (got %d)", fn, n);
    REQUIRE(d % m == 0, SA_ERR_INVALID_ARG, "%s: d (%lld) must be a multiple of m", fn,
            (long long)d);
    REQUIRE(cap >= d / m * n, SA_ERR_INVALID_ARG, "%s: cap (%lld) must be >= d*n/m", fn,
            (long long)cap);
  }
  return SA_OK;
}

int check_topk(const void* x, int64_t rows, int64_t d, int64_t k, const void* mask,
               const void* idx, const void* val, const void* nnz, int64_t cap) {
  const char* fn = "act_sparsify_topk";
  int st = check_rows_d(rows, d, fn);
  if (st) return st;
  st = check_list_outputs(x, mask, idx, val, nnz, fn);
  if (st) return st;
  REQUIRE(k >= 0 && k <= d, SA_ERR_INVALID_ARG, "%s: k = %lld not in [0, d = %lld]", fn,
          (long long)k, (long long)d);
  REQUIRE(cap >= k && cap >= 1, SA_ERR_INVALID_ARG, "%s: cap (%lld) must be >= max(k, 1)", fn,
          (long long)cap);
  return SA_OK;
}

int check_topk_cutoff(const void* x, int64_t rows, int64_t d, int64_t k, const void* cut,
                      const char* fn) {
  int st = check_rows_d(rows, d, fn);
  if (st) return st;
  REQUIRE(x != nullptr && (cut != nullptr || rows == 0), SA_ERR_INVALID_ARG,
          "%s: x and the cutoff output must not be NULL", fn);
  REQUIRE(aligned(x, 2) && aligned(cut, 8), SA_ERR_INVALID_ARG,
          "%s: x must be 2-byte and cut 8-byte aligned", fn);
  REQUIRE(k >= 0 && k <= d, SA_ERR_INVALID_ARG, "%s: k = %lld not in [0, d = %lld]", fn,
          (long long)k, (long long)d);
  return SA_OK;
}

int check_nm(const void* x, int64_t rows, int64_t d, int n, int m, const void* mask,
             const void* val) {
  const char* fn = "act_sparsify_nm";
  REQUIRE(rows >= 0, SA_ERR_INVALID_ARG, "%s: rows must be >= 0", fn);
  REQUIRE(m == 4 || m == 8 || m == 16 || m == 32, SA_ERR_INVALID_ARG,
          "%s: m must be 4, 8, 16 or 32 (got %d)", fn, m);
  REQUIRE(n >= 1 && n <= m, SA_ERR_INVALID_ARG, "%s: n = %d not in [1, m = %d]", fn, n, m);
  REQUIRE(d >= 32 && d % 32 == 0, SA_ERR_INVALID_ARG,
          "%s: d must be a positive multiple of 32 (got %lld)", fn, (long long)d);
  REQUIRE(x != nullptr && mask != nullptr && val != nullptr, SA_ERR_INVALID_ARG,
          "%s: x, mask and val must not be NULL", fn);
  REQUIRE(aligned(x, 16), SA_ERR_INVALID_ARG, "%s: x must be 16-byte aligned", fn);
  REQUIRE(aligned(mask, 4) && aligned(val, 2), SA_ERR_INVALID_ARG,
          "%s: mask must be 4-byte and val 2-byte aligned", fn);
  REQUIRE(rows * d / 8 <= (int64_t)0x7fffffff * 256, SA_ERR_UNSUPPORTED, "%s: too large", fn);
  return SA_OK;
}

int check_nm_shared(const void* x, int64_t rows, int64_t d, int n, int m, int tt,
                    const void* mask, const void* val) {
  const char* fn = "act_sparsify_nm_shared";
  REQUIRE(rows >= 0, SA_ERR_INVALID_ARG, "%s: rows must be >= 0", fn);
  REQUIRE(m == 4 || m == 8 || m == 16 || m == 32, SA_ERR_INVALID_ARG,
          "%s: m must be 4, 8, 16 or 32 (got %d)", fn, m);
  REQUIRE(n >= 1 && n <= m, SA_ERR_INVALID_ARG, "%s: n = %d not in [1, m = %d]", fn, n, m);
  REQUIRE(tt >= 1 && tt <= 256, SA_ERR_INVALID_ARG, "%s: tt = %d not in [1, 256]", fn, tt);
  REQUIRE(d >= 32 && d % 32 == 0, SA_ERR_INVALID_ARG,
          "%s: d must be a positive multiple of 32 (got %lld)", fn, (long long)d);
  REQUIRE(x != nullptr && mask != nullptr && val != nullptr, SA_ERR_INVALID_ARG,
          "%s: x, mask and val must not be NULL", fn);
  REQUIRE(aligned(x, 16), SA_ERR_INVALID_ARG, "%s: x must be 16-byte aligned", fn);
  REQUIRE(aligned(mask, 4) && aligned(val, 2), SA_ERR_INVALID_ARG,
          "%s: mask must be 4-byte and val 2-byte aligned", fn);
  REQUIRE(d <= (int64_t)65535 * 64, SA_ERR_UNSUPPORTED, "%s: d too large", fn);
  return SA_OK;
}

int check_calibrate(const void* samples, int64_t n, double s, const void* t_out) {
  const char* fn = "act_calibrate_threshold";
  REQUIRE(samples != nullptr && t_out != nullptr, SA_ERR_INVALID_ARG,
          "%s: samples and t_out must not be NULL", fn);
  REQUIRE(n >= 1 && n <= 0x7fffffffLL, SA_ERR_INVALID_ARG, "%s: n = %lld out of range", fn,
          (long long)n);
  REQUIRE(s >= 0.0 && s <= 1.0, SA_ERR_INVALID_ARG, "%s: s must be in [0, 1]", fn);
  REQUIRE(aligned(samples, 2) && aligned(t_out, 4), SA_ERR_INVALID_ARG,
          "%s: misaligned pointer", fn);
  return SA_OK;
}

int check_gemv_common(const void* wt, int64_t d_out, int64_t d_in, int64_t batch,
                      const void* y, const void* ws, size_t ws_bytes, size_t need_ws) {
  REQUIRE(wt != nullptr && y != nullptr, SA_ERR_INVALID_ARG, "gemv: wt and y must not be NULL");
  REQUIRE(d_out >= 8 && d_out % 8 == 0, SA_ERR_INVALID_ARG,
          "gemv: d_out must be a positive multiple of 8 (got %lld)", (long long)d_out);
  REQUIRE(d_out <= kMaxDOut, SA_ERR_UNSUPPORTED, "gemv: d_out = %lld exceeds %lld",
          (long long)d_out, (long long)kMaxDOut);
  REQUIRE(d_in >= 1 && d_in <= kMaxDIn, SA_ERR_INVALID_ARG, "gemv: d_in = %lld out of range",
          (long long)d_in);
  REQUIRE(batch >= 0 && batch <= SA_MAX_BATCH, SA_ERR_INVALID_ARG,
          "gemv: batch = %lld not in [0, %d]", (long long)batch, SA_MAX_BATCH);
  REQUIRE(aligned(wt, 16) && aligned(y, 16), SA_ERR_INVALID_ARG,
          "gemv: wt and y must be 16-byte aligned");
  REQUIRE(ws_bytes >= need_ws && (need_ws == 0 || ws != nullptr), SA_ERR_WORKSPACE,
          "gemv: workspace of %zu bytes needed, %zu given", need_ws, ws ? ws_bytes : (size_t)0);
  REQUIRE(aligned(ws, 256), SA_ERR_WORKSPACE, "gemv: workspace must be 256-byte aligned");
  return SA_OK;
}

int check_rows_gemv(const void* w, int64_t d_out, int64_t d_in, int64_t batch, const void* y,
                    const char* fn) {
  REQUIRE(w != nullptr && y != nullptr, SA_ERR_INVALID_ARG, "%s: the weight and its output must not be NULL", fn);
  REQUIRE(d_out >= 1 && d_out <= kMaxDOut, SA_ERR_INVALID_ARG,
          "%s: the row-major weight's row count %lld is not in [1, %lld]", fn, (long long)d_out,
          (long long)kMaxDOut);
  REQUIRE(d_in >= 1 && d_in <= kMaxDIn, SA_ERR_INVALID_ARG, "%s: d_in = %lld out of range", fn,
          (long long)d_in);
  REQUIRE(batch >= 0 && batch <= SA_MAX_BATCH, SA_ERR_INVALID_ARG,
          "%s: batch = %lld not in [0, %d]", fn, (long long)batch, SA_MAX_BATCH);
  REQUIRE(aligned(w, 2) && aligned(y, 2), SA_ERR_INVALID_ARG,
          "%s: the row-major weight and its output must be 2-byte aligned", fn);
  return SA_OK;
}

int check_sparse_gemv(const void* idx, const void* val, const void* nnz, int64_t batch,
                      int64_t cap) {
  (void)batch;
  REQUIRE(idx != nullptr && val != nullptr && nnz != nullptr, SA_ERR_INVALID_ARG,
          "sparse_gemv: idx, val and nnz must not be NULL");
  REQUIRE(cap >= 1, SA_ERR_INVALID_ARG, "sparse_gemv: cap must be >= 1");
  REQUIRE(aligned(idx, 4) && aligned(nnz, 4) && aligned(val, 2), SA_ERR_INVALID_ARG,
          "sparse_gemv: misaligned idx, val or nnz");
  return SA_OK;
}

int check_noalloc_size(size_t need, size_t have) {
  REQUIRE(need <= have, SA_ERR_UNSUPPORTED,
          "sparse_gemv_threshold_noalloc: this shape needs %zu bytes of scratch, more than "
          "the fixed %zu; use sparse_gemv_threshold with a workspace",
          need, have);
  return SA_OK;
}

int check_activation(const void* x, const char* name) {
  REQUIRE(x != nullptr, SA_ERR_INVALID_ARG, "%s must not be NULL", name);
  REQUIRE(aligned(x, 2), SA_ERR_INVALID_ARG, "%s must be 2-byte aligned", name);
  return SA_OK;
}

int check_threshold_value(float t) {
  REQUIRE(isfinite(t) && t >= 0.f, SA_ERR_INVALID_ARG, "t must be finite and >= 0");
  return SA_OK;
}

int check_swiglu(const void* g, const void* u, const void* colnorm, int64_t d_ff, double t,
                 int mode) {
  const char* fn = "masked_swiglu_down";
  REQUIRE(mode == 0 || mode == 1, SA_ERR_INVALID_ARG, "%s: mode must be 0 (CATS) or 1 (RaNA)",
          fn);
  REQUIRE(g != nullptr && u != nullptr, SA_ERR_INVALID_ARG, "%s: g and u must not be NULL", fn);
  REQUIRE(mode == 0 || colnorm != nullptr, SA_ERR_INVALID_ARG,
          "%s: colnorm is required for RaNA (mode 1)", fn);
  REQUIRE(aligned(g, 2) && aligned(u, 2) && aligned(colnorm, 8), SA_ERR_INVALID_ARG,
          "%s: misaligned g, u or colnorm", fn);
  REQUIRE(d_ff >= 1, SA_ERR_INVALID_ARG, "%s: d_ff must be >= 1", fn);
  REQUIRE(isfinite(t) && t >= 0.0, SA_ERR_INVALID_ARG, "%s: t must be finite and >= 0", fn);
  return SA_OK;
}

int check_col_norms(const void* wt, int64_t d_in, int64_t d_out, const void* out) {
  const char* fn = "weight_col_norms";
  REQUIRE(wt != nullptr && out != nullptr, SA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  REQUIRE(d_in >= 0 && d_out >= 8 && d_out % 8 == 0, SA_ERR_INVALID_ARG,
          "%s: d_out must be a positive multiple of 8", fn);
  REQUIRE(aligned(wt, 16) && aligned(out, 8), SA_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  REQUIRE(d_in <= (int64_t)0x7fffffff * 4, SA_ERR_UNSUPPORTED, "%s: d_in too large", fn);
  return SA_OK;
}

int check_nm_spmm(const void* xval, const void* mask, int64_t T, int64_t d_in, int n, int m,
                  const void* wt, int64_t d_out, const void* y) {
  const char* fn = "nm_act_spmm";
  REQUIRE(T >= 0, SA_ERR_INVALID_ARG, "%s: T must be >= 0", fn);
  REQUIRE(m == 4 || m == 8 || m == 16 || m == 32, SA_ERR_INVALID_ARG,
          "%s: m must be 4, 8, 16 or 32", fn);
  REQUIRE(n >= 1 && n <= m, SA_ERR_INVALID_ARG, "%s: n not in [1, m]", fn);
  REQUIRE(d_in >= 32 && d_in % 32 == 0, SA_ERR_INVALID_ARG,
          "%s: d_in must be a positive multiple of 32", fn);
  REQUIRE(d_out >= 8 && d_out % 8 == 0, SA_ERR_INVALID_ARG,
          "%s: d_out must be a positive multiple of 8", fn);
  REQUIRE(xval && mask && wt && y, SA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  REQUIRE(aligned(wt, 16) && aligned(y, 16) && aligned(mask, 4) && aligned(xval, 16),
          SA_ERR_INVALID_ARG, "%s: wt, y and xval must be 16-byte aligned, mask 4-byte", fn);
  return SA_OK;
}

int check_nm_shared_spmm(const void* xval, const void* mask, int64_t T, int64_t d_in, int n,
                         int m, int tt, const void* wt, int64_t d_out, const void* y) {
  const char* fn = "nm_shared_spmm";
  REQUIRE(tt >= 1 && tt <= 256, SA_ERR_INVALID_ARG, "%s: tt = %d not in [1, 256]", fn, tt);
  REQUIRE(T >= 0, SA_ERR_INVALID_ARG, "%s: T must be >= 0", fn);
  REQUIRE(m == 4 || m == 8 || m == 16 || m == 32, SA_ERR_INVALID_ARG,
          "%s: m must be 4, 8, 16 or 32", fn);
  REQUIRE(n >= 1 && n <= m, SA_ERR_INVALID_ARG, "%s: n not in [1, m]", fn);
  REQUIRE(d_in >= 32 && d_in % 32 == 0, SA_ERR_INVALID_ARG,
          "%s: d_in must be a positive multiple of 32", fn);
  REQUIRE(d_out >= 8 && d_out % 8 == 0, SA_ERR_INVALID_ARG,
          "%s: d_out must be a positive multiple of 8", fn);
  REQUIRE(xval && mask && wt && y, SA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  REQUIRE(aligned(wt, 16) && aligned(y, 16) && aligned(mask, 4) && aligned(xval, 16),
          SA_ERR_INVALID_ARG, "%s: wt, y and xval must be 16-byte aligned, mask 4-byte", fn);
  return SA_OK;
}

int check_dense_gemm(const void* x, int64_t T, int64_t d_in, const void* wt, int64_t d_out,
                     const void* y) {
  const char* fn = "dense_gemm";
  REQUIRE(T >= 0, SA_ERR_INVALID_ARG, "%s: T must be >= 0", fn);
  REQUIRE(d_in >= 8 && d_in % 8 == 0, SA_ERR_INVALID_ARG,
          "%s: d_in must be a positive multiple of 8", fn);
  REQUIRE(d_out >= 8 && d_out % 8 == 0, SA_ERR_INVALID_ARG,
          "%s: d_out must be a positive multiple of 8", fn);
  REQUIRE(x && wt && y, SA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  REQUIRE(aligned(x, 16) && aligned(wt, 16) && aligned(y, 16), SA_ERR_INVALID_ARG,
          "%s: x, wt and y must be 16-byte aligned", fn);
  return SA_OK;
}

int check_linear_sizes(const char* fn, int dtype, int64_t T, int64_t d_in, int64_t d_out,
                       int act) {
  REQUIRE(dtype == SA_F16 || dtype == SA_BF16, SA_ERR_INVALID_ARG,
          "%s: dtype must be SA_F16 or SA_BF16", fn);
  REQUIRE(act >= SA_ACT_NONE && act <= SA_ACT_GELU_TANH, SA_ERR_INVALID_ARG,
          "%s: unknown activation %d", fn, act);
  REQUIRE(T >= 0, SA_ERR_INVALID_ARG, "%s: T must be >= 0 (got %lld)", fn, (long long)T);
  REQUIRE(d_in >= 8 && d_in % 8 == 0, SA_ERR_INVALID_ARG,
          "%s: d_in must be a positive multiple of 8", fn);
  REQUIRE(d_out >= 8 && d_out % 8 == 0, SA_ERR_INVALID_ARG,
          "%s: d_out must be a positive multiple of 8", fn);
  REQUIRE(d_in <= kMaxLinDim && d_out <= kMaxLinDim, SA_ERR_UNSUPPORTED,
          "%s: d_in and d_out must be at most %lld", fn, (long long)kMaxLinDim);
  REQUIRE(T <= kMaxLinRows, SA_ERR_UNSUPPORTED, "%s: T must be at most %lld", fn,
          (long long)kMaxLinRows);
  return SA_OK;
}

int check_linear_matrix(const char* fn, const char* name, const void* p, int64_t ld, int64_t len,
                        bool optional) {
  if (optional && p == nullptr) return SA_OK;
  REQUIRE(p != nullptr, SA_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
  REQUIRE(aligned(p, 16), SA_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", fn, name);
  REQUIRE(ld >= len && ld % 8 == 0, SA_ERR_INVALID_ARG,
          "%s: the row stride of %s must be a multiple of 8 and at least %lld (got %lld)", fn, name,
          (long long)len, (long long)ld);
  REQUIRE(ld <= kMaxLinDim, SA_ERR_UNSUPPORTED, "%s: the row stride of %s must be at most %lld", fn,
          name, (long long)kMaxLinDim);
  return SA_OK;
}

int check_linear_vector(const char* fn, const char* name, const void* p) {
  REQUIRE(aligned(p, 16), SA_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", fn, name);
  return SA_OK;
}

int check_linear_distinct(const char* fn, const char* out, const void* o, const char* in,
                          const void* i) {
  REQUIRE(o == nullptr || o != i, SA_ERR_INVALID_ARG, "%s: %s must not be %s", fn, out, in);
  return SA_OK;
}

int check_linear_both(const char* fn, const char* a, const void* pa, const char* b,
                      const void* pb) {
  REQUIRE((pa == nullptr) == (pb == nullptr), SA_ERR_INVALID_ARG,
          "%s: %s and %s must be given together", fn, a, b);
  return SA_OK;
}

int check_int8_sizes(const char* fn, int dtype, int64_t T, int64_t d_in, int64_t d_out, int act) {
  const int st = check_linear_sizes(fn, dtype, T, d_in, d_out, act);
  if (st != SA_OK) return st;
  REQUIRE(d_in % 16 == 0, SA_ERR_INVALID_ARG, "%s: d_in must be a positive multiple of 16", fn);
  REQUIRE(d_in <= kMaxInt8Dim, SA_ERR_UNSUPPORTED, "%s: d_in must be at most %lld", fn, (long long)kMaxInt8Dim);
  return SA_OK;
}

int check_int8_codes(const char* fn, const char* name, const void* p, int64_t ld, int64_t len, bool optional) {
  if (optional && p == nullptr) return SA_OK;
  REQUIRE(p != nullptr, SA_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
  REQUIRE(aligned(p, 16), SA_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", fn, name);
  REQUIRE(ld >= len && ld % 16 == 0, SA_ERR_INVALID_ARG,
          "%s: the row stride of %s must be a multiple of 16 and at least %lld (got %lld)", fn, name,
          (long long)len, (long long)ld);
  REQUIRE(ld <= kMaxLinDim, SA_ERR_UNSUPPORTED, "%s: the row stride of %s must be at most %lld", fn, name,
          (long long)kMaxLinDim);
  return SA_OK;
}

int check_scales(const char* fn, const char* name, const void* p, bool optional) {
  REQUIRE(optional || p != nullptr, SA_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
  REQUIRE(aligned(p, 4), SA_ERR_INVALID_ARG, "%s: %s must be 4-byte aligned", fn, name);
  return SA_OK;
}

int check_grouped(const char* fn, int64_t experts, const void* offsets) {
  REQUIRE(experts >= 1, SA_ERR_INVALID_ARG, "%s: experts must be >= 1 (got %lld)", fn, (long long)experts);
  REQUIRE(experts <= SA_MAX_EXPERTS, SA_ERR_UNSUPPORTED, "%s: experts must be at most %d", fn, SA_MAX_EXPERTS);
  REQUIRE(offsets != nullptr, SA_ERR_INVALID_ARG, "%s: offsets is NULL", fn);
  REQUIRE(aligned(offsets, 4), SA_ERR_INVALID_ARG, "%s: offsets must be 4-byte aligned", fn);
  return SA_OK;
}

int check_grouped_stride(const char* fn, const char* name, const void* p, int64_t experts, int64_t stride,
                         int64_t rows, int64_t cols, int64_t ld, bool output) {
  if (p == nullptr || experts == 1) return SA_OK;
  REQUIRE(stride >= 0 && stride % 8 == 0, SA_ERR_INVALID_ARG,
          "%s: the expert stride of %s must be a multiple of 8, not negative (got %lld)", fn, name,
          (long long)stride);
  REQUIRE(stride <= kMaxLinDim * kMaxLinDim, SA_ERR_UNSUPPORTED,
          "%s: the expert stride of %s must be at most 2^42", fn, name);
  if (!output) return SA_OK;
  // one after another, or every expert's columns within each row
  REQUIRE(stride >= (rows - 1) * ld + cols || (stride >= cols && ld >= (experts - 1) * stride + cols),
          SA_ERR_INVALID_ARG, "%s: experts' matrices of %s overlap", fn, name);
  return SA_OK;
}

int check_linear_ws(const char* fn, const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return SA_OK;
  REQUIRE(ws != nullptr && ws_bytes >= need, SA_ERR_WORKSPACE,
          "%s: workspace of %zu bytes needed, %zu given", fn, need, ws ? ws_bytes : (size_t)0);
  REQUIRE(aligned(ws, 16), SA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
  return SA_OK;
}

}  // namespace sa
