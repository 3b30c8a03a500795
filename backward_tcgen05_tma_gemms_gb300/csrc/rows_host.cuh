// rows_host.cuh -- host pieces of the entry points that work on the rows of
// matrices: views of (..., d) tensors and their checks.
#pragma once
#include "api_common.cuh"
#include "rows.cuh"

namespace tps {

inline int es_of(int dtype) { return dtype == TPS_F32 ? 4 : dtype == TPS_BF16 ? 2 : 1; }

inline bool starts_runs(const void* p, int64_t ld, int dtype, int64_t rows) {  // 8 elements: 32, 16 or 8 bytes
  const int64_t by = dtype == TPS_E4M3 ? 8 : 16;
  return reinterpret_cast<uintptr_t>(p) % by == 0 && (rows <= 1 || ld * es_of(dtype) % by == 0);
}
inline bool starts_runs(const Rows& r, int64_t rows) { return r.p == nullptr || starts_runs(r.p, r.ld, r.dtype, rows); }

// Rows of (..., d) with unit stride along d.
inline int rows_view(const tps_tensor* t, const char* name, bool out, Rows* r, int64_t* rows, int64_t* d) {
  Mat m;
  int rc;
  if ((rc = as_mat(t, name, true, &m))) return rc;
  if (m.cols > 1 && m.sc != 1) return fail(TPS_ERR_LAYOUT, "%s: rows must have unit stride", name);
  if (m.rows > 1 && m.sr < 0) return fail(TPS_ERR_LAYOUT, "%s: negative row stride", name);
  if (out && m.rows > 1 && m.sr < m.cols) return fail(TPS_ERR_LAYOUT, "%s: rows overlap", name);
  if (m.dtype != TPS_F32 && m.dtype != TPS_BF16 && m.dtype != TPS_E4M3)
    return fail(TPS_ERR_DTYPE, "%s: unsupported type", name);
  if (reinterpret_cast<uintptr_t>(m.data) % es_of(m.dtype) != 0) return fail(TPS_ERR_LAYOUT, "%s: misaligned data", name);
  r->p = static_cast<char*>(m.data);
  r->ld = m.sr;
  r->dtype = m.dtype;
  *rows = m.rows;
  *d = m.cols;
  return TPS_OK;
}
inline int float_rows(const tps_tensor* t, const char* name, bool out, int64_t rows, int64_t d, Rows* r) {
  int64_t n, c;
  int rc;
  if ((rc = rows_view(t, name, out, r, &n, &c))) return rc;
  if (n != rows || c != d)
    return fail(TPS_ERR_SHAPE, "%s: shape (%lld, %lld), expected (%lld, %lld)", name, (long long)n, (long long)c,
                (long long)rows, (long long)d);
  if (r->dtype == TPS_E4M3) return fail(TPS_ERR_DTYPE, "%s must be f32 or bf16", name);
  return TPS_OK;
}
// n contiguous entries, each at a multiple of its size.
inline int aligned_vector(const tps_tensor* t, const char* name, int dtype, int64_t n) {
  const int rc = expect_vector(t, name, dtype, n);
  if (rc) return rc;
  return reinterpret_cast<uintptr_t>(t->data) % es_of(dtype) == 0 ? TPS_OK : fail(TPS_ERR_LAYOUT, "%s: misaligned data", name);
}
inline int weight_vector(const tps_tensor* w, int64_t d, const char** p, int* dtype) {
  *p = nullptr;
  *dtype = TPS_F32;
  if (w == nullptr) return TPS_OK;
  if (w->dtype != TPS_F32 && w->dtype != TPS_BF16) return fail(TPS_ERR_DTYPE, "weight must be f32 or bf16");
  int rc;
  if ((rc = aligned_vector(w, "weight", w->dtype, d))) return rc;
  *p = static_cast<const char*>(w->data);
  *dtype = w->dtype;
  return TPS_OK;
}
inline int too_large(int64_t rows, int64_t d) {
  if (rows >= (1ll << 31) || d >= (1ll << 31)) return fail(TPS_ERR_SHAPE, "an extent of 2^31 or more");
  return TPS_OK;
}

inline int launched(const char* what) {
  note_launch();
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? TPS_OK : fail(TPS_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(cudaGetLastError()));
}
// Checks and fills a dropout (defined in dropout.cu; nullptr: none).
int dropout_of(const tps_dropout* o, Dropout* d);
// Sum of `n` rows of d floats to `out` (f32 or bf16), in a fixed order (norm.cu).
// early: see early_attribute.
int launch_sum_rows(const float* part, int64_t n, int64_t d, void* out, int dtype, bool early, cudaStream_t s);

}  // namespace tps
