// api_common.cuh -- host pieces shared by the translation units that
// implement entry points of include/tps.h: error reporting, tensor views and
// the GEMM dispatch (defined in api.cu).
#pragma once
#include "internal.cuh"

namespace tps {

struct Mat {  // 2-D strided view
  void* data = nullptr;
  int dtype = 0;
  int64_t rows = 0, cols = 0, sr = 0, sc = 0;
};

// Records the detail text of this host thread and returns `code`.
int fail(int code, const char* fmt, ...);
void clear_detail();
const char* dtname(int dtype);
// View `t` as a matrix (flatten: leading dimensions merge into rows).
int as_mat(const tps_tensor* t, const char* name, bool flatten, Mat* m);
int expect(const Mat& m, const char* name, int64_t rows, int64_t cols);
// Strides of a weight's (in, out) element under its layout.
void weight_strides(const Mat& w, int layout, int64_t* s_in, int64_t* s_out);
int launch_fill(void* base, int dtype, int64_t rows, int64_t cols, int64_t sr, int64_t sc, cudaStream_t stream);
int run_gemm(GemmDesc g, int64_t d_sm, int64_t d_sn, cudaStream_t stream);
// Elements of `t` if it is a contiguous vector-like tensor of `n` entries.
int expect_vector(const tps_tensor* t, const char* name, int dtype, int64_t n);

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace tps
