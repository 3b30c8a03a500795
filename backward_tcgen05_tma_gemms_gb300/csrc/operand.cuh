// operand.cuh -- GEMM operands as TMA takes them: the caller's own, or laid
// out anew in a workspace (padded rows; fp32 values as three bf16 planes).
#pragma once
#include "api_common.cuh"

namespace tps {

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// An operand X(i, j) as the GEMMs take it: the caller's, or laid out anew.
struct Operand {
  const char* p = nullptr;
  int64_t si = 0, sj = 0;         // strides of i and j, one of them 1
  int64_t plane = 0, cols = 0;    // GemmDesc::a_plane, a_cols when laid out
};
inline bool tma_can(const void* p, int64_t si, int64_t sj) {
  const int64_t outer = sj == 1 ? si : sj;
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (si == 1 || sj == 1) && outer % 8 == 0;
}
// Bytes of X (ni x nj) laid out, in either orientation.
inline int64_t laid_bytes(int64_t ni, int64_t nj, int planes) {
  const int64_t a = ni * round_up(nj, 64), b = nj * round_up(ni, 64);
  return 2 * planes * (a > b ? a : b);
}
// X (ni x nj, strides si, sj, f32 or bf16) laid out at `dst`: rows of whole K
// tiles with zeros behind, three planes side by side for f32 (operand.cu).
int lay_operand(int dtype, const char* src, int64_t ni, int64_t nj, int64_t si, int64_t sj, char* dst, const char* label,
                cudaStream_t s, Operand* o);
// The same of up to kLayJobs operands of one type in one launch.
constexpr int kLayJobs = 3;
struct LayJob {
  const void* src;
  void* dst;
  int64_t rows, cols, ld, plane;
};
void lay_job(int dtype, const char* src, int64_t ni, int64_t nj, int64_t si, int64_t sj, char* dst, LayJob* job, Operand* o);
int launch_lay(int dtype, const LayJob* jobs, int n, const char* label, cudaStream_t s);

// A(m, k) = X(i, j) or, transposed, X(j, i); B(k, n) alike.
inline void set_a(GemmDesc* g, const Operand& x, bool t) {
  g->a = x.p; g->a_sm = t ? x.sj : x.si; g->a_sk = t ? x.si : x.sj; g->a_plane = x.plane; g->a_cols = x.cols;
}
inline void set_b(GemmDesc* g, const Operand& x, bool t) {
  g->b = x.p; g->b_sk = t ? x.sj : x.si; g->b_sn = t ? x.si : x.sj; g->b_plane = x.plane; g->b_cols = x.cols;
}

}  // namespace tps
