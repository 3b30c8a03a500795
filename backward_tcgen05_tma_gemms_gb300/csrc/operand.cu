// operand.cu -- lays GEMM operands out for TMA (operand.cuh).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "operand.cuh"
#include "ptx.cuh"

namespace tps {

namespace {

// Lays an operand out for TMA: rows x cols of bf16, or three planes of an
// fp32 one side by side, each `plane` columns with zeros from `cols` on.
// Plane 1 holds what plane 0's rounding left, plane 2 what both left: exactly
// the value, unless its last bits are below bf16's smallest number.
struct LayJobs {
  LayJob j[kLayJobs];
};
template <class T>
__global__ void __launch_bounds__(256) lay_kernel(const LayJobs jobs) {
  let_next_kernel_start();
  constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
#pragma unroll
  for (int q = 0; q < kLayJobs; ++q) {
    const LayJob& job = jobs.j[q];
    const T* src = static_cast<const T*>(job.src);
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(job.dst);
    const int64_t rows = job.rows, cols = job.cols, ld = job.ld, plane = job.plane, per = plane / 8;
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < rows * per; i += int64_t(gridDim.x) * 256) {
      const int64_t r = i / per, c = (i - r * per) * 8;
      const T* p = src + r * ld + c;
      T x[8];
      if (c + 8 <= cols && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(x)) / 16; ++q) reinterpret_cast<uint4*>(x)[q] = reinterpret_cast<const uint4*>(p)[q];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = c + j < cols ? p[j] : T(0.0f);
      }
      __nv_bfloat16* out = dst + r * kPlanes * plane + c;
      if constexpr (kPlanes == 1) {
        *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(x);
      } else {
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) {
          __align__(16) __nv_bfloat16 b[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            b[j] = __float2bfloat16_rn(x[j]);
            if (__hisinf(b[j]) && isfinite(x[j])) b[j] = __float2bfloat16_rz(x[j]);
            // infinities and NaN stay in plane 0, whose product alone decides about them (T2Drains)
            x[j] = isfinite(x[j]) ? x[j] - __bfloat162float(b[j]) : 0.0f;
          }
          *reinterpret_cast<uint4*>(out + pl * plane) = *reinterpret_cast<const uint4*>(b);
        }
      }
    }
  }
}

}  // namespace

void lay_job(int dtype, const char* src, int64_t ni, int64_t nj, int64_t si, int64_t sj, char* dst, LayJob* job, Operand* o) {
  const bool j_inner = sj == 1;
  const int planes = dtype == TPS_F32 ? 3 : 1;
  job->src = src;
  job->dst = dst;
  job->rows = j_inner ? ni : nj;
  job->cols = j_inner ? nj : ni;
  job->ld = j_inner ? si : sj;
  job->plane = round_up(job->cols, 64);
  o->p = dst;
  o->si = j_inner ? planes * job->plane : 1;
  o->sj = j_inner ? 1 : planes * job->plane;
  o->plane = job->plane;
  o->cols = planes * job->plane;
}
int launch_lay(int dtype, const LayJob* jobs, int n, const char* label, cudaStream_t s) {
  if (n == 0) return TPS_OK;
  LayJobs all = {};
  int64_t most = 0;
  double bytes = 0.0;
  for (int i = 0; i < n; ++i) {
    const LayJob& j = all.j[i] = jobs[i];
    const int64_t blocks = (j.rows * j.plane / 8 + 255) / 256;
    if (blocks > most) most = blocks;
    bytes += double(j.rows) * (double(j.cols) * (dtype == TPS_F32 ? 4 : 2) + (dtype == TPS_F32 ? 6.0 : 2.0) * double(j.plane));
  }
  const unsigned grid = static_cast<unsigned>(most < 152 * 16 ? most : 152 * 16);
  ProfScope prof("lay", label, 0.0, bytes, s);
  if (dtype == TPS_F32)
    lay_kernel<float><<<grid, 256, 0, s>>>(all);
  else
    lay_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(all);
  note_launch();
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? TPS_OK : fail(TPS_ERR_CUDA, "lay: launch failed: %s", cudaGetErrorString(cudaGetLastError()));
}
int lay_operand(int dtype, const char* src, int64_t ni, int64_t nj, int64_t si, int64_t sj, char* dst, const char* label,
                cudaStream_t s, Operand* o) {
  LayJob job;
  lay_job(dtype, src, ni, nj, si, sj, dst, &job, o);
  return launch_lay(dtype, &job, 1, label, s);
}

}  // namespace tps
