// operand.cu -- lays GEMM operands out for TMA (operand.cuh).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "operand.cuh"

namespace tps {

namespace {

// Lays an operand out for TMA: rows x cols of bf16, or three planes of an
// fp32 one side by side, each `plane` columns with zeros from `cols` on.
// Plane 1 holds what plane 0's rounding left, plane 2 what both left: exactly
// the value, unless its last bits are below bf16's smallest number.
template <class T>
__global__ void __launch_bounds__(256) lay_kernel(const T* src, int64_t rows, int64_t cols, int64_t ld,
                                                     __nv_bfloat16* dst, int64_t plane) {
  constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
  const int64_t per = plane / 8;
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

}  // namespace

int lay_operand(int dtype, const char* src, int64_t ni, int64_t nj, int64_t si, int64_t sj, char* dst, const char* label,
                cudaStream_t s, Operand* o) {
  const bool j_inner = sj == 1;
  const int64_t rows = j_inner ? ni : nj, cols = j_inner ? nj : ni, ld = j_inner ? si : sj;
  const int64_t plane = round_up(cols, 64), blocks = (rows * plane / 8 + 255) / 256;
  const int planes = dtype == TPS_F32 ? 3 : 1;
  const unsigned grid = static_cast<unsigned>(blocks < 152 * 16 ? blocks : 152 * 16);
  ProfScope prof("lay", label, 0.0, double(rows) * (double(cols) * (dtype == TPS_F32 ? 4 : 2) + 2.0 * planes * double(plane)), s);
  if (planes == 3)
    lay_kernel<float><<<grid, 256, 0, s>>>(reinterpret_cast<const float*>(src), rows, cols, ld,
                                              reinterpret_cast<__nv_bfloat16*>(dst), plane);
  else
    lay_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(reinterpret_cast<const __nv_bfloat16*>(src), rows, cols, ld,
                                                      reinterpret_cast<__nv_bfloat16*>(dst), plane);
  o->p = dst;
  o->si = j_inner ? planes * plane : 1;
  o->sj = j_inner ? 1 : planes * plane;
  o->plane = plane;
  o->cols = planes * plane;
  note_launch();
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? TPS_OK : fail(TPS_ERR_CUDA, "lay: launch failed: %s", cudaGetErrorString(cudaGetLastError()));
}
}  // namespace tps
