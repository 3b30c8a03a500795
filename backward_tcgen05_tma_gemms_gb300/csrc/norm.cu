// norm.cu -- residual addition and root-mean-square norm of the rows between
// the products of a layer, forward and backward, and rows as e4m3 codes.
//
//   h = residual + D(x)         rounded to the residual's type; D: dropout
//   r = (mean h^2 + eps)^-1/2,  y_i = h_i w_i r
// and backwards, with g_i = dy_i w_i:
//   dH_i = dh_i + r (g_i - h_i r mean_j(g_j h_j r)),  dx = D(dH)
//   dw_i = sum over the rows of dy_i h_i r
// The norm is that of the stored, rounded sum: the backward pass, which reads
// it, differentiates what the forward pass computed.
//
// All of it is bound by memory.  A row passes through the registers of a group
// of threads once, 16 bytes a load, and the group joins its sums by shuffles
// and one round through shared memory; blocks walk the rows, and the loads of
// the next row are issued before the sums of the present one.  The weights,
// and in the backward pass the sums of dw, lie in shared memory as floats.  The
// e4m3 output needs the largest |h w| of the row, which is reduced together
// with the sum of squares: the codes do not depend on r.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "api_common.cuh"
#include "rows.cuh"
#include "rows_host.cuh"

namespace tps {

namespace {

constexpr int kMaxGroup = 512;     // threads of a row at most
constexpr int kMaxWarps = kMaxGroup / 32;
constexpr int kLongThreads = 512;  // of a row that does not fit into registers
static_assert(kLongThreads <= kMaxGroup, "the warps' sums fit");
constexpr int64_t kDwCols = 256;   // columns of a block of the wide weight gradient

struct NormParams {
  Rows x, res, h, y;  // p of res, h: nullptr when absent
  const char* w;      // nullptr: ones
  int w_dtype;
  float* rstd;        // nullptr: no norm (codes of x)
  float* scale;       // e4m3 output
  int64_t rows, d;
  float eps, inv_d;
  Dropout drop;
};

// Sums (and the NaN-keeping maximum of magnitudes) over the G threads of a
// row group.  `buf` alternates between two halves, so that one barrier a call
// is enough.
struct Joined {
  float sum, top;
};
template <bool TOP>
__device__ __forceinline__ Joined join_group(Joined v, int G, float2 (&buf)[kMaxWarps]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.sum += __shfl_xor_sync(0xffffffffu, v.sum, o);
    if (TOP) v.top = max_nan(v.top, __shfl_xor_sync(0xffffffffu, v.top, o), 0.0f);
  }
  if (G <= 32) return v;
  const int warp = threadIdx.x >> 5, per = G >> 5, first = warp / per * per;
  if ((threadIdx.x & 31) == 0) buf[warp] = make_float2(v.sum, v.top);
  __syncthreads();
  Joined all = {0.0f, 0.0f};
  for (int i = 0; i < per; ++i) {  // the same order in every warp
    const float2 b = buf[first + i];
    all.sum += b.x;
    if (TOP) all.top = max_nan(all.top, b.y, 0.0f);
  }
  return all;
}

// ---- rows that fit into a group's registers --------------------------------
// R runs of N elements a thread, lane + k G in the row; blockDim.x / G rows at a
// time.  TX: x; TR: the residual and h (x's type without a residual).
template <class TX, class TR, int N, int R, bool CODES>
__global__ void __launch_bounds__(kMaxGroup, R <= 2 || N == 1 ? 2 : 1) norm_fwd_kernel(const NormParams p, const int G) {
  __shared__ float2 buf[2][kMaxWarps];
  extern __shared__ __align__(16) float ws[];  // [d] weights, if there are any
  const int groups = blockDim.x / G, group = threadIdx.x / G, lane = threadIdx.x & (G - 1), d = static_cast<int>(p.d);
  const bool normed = p.rstd != nullptr, summed = p.h.p != nullptr, weighted = p.w != nullptr;
  Typed<TX, N> x[R];
  Typed<TR, N> r[R];
  auto fetch = [&](int64_t row) {
    const TX* xp = reinterpret_cast<const TX*>(p.x.p) + row * p.x.ld;
    const TR* rp = reinterpret_cast<const TR*>(p.res.p) + row * p.res.ld;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = (lane + k * G) * N;
      if (c < d) {
        x[k].load(xp + c);
        if (p.res.p != nullptr) r[k].load(rp + c);
      }
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups;
  if (row0 + group < p.rows) fetch(row0 + group);
  if (weighted) {
    if (p.w_dtype == TPS_F32)
      for (int i = threadIdx.x; i < d; i += blockDim.x) ws[i] = reinterpret_cast<const float*>(p.w)[i];
    else
      for (int i = threadIdx.x; i < d; i += blockDim.x)
        ws[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.w)[i]);
    __syncthreads();
  }
  const uint64_t key = p.drop.step != 0u ? p.drop.key() : 0;
  int turn = 0;
  for (; row0 < p.rows; row0 += step) {
    const int64_t row = row0 + group;
    const bool live = row < p.rows;
    float v[R][N];
    Joined own = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = (lane + k * G) * N;
      if (live && c < d) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[k][i] = x[k].at(i);
        if (p.drop.step != 0u) drop(p.drop, key, row * d + c, v[k]);
        if (p.res.p != nullptr) {
#pragma unroll
          for (int i = 0; i < N; ++i) v[k][i] += r[k].at(i);
        }
        if (summed) {
          run_round<N>(dtype_of<TR>(), v[k]);
          run_store(reinterpret_cast<char*>(reinterpret_cast<TR*>(p.h.p) + row * p.h.ld + c), dtype_of<TR>(), v[k]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) own.sum = fmaf(v[k][i], v[k][i], own.sum);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[k][i] = 0.0f;
      }
    }
    if (row + step < p.rows) fetch(row + step);
    auto weigh = [&](int k, float(&u)[N]) {
      const int c = (lane + k * G) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = v[k][i];
      if (weighted) {
        if constexpr (N == 8) {
          const float4 a = *reinterpret_cast<const float4*>(ws + c), b = *reinterpret_cast<const float4*>(ws + c + 4);
          u[0] *= a.x; u[1] *= a.y; u[2] *= a.z; u[3] *= a.w;
          u[4] *= b.x; u[5] *= b.y; u[6] *= b.z; u[7] *= b.w;
        } else {
          u[0] *= ws[c];
        }
      }
    };
    if (CODES) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if ((lane + k * G) * N >= d) continue;
        float u[N];
        weigh(k, u);
#pragma unroll
        for (int i = 0; i < N; ++i) own.top = max_nan(own.top, fabsf(u[i]), 0.0f);
      }
    }
    own = join_group<CODES>(own, G, buf[turn]);
    turn ^= 1;
    const float rstd = normed ? __frcp_rn(__fsqrt_rn(fmaf(own.sum, p.inv_d, p.eps))) : 1.0f;
    const RowCodes codes(own.top);
    if (!live) continue;
    if (lane == 0) {
      if (normed) p.rstd[row] = rstd;
      if (CODES) p.scale[row] = codes.scale() * rstd;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = (lane + k * G) * N;
      if (c >= d) continue;
      float u[N];
      weigh(k, u);
      if (CODES) {
        codes_store(p.y.p + row * p.y.ld + c, codes, u);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] *= rstd;
        run_store(p.y.at(row, c), p.y.dtype, u);
      }
    }
  }
}

struct NormBwdParams {
  Rows dy, h, dh, dsum, dx;  // p of dh, dsum, dx: nullptr when absent
  const char* w;
  int w_dtype;
  const float* rstd;
  float* part;               // partial weight gradients [block][d], nullptr: none
  int64_t rows, d;
  float inv_d;
  Dropout drop;
};

// TD: dy; TH: h, dh and dsum.
template <class TD, class TH, int N, int R>
__global__ void __launch_bounds__(kMaxGroup, R <= 2 || N == 1 ? 2 : 1) norm_bwd_kernel(const NormBwdParams p, const int G) {
  __shared__ float2 buf[2][kMaxWarps];
  extern __shared__ __align__(16) float ws[];  // [d] weights, then [row group][d] sums of dw
  const int groups = blockDim.x / G, group = threadIdx.x / G, lane = threadIdx.x & (G - 1), d = static_cast<int>(p.d);
  float* sums = ws + d + group * d;
  if (p.w_dtype == TPS_F32)
    for (int i = threadIdx.x; i < d; i += blockDim.x) ws[i] = p.w != nullptr ? reinterpret_cast<const float*>(p.w)[i] : 1.0f;
  else
    for (int i = threadIdx.x; i < d; i += blockDim.x) ws[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.w)[i]);
  if (p.part != nullptr)
    for (int i = threadIdx.x; i < groups * d; i += blockDim.x) ws[d + i] = 0.0f;
  __syncthreads();
  const uint64_t key = p.drop.step != 0u ? p.drop.key() : 0;
  int turn = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups; row0 < p.rows; row0 += static_cast<int64_t>(gridDim.x) * groups) {
    const int64_t row = row0 + group;
    const bool live = row < p.rows;
    const float r = live ? __ldg(p.rstd + row) : 0.0f;
    Typed<TD, N> a[R];
    Typed<TH, N> b[R], in[R];
    const TD* dyp = reinterpret_cast<const TD*>(p.dy.p) + row * p.dy.ld;
    const TH* hp = reinterpret_cast<const TH*>(p.h.p) + row * p.h.ld;
    const TH* dhp = reinterpret_cast<const TH*>(p.dh.p) + row * p.dh.ld;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = (lane + k * G) * N;
      if (live && c < d) {
        a[k].load(dyp + c);
        b[k].load(hp + c);
        if (p.dh.p != nullptr) in[k].load(dhp + c);
      }
    }
    // of the columns of run k: g = dy w and n = h r
    auto terms = [&](int k, float(&g)[N], float(&n)[N]) {
      const int c = (lane + k * G) * N;
      if constexpr (N == 8) {
        const float4 x = *reinterpret_cast<const float4*>(ws + c), y = *reinterpret_cast<const float4*>(ws + c + 4);
        const float w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = a[k].at(i) * w[i];
      } else {
        g[0] = a[k].at(0) * ws[c];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) n[i] = b[k].at(i) * r;
    };
    Joined own = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = (lane + k * G) * N;
      if (!live || c >= d) continue;
      float g[N], n[N];
      terms(k, g, n);
#pragma unroll
      for (int i = 0; i < N; ++i) own.sum = fmaf(g[i], n[i], own.sum);
      if (p.part != nullptr) {
        if constexpr (N == 8) {
          float4 x = *reinterpret_cast<const float4*>(sums + c), y = *reinterpret_cast<const float4*>(sums + c + 4);
          x.x = fmaf(a[k].at(0), n[0], x.x);
          x.y = fmaf(a[k].at(1), n[1], x.y);
          x.z = fmaf(a[k].at(2), n[2], x.z);
          x.w = fmaf(a[k].at(3), n[3], x.w);
          y.x = fmaf(a[k].at(4), n[4], y.x);
          y.y = fmaf(a[k].at(5), n[5], y.y);
          y.z = fmaf(a[k].at(6), n[6], y.z);
          y.w = fmaf(a[k].at(7), n[7], y.w);
          *reinterpret_cast<float4*>(sums + c) = x;
          *reinterpret_cast<float4*>(sums + c + 4) = y;
        } else {
          sums[c] = fmaf(a[k].at(0), n[0], sums[c]);
        }
      }
    }
    own = join_group<false>(own, G, buf[turn]);
    turn ^= 1;
    const float mean = own.sum * p.inv_d;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = (lane + k * G) * N;
      if (!live || c >= d) continue;
      float v[N], n[N];
      terms(k, v, n);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = fmaf(-n[i], mean, v[i]) * r;
        if (p.dh.p != nullptr) v[i] += in[k].at(i);
      }
      if (p.dsum.p != nullptr)
        run_store(reinterpret_cast<char*>(reinterpret_cast<TH*>(p.dsum.p) + row * p.dsum.ld + c), dtype_of<TH>(), v);
      if (p.dx.p != nullptr) {
        if (p.drop.step != 0u) drop(p.drop, key, row * d + c, v);
        run_store(p.dx.at(row, c), p.dx.dtype, v);
      }
    }
  }
  if (p.part == nullptr) return;
  __syncthreads();
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * d;
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float s = 0.0f;
    for (int q = 0; q < groups; ++q) s += ws[d + q * d + c];
    out[c] = s;
  }
}

// ---- other rows -------------------------------------------------------------
// Rows wider than the registers hold, and rows of single elements whose types
// differ: a block a row, which is read a second time (out of L2) after its sums.
template <int N, bool CODES>
__global__ void __launch_bounds__(kLongThreads) norm_fwd_long_kernel(const NormParams p) {
  __shared__ float2 buf[kMaxWarps];
  const int64_t row = blockIdx.x;
  const uint64_t key = p.drop.step != 0u ? p.drop.key() : 0;
  const int w_es = p.w_dtype == TPS_F32 ? 4 : 2;
  const bool normed = p.rstd != nullptr;
  auto weigh = [&](int64_t c, float(&v)[N]) {
    if (p.w == nullptr) return;
    Raw<N> q;
    float w[N];
    raw_load(p.w + c * w_es, p.w_dtype, q);
    raw_value(q, p.w_dtype, w);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= w[i];
  };
  Joined own = {0.0f, 0.0f};
  for (int64_t c = threadIdx.x * N; c < p.d; c += kLongThreads * N) {
    Raw<N> x, r;
    float v[N];
    raw_load(p.x.at(row, c), p.x.dtype, x);
    if (p.res.p != nullptr) raw_load(p.res.at(row, c), p.res.dtype, r);
    raw_value(x, p.x.dtype, v);
    if (p.drop.step != 0u) drop(p.drop, key, row * p.d + c, v);
    if (p.res.p != nullptr) {
      float q[N];
      raw_value(r, p.res.dtype, q);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += q[i];
    }
    if (p.h.p != nullptr) {
      run_round<N>(p.h.dtype, v);
      run_store(p.h.at(row, c), p.h.dtype, v);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) own.sum = fmaf(v[i], v[i], own.sum);
    if (CODES) {
      weigh(c, v);
#pragma unroll
      for (int i = 0; i < N; ++i) own.top = max_nan(own.top, fabsf(v[i]), 0.0f);
    }
  }
  own = join_group<CODES>(own, kLongThreads, buf);
  const float rstd = normed ? __frcp_rn(__fsqrt_rn(fmaf(own.sum, p.inv_d, p.eps))) : 1.0f;
  const RowCodes codes(own.top);
  if (threadIdx.x == 0) {
    if (normed) p.rstd[row] = rstd;
    if (CODES) p.scale[row] = codes.scale() * rstd;
  }
  const Rows& src = p.h.p != nullptr ? p.h : p.x;  // h where this thread has written it
  for (int64_t c = threadIdx.x * N; c < p.d; c += kLongThreads * N) {
    Raw<N> x;
    float v[N];
    raw_load(src.at(row, c), src.dtype, x);
    raw_value(x, src.dtype, v);
    weigh(c, v);
    if (CODES) {
      codes_store(p.y.at(row, c), codes, v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= rstd;
      run_store(p.y.at(row, c), p.y.dtype, v);
    }
  }
}
template <int N>
__global__ void __launch_bounds__(kLongThreads) norm_bwd_long_kernel(const NormBwdParams p) {
  __shared__ float2 buf[kMaxWarps];
  const int64_t row = blockIdx.x;
  const uint64_t key = p.drop.step != 0u ? p.drop.key() : 0;
  const int w_es = p.w_dtype == TPS_F32 ? 4 : 2;
  const float r = __ldg(p.rstd + row);
  auto terms = [&](int64_t c, float(&g)[N], float(&n)[N]) {
    Raw<N> a, b, q;
    raw_load(p.dy.at(row, c), p.dy.dtype, a);
    raw_load(p.h.at(row, c), p.h.dtype, b);
    raw_value(a, p.dy.dtype, g);
    raw_value(b, p.h.dtype, n);
    if (p.w != nullptr) {
      float w[N];
      raw_load(p.w + c * w_es, p.w_dtype, q);
      raw_value(q, p.w_dtype, w);
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) n[i] *= r;
  };
  Joined own = {0.0f, 0.0f};
  for (int64_t c = threadIdx.x * N; c < p.d; c += kLongThreads * N) {
    float g[N], n[N];
    terms(c, g, n);
#pragma unroll
    for (int i = 0; i < N; ++i) own.sum = fmaf(g[i], n[i], own.sum);
  }
  own = join_group<false>(own, kLongThreads, buf);
  const float mean = own.sum * p.inv_d;
  for (int64_t c = threadIdx.x * N; c < p.d; c += kLongThreads * N) {
    float v[N], n[N];
    terms(c, v, n);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = fmaf(-n[i], mean, v[i]) * r;
    if (p.dh.p != nullptr) {
      Raw<N> in;
      float q[N];
      raw_load(p.dh.at(row, c), p.dh.dtype, in);
      raw_value(in, p.dh.dtype, q);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += q[i];
    }
    if (p.dsum.p != nullptr) run_store(p.dsum.at(row, c), p.dsum.dtype, v);
    if (p.dx.p != nullptr) {
      if (p.drop.step != 0u) drop(p.drop, key, row * p.d + c, v);
      run_store(p.dx.at(row, c), p.dx.dtype, v);
    }
  }
}

// Their partial weight gradients: a block takes kDwCols columns of every
// gridDim.y-th row.
__global__ void __launch_bounds__(kDwCols) norm_dw_kernel(const NormBwdParams p) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kDwCols + threadIdx.x;
  if (c >= p.d) return;
  float s = 0.0f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    Raw<1> a, b;
    float g[1], h[1];
    raw_load(p.dy.at(row, c), p.dy.dtype, a);
    raw_load(p.h.at(row, c), p.h.dtype, b);
    raw_value(a, p.dy.dtype, g);
    raw_value(b, p.h.dtype, h);
    s = fmaf(g[0], h[0] * __ldg(p.rstd + row), s);
  }
  p.part[static_cast<int64_t>(blockIdx.y) * p.d + c] = s;
}

// ------------------------------------------------------------------ host

int round_pow2(int64_t x) {
  int r = 1;
  while (r < x) r *= 2;
  return r;
}
// How a row is spread over threads: runs of N elements, R of them a thread, G
// threads a row; N = 0: the kernels of long rows.
// 16-byte loads where every row of every tensor starts on one and holds whole
// runs of eight; else single elements, eight a thread, where the types agree.
// Two runs a thread in bf16, one where fp32 is among the types (as many bytes),
// up to kMaxGroup threads; then more runs, up to 16384 columns.
struct Spread {
  int N, R, G, threads;
};
Spread spread_of(int64_t d, bool wide, bool fp32, bool mixed) {
  Spread s = {0, 0, 0, 0};
  if (!wide && (mixed || d > 8 * kMaxGroup)) return s;
  s.N = wide ? 8 : 1;
  s.R = wide ? (fp32 ? 1 : 2) : 8;
  const int64_t runs = (d + s.N - 1) / s.N;
  while (wide && runs > int64_t(s.R) * kMaxGroup && s.R < 4) s.R *= 2;
  if (runs > int64_t(s.R) * kMaxGroup) return Spread{0, 0, 0, 0};
  const int64_t need = (runs + s.R - 1) / s.R;
  s.G = need <= 32 ? 32 : round_pow2(need);
  s.threads = s.G < 256 ? 256 : s.G;
  return s;
}

// Blocks that walk the rows: as many as the launch bounds (1024 threads an SM,
// 512 with four runs a thread) and shared memory let be resident.
constexpr int64_t kSms = 152, kMostBlocks = kSms * 4;
template <class F>
int resident(F f, const Spread& sp, size_t shared, int64_t* blocks) {
  if (shared > (48u << 10) &&
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(shared)) != cudaSuccess)
    return fail(TPS_ERR_CUDA, "norm: %s", cudaGetErrorString(cudaGetLastError()));
  const int64_t by_threads = (sp.N == 8 && sp.R > 2 ? 512 : 1024) / sp.threads, by_shared = (224 << 10) / (int64_t(shared) + 2048);
  const int64_t per = by_threads < by_shared ? by_threads : by_shared;
  *blocks = kSms * (per < 1 ? 1 : per);
  return TPS_OK;
}

template <class TX, class TR, int N, int R, bool CODES>
int launch_fwd(const NormParams& p, const Spread& sp, cudaStream_t s) {
  const size_t shared = p.w != nullptr ? sizeof(float) * p.d : 0;
  const int64_t per = sp.threads / sp.G, blocks = (p.rows + per - 1) / per;
  int64_t most = 0;
  const int rc = resident(norm_fwd_kernel<TX, TR, N, R, CODES>, sp, shared, &most);
  if (rc) return rc;
  norm_fwd_kernel<TX, TR, N, R, CODES>
      <<<static_cast<unsigned>(blocks < most ? blocks : most), sp.threads, shared, s>>>(p, sp.G);
  return launched("norm");
}
template <class TX, class TR, bool CODES>
int launch_fwd_typed(const NormParams& p, const Spread& sp, cudaStream_t s) {
  constexpr bool kBf16 = sizeof(TX) == 2 && sizeof(TR) == 2;
  if (sp.N == 1) {
    if constexpr (sizeof(TX) == sizeof(TR)) return launch_fwd<TX, TR, 1, 8, CODES>(p, sp, s);
    return fail(TPS_ERR_DTYPE, "norm: single elements of two types");
  }
  if constexpr (!kBf16)
    if (sp.R == 1) return launch_fwd<TX, TR, 8, 1, CODES>(p, sp, s);
  if (sp.R == 2) return launch_fwd<TX, TR, 8, 2, CODES>(p, sp, s);
  return launch_fwd<TX, TR, 8, 4, CODES>(p, sp, s);
}
template <bool CODES>
int launch_fwd_codes(const NormParams& p, const Spread& sp, int tx, int tr, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  if (tx == TPS_F32) return tr == TPS_F32 ? launch_fwd_typed<float, float, CODES>(p, sp, s) : launch_fwd_typed<float, bf16, CODES>(p, sp, s);
  return tr == TPS_F32 ? launch_fwd_typed<bf16, float, CODES>(p, sp, s) : launch_fwd_typed<bf16, bf16, CODES>(p, sp, s);
}

int launch_norm_fwd(const NormParams& p, const char* label, cudaStream_t s) {
  const bool wide = p.d % 8 == 0 && starts_runs(p.x, p.rows) && starts_runs(p.res, p.rows) && starts_runs(p.h, p.rows) &&
                    starts_runs(p.y, p.rows) && (p.w == nullptr || starts_runs(p.w, 0, p.w_dtype, 1));
  const int tx = p.x.dtype, tr = p.res.p != nullptr ? p.res.dtype : tx;
  const bool codes = p.y.dtype == TPS_E4M3;
  const Spread sp = spread_of(p.d, wide, tx == TPS_F32 || tr == TPS_F32, tx != tr);
  const double bytes = double(p.rows) * double(p.d) *
                       (es_of(p.x.dtype) + (p.res.p ? es_of(p.res.dtype) : 0) + (p.h.p ? es_of(p.h.dtype) : 0) + es_of(p.y.dtype));
  ProfScope prof("norm", label, 0.0, bytes, s);
  if (sp.N != 0) return codes ? launch_fwd_codes<true>(p, sp, tx, tr, s) : launch_fwd_codes<false>(p, sp, tx, tr, s);
  const unsigned grid = static_cast<unsigned>(p.rows);
  if (wide)
    codes ? norm_fwd_long_kernel<8, true><<<grid, kLongThreads, 0, s>>>(p) : norm_fwd_long_kernel<8, false><<<grid, kLongThreads, 0, s>>>(p);
  else
    codes ? norm_fwd_long_kernel<1, true><<<grid, kLongThreads, 0, s>>>(p) : norm_fwd_long_kernel<1, false><<<grid, kLongThreads, 0, s>>>(p);
  return launched("norm_long");
}

template <class TD, class TH, int N, int R>
int launch_bwd(const NormBwdParams& p, const Spread& sp, int64_t* parts, cudaStream_t s) {
  const int64_t per = sp.threads / sp.G, blocks = (p.rows + per - 1) / per;
  const size_t shared = sizeof(float) * p.d * (1 + (p.part != nullptr ? per : 0));
  int64_t most = 0;
  const int rc = resident(norm_bwd_kernel<TD, TH, N, R>, sp, shared, &most);
  if (rc) return rc;
  *parts = blocks < most ? blocks : most;
  norm_bwd_kernel<TD, TH, N, R><<<static_cast<unsigned>(*parts), sp.threads, shared, s>>>(p, sp.G);
  return launched("norm_bwd");
}
template <class TD, class TH>
int launch_bwd_typed(const NormBwdParams& p, const Spread& sp, int64_t* parts, cudaStream_t s) {
  constexpr bool kBf16 = sizeof(TD) == 2 && sizeof(TH) == 2;
  if (sp.N == 1) {
    if constexpr (sizeof(TD) == sizeof(TH)) return launch_bwd<TD, TH, 1, 8>(p, sp, parts, s);
    return fail(TPS_ERR_DTYPE, "norm: single elements of two types");
  }
  if constexpr (!kBf16)
    if (sp.R == 1) return launch_bwd<TD, TH, 8, 1>(p, sp, parts, s);
  if (sp.R == 2) return launch_bwd<TD, TH, 8, 2>(p, sp, parts, s);
  return launch_bwd<TD, TH, 8, 4>(p, sp, parts, s);
}

}  // namespace

// Sum of `n` rows of d floats to out (f32 or bf16), in row order.
__global__ void __launch_bounds__(256) sum_rows_kernel(const float* part, int64_t n, int64_t d, void* out, int dtype) {
  __shared__ float s[8][33];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float acc = 0.0f;
  if (c < d) {
    constexpr int U = 8;  // loads in flight
    int64_t i = w;
    for (; i + (U - 1) * 8 < n; i += U * 8) {
      float x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] = __ldg(part + (i + u * 8) * d + c);
#pragma unroll
      for (int u = 0; u < U; ++u) acc += x[u];
    }
    for (; i < n; i += 8) acc += __ldg(part + i * d + c);
  }
  s[w][lane] = acc;
  __syncthreads();
  if (w != 0 || c >= d) return;
  acc = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc += s[i][lane];
  if (dtype == TPS_F32)
    static_cast<float*>(out)[c] = acc;
  else
    static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(acc);
}

int launch_sum_rows(const float* part, int64_t n, int64_t d, void* out, int dtype, cudaStream_t s) {
  ProfScope prof("sum_rows", "dw", 0.0, 4.0 * double(n) * double(d), s);
  sum_rows_kernel<<<static_cast<unsigned>((d + 31) / 32), 256, 0, s>>>(part, n, d, out, dtype);
  return launched("sum_rows");
}

}  // namespace tps

using namespace tps;

extern "C" int tps_rmsnorm_fwd(const tps_tensor* X, const tps_tensor* residual, const tps_tensor* weight, double eps,
                               const tps_dropout* dropout, const tps_tensor* H, const tps_tensor* Y,
                               const tps_tensor* scale, const tps_tensor* rstd, void* cuda_stream) {
  clear_detail();
  NormParams p = {};
  int64_t rows, d;
  int rc;
  if ((rc = rows_view(X, "X", false, &p.x, &rows, &d))) return rc;
  if (p.x.dtype == TPS_E4M3) return fail(TPS_ERR_DTYPE, "X must be f32 or bf16");
  if ((rc = too_large(rows, d))) return rc;
  if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(TPS_ERR_ARG, "eps must be finite and >= 0");
  if ((rc = dropout_of(dropout, &p.drop))) return rc;
  if (residual != nullptr && (rc = float_rows(residual, "residual", false, rows, d, &p.res))) return rc;
  const bool summed = residual != nullptr || (dropout != nullptr && dropout->p > 0.0);
  if (summed) {
    if ((rc = float_rows(H, "H", true, rows, d, &p.h))) return rc;
    if (p.h.dtype != (residual != nullptr ? p.res.dtype : p.x.dtype))
      return fail(TPS_ERR_DTYPE, "H must have the type of the %s", residual != nullptr ? "residual" : "input");
  } else if (H != nullptr) {
    return fail(TPS_ERR_ARG, "H is the input itself without a residual and without dropout");
  }
  int64_t n, c;
  if ((rc = rows_view(Y, "Y", true, &p.y, &n, &c))) return rc;
  if (n != rows || c != d) return fail(TPS_ERR_SHAPE, "Y: another shape than X");
  if ((rc = weight_vector(weight, d, &p.w, &p.w_dtype))) return rc;
  if ((p.y.dtype == TPS_E4M3) != (scale != nullptr)) return fail(TPS_ERR_ARG, "scale goes with an e4m3 output");
  if (scale != nullptr && (rc = expect_vector(scale, "scale", TPS_F32, rows))) return rc;
  if ((rc = expect_vector(rstd, "rstd", TPS_F32, rows))) return rc;
  if (rows == 0) return TPS_OK;
  if (d == 0) return fail(TPS_ERR_SHAPE, "rows without elements");
  p.rstd = static_cast<float*>(rstd->data);
  p.scale = scale != nullptr ? static_cast<float*>(scale->data) : nullptr;
  p.rows = rows;
  p.d = d;
  p.eps = static_cast<float>(eps);
  p.inv_d = static_cast<float>(1.0 / static_cast<double>(d));
  return launch_norm_fwd(p, "fwd", static_cast<cudaStream_t>(cuda_stream));
}

extern "C" int tps_quantize_e4m3(const tps_tensor* X, const tps_tensor* Q, const tps_tensor* scale, void* cuda_stream) {
  clear_detail();
  NormParams p = {};
  int64_t rows, d, n, c;
  int rc;
  if ((rc = rows_view(X, "X", false, &p.x, &rows, &d))) return rc;
  if (p.x.dtype == TPS_E4M3) return fail(TPS_ERR_DTYPE, "X must be f32 or bf16");
  if ((rc = too_large(rows, d))) return rc;
  if ((rc = rows_view(Q, "Q", true, &p.y, &n, &c))) return rc;
  if (n != rows || c != d) return fail(TPS_ERR_SHAPE, "Q: another shape than X");
  if (p.y.dtype != TPS_E4M3) return fail(TPS_ERR_DTYPE, "Q must be e4m3");
  if ((rc = expect_vector(scale, "scale", TPS_F32, rows))) return rc;
  if (rows == 0) return TPS_OK;
  p.scale = static_cast<float*>(scale->data);
  p.rows = rows;
  p.d = d;
  return launch_norm_fwd(p, "quantize", static_cast<cudaStream_t>(cuda_stream));
}

extern "C" size_t tps_rmsnorm_workspace_bytes(int64_t T, int64_t d) {
  if (T < 0 || d < 0) return 0;
  return align256(static_cast<size_t>(4 * (T < kMostBlocks ? T : kMostBlocks) * d));
}

extern "C" int tps_rmsnorm_bwd(const tps_tensor* dY, const tps_tensor* H, const tps_tensor* weight,
                               const tps_tensor* rstd, const tps_tensor* dH, const tps_dropout* dropout,
                               const tps_tensor* dSum, const tps_tensor* dX, const tps_tensor* dweight, void* workspace,
                               size_t workspace_bytes, void* cuda_stream) {
  clear_detail();
  NormBwdParams p = {};
  int64_t rows, d;
  int rc;
  if ((rc = rows_view(dY, "dY", false, &p.dy, &rows, &d))) return rc;
  if (p.dy.dtype == TPS_E4M3) return fail(TPS_ERR_DTYPE, "dY must be f32 or bf16");
  if ((rc = too_large(rows, d))) return rc;
  if ((rc = float_rows(H, "H", false, rows, d, &p.h))) return rc;
  if ((rc = weight_vector(weight, d, &p.w, &p.w_dtype))) return rc;
  if ((rc = expect_vector(rstd, "rstd", TPS_F32, rows))) return rc;
  if (dH != nullptr && (rc = float_rows(dH, "dH", false, rows, d, &p.dh))) return rc;
  if ((rc = dropout_of(dropout, &p.drop))) return rc;
  if (dSum != nullptr && (rc = float_rows(dSum, "dSum", true, rows, d, &p.dsum))) return rc;
  for (const Rows* g : {&p.dh, &p.dsum})
    if (g->p != nullptr && g->dtype != p.h.dtype) return fail(TPS_ERR_DTYPE, "dH and dSum must have H's type");
  if (dX != nullptr && (rc = float_rows(dX, "dX", true, rows, d, &p.dx))) return rc;
  if (dweight != nullptr && (rc = expect_vector(dweight, "dweight", TPS_F32, d))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (d == 0) return rows == 0 ? TPS_OK : fail(TPS_ERR_SHAPE, "rows without elements");
  if (rows == 0) return dweight != nullptr ? launch_fill(dweight->data, TPS_F32, 1, d, d, 1, s) : TPS_OK;
  const size_t need = dweight != nullptr ? tps_rmsnorm_workspace_bytes(rows, d) : 0;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255)))
    return fail(TPS_ERR_WORKSPACE, "workspace needs %zu bytes, 256-byte aligned", need);
  p.rstd = static_cast<const float*>(rstd->data);
  p.part = dweight != nullptr ? static_cast<float*>(workspace) : nullptr;
  p.rows = rows;
  p.d = d;
  p.inv_d = static_cast<float>(1.0 / static_cast<double>(d));
  const bool wide = d % 8 == 0 && starts_runs(p.dy, rows) && starts_runs(p.h, rows) && starts_runs(p.dh, rows) &&
                    starts_runs(p.dsum, rows) && starts_runs(p.dx, rows) &&
                    (p.w == nullptr || starts_runs(p.w, 0, p.w_dtype, 1));
  const int td = p.dy.dtype, th = p.h.dtype;
  const Spread sp = spread_of(d, wide, td == TPS_F32 || th == TPS_F32, td != th);
  int64_t parts = rows < kMostBlocks ? rows : kMostBlocks;
  if (p.part != nullptr || p.dsum.p != nullptr || p.dx.p != nullptr) {
    using bf16 = __nv_bfloat16;
    const double bytes = double(rows) * double(d) *
                         (es_of(p.dy.dtype) + es_of(p.h.dtype) + (p.dh.p ? es_of(p.dh.dtype) : 0) +
                          (p.dsum.p ? es_of(p.dsum.dtype) : 0) + (p.dx.p ? es_of(p.dx.dtype) : 0));
    ProfScope prof("norm", "bwd", 0.0, bytes, s);
    if (sp.N != 0) {
      rc = td == TPS_F32 ? (th == TPS_F32 ? launch_bwd_typed<float, float>(p, sp, &parts, s) : launch_bwd_typed<float, bf16>(p, sp, &parts, s))
                         : (th == TPS_F32 ? launch_bwd_typed<bf16, float>(p, sp, &parts, s) : launch_bwd_typed<bf16, bf16>(p, sp, &parts, s));
    } else {
      if (p.part != nullptr) {  // before the rows' kernel, which may write over dY
        norm_dw_kernel<<<dim3(static_cast<unsigned>((d + kDwCols - 1) / kDwCols), static_cast<unsigned>(parts)), kDwCols, 0, s>>>(p);
        if ((rc = launched("norm_dw"))) return rc;
      }
      if (wide)
        norm_bwd_long_kernel<8><<<static_cast<unsigned>(rows), kLongThreads, 0, s>>>(p);
      else
        norm_bwd_long_kernel<1><<<static_cast<unsigned>(rows), kLongThreads, 0, s>>>(p);
      rc = launched("norm_bwd_long");
    }
    if (rc) return rc;
  }
  return p.part != nullptr ? launch_sum_rows(p.part, parts, d, dweight->data, TPS_F32, s) : TPS_OK;
}
