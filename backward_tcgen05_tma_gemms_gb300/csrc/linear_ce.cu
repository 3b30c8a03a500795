// linear_ce.cu -- softmax cross entropy of a vocabulary head without keeping
// its logits, in pieces of the vocabulary.
//
//   z = h W,  lse_t = log sum_j e^{z_tj},  loss_t = lse_t - z_{t,y_t}
//   dz_tj = g_t (e^{z_tj - lse_t} - 1[j = y_t]),  dh = dz W^T,  dW = h^T dz
//
// ("多卡张量：拆开计算，再合回同一结果", 04 / VOCABULARY SHARDS gives the loss
// and dz over shards of the vocabulary: the maxima and sums of the pieces are
// what has to be combined, never the logits.)
//
// Forward, bf16: one tensor-core GEMM whose epilogue reduces each row's 128
// columns to (max, sum of e^{z - max}) while they are in tensor memory
// (EPI_CE_LSE), so T x V logits become T x V / 128 pairs, and one kernel that
// joins the pairs of a row.  2 T d V operations; the pairs are 1/32 of what
// bf16 logits would be.
//
// Backward, bf16: nothing but lse is kept, so each piece of the vocabulary
// has its logits formed again, and the epilogue turns them into dz at once
// (EPI_CE_GRAD: one exponential and one product an element; dz leaves as
// bf16, the type in which the tensor cores take it.  That leaves fp32 gradients
// 3e-5 to 3e-4 off, in the norm, where the rows share their upstream gradient,
// and 1.6e-3 where each token has one of its own, as much as bf16 gradients
// are; dz in two planes would double both products that read it).  The piece is
// then the K-major operand of dh += dz W_piece^T, summed over the pieces in
// fp32 by TMA reductions in piece order, and the MN-major operand of dW_piece.
// 6 T d V operations; forward and backward together take 8 T d V, where a
// pass that keeps T x V logits takes 6: a third more is what not keeping them
// costs.
//
// T = 8192, d = 4096, V = 128256, bf16: forward 4.9-5.0 ms (1720-1750
// TFLOP/s), backward 15.1-15.4 ms (1680-1710 TFLOP/s), the power cap's rate;
// workspace 66 MB and 0.65 GB, where the logits would be 2.1 GB in bf16.
//
// fp32 operands take the tensor cores too: each value is the sum of three
// bf16 values exactly (8 + 8 + 8 bits), and of the nine products of such
// planes the six that reach fp32's 2^-24 are summed into one fp32
// accumulator, smallest first (GemmDesc::planes); dz is split the same way in
// the epilogue.  Six times the tensor-core work of bf16 is still a fraction of
// the fp32 pipes' time (T = 512, d = 1024, V = 8192 backward: 247 us, 2216 us
// on the fp32 pipes).  These planes, and bf16 operands that TMA cannot
// describe, are laid out in the workspace, Whead one piece at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdlib>

#include "api_common.cuh"
#include "operand.cuh"
#include "ptx.cuh"

namespace tps {

namespace {

constexpr int64_t kRowBlock = 65536;       // rows of one forward GEMM: bounds the pairs' workspace
constexpr int64_t kPieceStep = 256;        // pieces start on whole pair tiles
constexpr int64_t kPieceBytes = 512ll << 20;  // one piece of dz by default

struct Labels {
  const void* p;
  int i64;
  int64_t ignore;
  int64_t vreal;
  __device__ int64_t at(int64_t t) const {
    return i64 ? static_cast<const int64_t*>(p)[t] : static_cast<int64_t>(static_cast<const int32_t*>(p)[t]);
  }
  // 0: a supervised label in [0, vreal); 1: ignore_index; 2: invalid.
  __device__ int kind(int64_t y) const {
    if (ignore != TPS_NO_IGNORE && y == ignore) return 1;
    return y >= 0 && y < vreal ? 0 : 2;
  }
};

// (m, s) += (m2, s2); (-inf, 0) is empty, a NaN in either s stays.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float M = fmaxf(m, m2);
  if (M == -INFINITY) {
    s += s2;
    return;
  }
  s = (m == -INFINITY ? s : s * ex2_approx((m - M) * kCeLog2e)) +
      (m2 == -INFINITY ? s2 : s2 * ex2_approx((m2 - M) * kCeLog2e));
  m = M;
}

// lse and loss of 32 rows from their pairs, pairs[tile * ld + row]: lane =
// row, each warp a run of tiles (consecutive rows are consecutive in memory,
// so every load of a warp is one 256-byte line pair), then the 32 partial
// pairs of a row in warp order.  At T = 8192 this reads 66 MB.
constexpr int kJoinWarps = 32;
__device__ __forceinline__ void ce_finish(int64_t t, float m, float s, float zy, const Labels& lab, float* loss,
                                          float* lse, uint32_t* err) {
  const float l = m + logf(s);
  lse[t] = l;
  const int kind = lab.kind(lab.at(t));
  loss[t] = kind == 1 ? 0.0f : (kind == 0 ? l - zy : __int_as_float(0x7fc00000));
  if (kind == 2) atomicOr(err, TPS_DEVERR_LABEL);
}
__global__ void __launch_bounds__(32 * kJoinWarps)
    ce_join_kernel(const float2* pairs, int64_t ld, int64_t tiles, int64_t rows, int64_t row0, const float* zy,
                   Labels lab, float* loss, float* lse, uint32_t* err) {
  __shared__ float2 part[kJoinWarps][33];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float m = -INFINITY, s = 0.0f;
  if (r < rows) {
    constexpr int U = 8;  // loads in flight
    for (int64_t i = w; i < tiles; i += U * kJoinWarps) {
      float2 e[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        e[u] = i + u * kJoinWarps < tiles ? __ldg(pairs + (i + u * kJoinWarps) * ld + r) : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int u = 0; u < U; ++u) join(m, s, e[u].x, e[u].y);
    }
  }
  part[w][lane] = make_float2(m, s);
  __syncthreads();
  if (w != 0 || r >= rows) return;
  m = -INFINITY;
  s = 0.0f;
  for (int i = 0; i < kJoinWarps; ++i) join(m, s, part[i][lane].x, part[i][lane].y);
  ce_finish(row0 + r, m, s, zy[r], lab, loss, lse, err);
}
// The same for a few rows: one block a row, threads along the tiles.
__global__ void __launch_bounds__(32 * kJoinWarps)
    ce_join_row_kernel(const float2* pairs, int64_t ld, int64_t tiles, const float* zy, Labels lab, float* loss,
                       float* lse, uint32_t* err) {
  __shared__ float2 part[kJoinWarps];
  const int64_t r = blockIdx.x;
  float m = -INFINITY, s = 0.0f;
  for (int64_t i = threadIdx.x; i < tiles; i += 32 * kJoinWarps) {
    const float2 e = __ldg(pairs + i * ld + r);
    join(m, s, e.x, e.y);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    join(m, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x != 0) return;
  m = -INFINITY;
  s = 0.0f;
  for (int i = 0; i < kJoinWarps; ++i) join(m, s, part[i].x, part[i].y);
  ce_finish(r, m, s, zy[r], lab, loss, lse, err);
}

// Sum over a block of 1024 threads, to thread 0.
template <class V>
__device__ __forceinline__ V block_sum(V x, V* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  V total = 0;
  if (threadIdx.x == 0)
    for (int i = 0; i < 32; ++i) total += red[i];
  return total;
}

// One block: the reduced loss, sum or mean, summed in fp64 in a fixed order.
__global__ void __launch_bounds__(1024) ce_total_kernel(const float* loss, int64_t T, Labels lab, int reduction,
                                                        double denominator, float* out) {
  __shared__ double red[32];
  __shared__ int64_t redi[32];
  double acc = 0.0;
  int64_t n = 0;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    acc += loss[t];
    if (reduction == TPS_REDUCE_MEAN && denominator == 0.0) n += lab.kind(lab.at(t)) == 0;
  }
  acc = block_sum(acc, red);
  n = block_sum(n, redi);
  if (threadIdx.x == 0) {
    double D = 1.0;
    if (reduction == TPS_REDUCE_MEAN) D = denominator > 0.0 ? denominator : (n > 0 ? double(n) : 1.0);
    *out = static_cast<float>(acc / D);
  }
}

// What the gradient epilogue knows of each row (Epilogue::ce_rows).  A mean
// over this call's labels needs their count first, and a gradient for each
// token their largest: one block then does both, else the rows are spread
// over blocks.  alpha (bf16 operands): the gradient that all rows share, a
// sum's or a mean's, or the largest of the tokens' magnitudes, is kept apart
// and the products multiplied by it in fp32; a row keeps its share of it.
// Inside dz it would be rounded to bf16 with the one-hot term, the same way in
// every row that has the same gradient, and leave the whole result off by up
// to 2^-9.  (One that is not finite stays in its rows.)
__global__ void __launch_bounds__(1024) ce_rows_kernel(int64_t T, Labels lab, const float* lse, const float* g,
                                                       int64_t g_step, int reduction, double denominator,
                                                       float4* rows, float* alpha, uint32_t* err) {
  __shared__ int64_t redi[32];
  __shared__ float redf[32];
  __shared__ float share, common;
  if (reduction == TPS_REDUCE_MEAN && denominator == 0.0) {  // one block
    int64_t n = 0;
    for (int64_t t = threadIdx.x; t < T; t += 1024) n += lab.kind(lab.at(t)) == 0;
    n = block_sum(n, redi);
    if (threadIdx.x == 0) share = static_cast<float>(1.0 / (n > 0 ? double(n) : 1.0));
  } else if (threadIdx.x == 0) {
    share = reduction == TPS_REDUCE_MEAN ? static_cast<float>(1.0 / denominator) : 1.0f;
  }
  float most = 0.0f;
  if (alpha != nullptr && g_step != 0) {  // one block: the largest finite magnitude
    for (int64_t t = threadIdx.x; t < T; t += 1024) {
      const float x = fabsf(g[t]);
      if (x < INFINITY && lab.kind(lab.at(t)) != 1) most = fmaxf(most, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if ((threadIdx.x & 31) == 0) redf[threadIdx.x >> 5] = most;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    common = 1.0f;
    if (alpha != nullptr) {
      if (g_step != 0) {
        for (int i = 0; i < 32; ++i) most = fmaxf(most, redf[i]);
        if (most > 0.0f) common = most;
      } else {
        const float x = (g == nullptr ? 1.0f : *g) * share;
        if (fabsf(x) < INFINITY && x != 0.0f) common = x;
      }
      if (blockIdx.x == 0) *alpha = common;
    }
  }
  __syncthreads();
  for (int64_t t = blockIdx.x * int64_t(1024) + threadIdx.x; t < T; t += int64_t(gridDim.x) * 1024) {
    const int64_t y = lab.at(t);
    const int kind = lab.kind(y);
    if (kind == 2) atomicOr(err, TPS_DEVERR_LABEL);
    const float up = (g == nullptr ? 1.0f : g[t * g_step]) * share;
    const float l = lse[t];
    rows[t] = make_float4(l * kCeLog2e, kind == 1 ? 0.0f : (alpha != nullptr ? __fdiv_rn(up, common) : up),
                          __int_as_float(kind == 0 ? static_cast<int>(y) : -1), l);
  }
}

// ---- a few tokens -----------------------------------------------------------
// With up to kFewTokens tokens the forward pass is one reading of Whead, and
// the 256-row tiles of the GEMM do it at half of the memory's rate (T = 1,
// d = 4096, V = 128256: 291 us, 3.6 TB/s: five stages of 16 KB of Whead an SM
// are not enough bytes in flight).  Here a block takes 128 columns, 16 bytes
// a thread and load with eight loads in flight, fp32 sums on the fp32 pipes,
// and leaves the pair of its columns for each token.
// Measured (us, d = 4096; bf16 V = 128256, fp32 V = 65536, (d, V) and (V, d)
// layout, the GEMM's time after the stroke): bf16 1 token 182 / 251 and
// 192 / 276, 2 tokens 243 / 270 and 240 / 237, from 4 on the GEMM is ahead;
// fp32 1 token 181 / 1720 and 206 / 1760, 4 tokens 271 / 1640 and 320 / 1740,
// 8 tokens 281 / 1530 (the GEMM lays the head out and has 256 rows of six
// products to do for them).
constexpr int kFewTokens = 8, kFewTokensBf16 = 2;
constexpr int kFewWarps = 8;
constexpr int kFewChunk = 1024;       // rows of Whead whose h is in shared memory
constexpr int kFewShared = 96 << 10;  // h of an OUT_IN call, whole

struct FewParams {
  const void* h;
  int64_t h_t, h_k;  // strides of token and k
  const void* w;
  int64_t ld;        // Whead's pitch
  int64_t T, d, V, vreal;
  Labels lab;
  float2* pairs;     // pairs[tile * T + t]
  float* zy;
};

template <class E> __device__ __forceinline__ float few_f(E x);
template <> __device__ __forceinline__ float few_f(float x) { return x; }
template <> __device__ __forceinline__ float few_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// 16 bytes from p, of which `left` elements exist.
template <class E, int N>
__device__ __forceinline__ void few_load(const E* p, int64_t left, E (&x)[N]) {
  if (left >= N) {
    *reinterpret_cast<uint4*>(x) = __ldg(reinterpret_cast<const uint4*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < left ? p[i] : E(0.0f);
  }
}

// The pair of 128 logits of each token, z[t * 128 + column], and the label's logit.
template <int TT>
__device__ __forceinline__ void few_pairs(const FewParams& p, const float* z, int64_t tile) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (w >= TT || w >= p.T) return;
  const int64_t col0 = tile * 128 + lane * 4;
  float4 q = reinterpret_cast<const float4*>(z + w * 128)[lane];
  float v[4] = {q.x, q.y, q.z, q.w}, m = -INFINITY, s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (col0 + i >= p.vreal) v[i] = -INFINITY;
    m = fmaxf(m, v[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
  for (int i = 0; i < 4; ++i) s += v[i] == -INFINITY ? 0.0f : expf(v[i] - m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) p.pairs[tile * p.T + w] = make_float2(m, s);
  const int64_t y = p.lab.at(w) - col0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (y == i && col0 + i < p.vreal) p.zy[w] = v[i];
}

// Whead with unit stride along the vocabulary: lanes along columns, warps
// (and halves of a warp) along k.
template <class E, int TT>
__global__ void __launch_bounds__(32 * kFewWarps) ce_few_in_out_kernel(const FewParams p) {
  constexpr int N = 16 / sizeof(E), kLanes = 128 / N, kRows = 32 / kLanes * kFewWarps, U = 8;
  __shared__ __align__(16) float sh[TT * 1024];  // h of a chunk [k][t], then the warps' sums [warp][t][128]
  static_assert(kFewWarps * 128 <= 1024 && kFewChunk <= 1024, "both uses fit");
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % kLanes * N, r0 = w * (32 / kLanes) + lane / kLanes;
  const int64_t tile = blockIdx.x, col = tile * 128 + c;
  float acc[TT][N];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int i = 0; i < N; ++i) acc[t][i] = 0.0f;
  for (int64_t k0 = 0; k0 < p.d; k0 += kFewChunk) {
    const int kn = static_cast<int>(p.d - k0 < kFewChunk ? p.d - k0 : kFewChunk);
    __syncthreads();
    for (int i = threadIdx.x; i < kn * TT; i += 32 * kFewWarps) {
      const int k = i / TT, t = i % TT;
      sh[i] = t < p.T ? few_f(static_cast<const E*>(p.h)[t * p.h_t + (k0 + k) * p.h_k]) : 0.0f;
    }
    __syncthreads();
    const E* src = static_cast<const E*>(p.w) + k0 * p.ld + col;
    auto add = [&](const E(&x)[N], int k) {
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const float hv = sh[k * TT + t];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[t][i] = fmaf(few_f(x[i]), hv, acc[t][i]);
      }
    };
    // U loads in flight, each behind its own test: written without the tests
    // the compiler took the loads one by one (T = 1: 215 us against 185).
    if (col < p.vreal) {
      for (int k = r0; k < kn; k += kRows * U) {
        __align__(16) E x[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k + u * kRows < kn) few_load<E, N>(src + (k + u * kRows) * p.ld, p.V - col, x[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k + u * kRows < kn) add(x[u], k + u * kRows);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float a = acc[t][i];
      if (kLanes == 16) a += __shfl_xor_sync(0xffffffffu, a, 16);
      if (lane < kLanes) sh[(w * TT + t) * 128 + c + i] = a;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < TT * 128; i += 32 * kFewWarps) {
    float a = 0.0f;
#pragma unroll
    for (int q = 0; q < kFewWarps; ++q) a += sh[q * TT * 128 + i];
    sh[i] = a;  // read and written by this thread alone: warp 0's part
  }
  __syncthreads();
  few_pairs<TT>(p, sh, tile);
}

// Whead with unit stride along k: a warp takes four vocabulary rows at a
// time, lanes along k.
template <class E, int TT>
__global__ void __launch_bounds__(32 * kFewWarps) ce_few_out_in_kernel(const FewParams p) {
  constexpr int N = 16 / sizeof(E), R = 4, kWarpRows = 128 / kFewWarps;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ __align__(16) float z[TT * 128];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tile = blockIdx.x, dp = (p.d + N - 1) / N * N;
  E* hs = reinterpret_cast<E*>(raw);  // [t][dp], zeros past d
  for (int64_t i = threadIdx.x; i < TT * dp; i += 32 * kFewWarps) {
    const int64_t t = i / dp, k = i - t * dp;
    hs[i] = t < p.T && k < p.d ? static_cast<const E*>(p.h)[t * p.h_t + k * p.h_k] : E(0.0f);
  }
  __syncthreads();
  for (int g = 0; g < kWarpRows; g += R) {
    const int row = w * kWarpRows + g;
    const int64_t v = tile * 128 + row;
    float acc[R][TT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[r][t] = 0.0f;
    const E* src[R];  // rows past the vocabulary read the last one; their sums are masked
#pragma unroll
    for (int r = 0; r < R; ++r)
      src[r] = static_cast<const E*>(p.w) + (v + r < p.V ? v + r : p.V - 1) * p.ld;
    auto add = [&](const E(&x)[R][N], int64_t k) {
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        __align__(16) E y[N];
        *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(hs + t * dp + k);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < N; ++i) acc[r][t] = fmaf(few_f(x[r][i]), few_f(y[i]), acc[r][t]);
      }
    };
    int64_t k = lane * N;
    for (; k + 32 * N + N <= p.d; k += 64 * N) {  // straight-line: 2 R loads in flight
      __align__(16) E x[2][R][N];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r)
          *reinterpret_cast<uint4*>(x[u][r]) = __ldg(reinterpret_cast<const uint4*>(src[r] + k + u * 32 * N));
#pragma unroll
      for (int u = 0; u < 2; ++u) add(x[u], k + u * 32 * N);
    }
    for (; k < p.d; k += 32 * N) {
      __align__(16) E x[R][N];
#pragma unroll
      for (int r = 0; r < R; ++r) few_load<E, N>(src[r] + k, p.d - k, x[r]);
      add(x, k);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        float a = acc[r][t];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if (lane == 0) z[t * 128 + row + r] = a;
      }
  }
  __syncthreads();
  few_pairs<TT>(p, z, tile);
}

// The fp32 sum over pieces to the caller's dHidden.
__global__ void __launch_bounds__(256) ce_convert_kernel(const float* a, int64_t lda, void* out, int dtype, int64_t rows,
                                                         int64_t cols, int64_t sr, int64_t sc, int vec) {
  if (vec) {  // 8 columns a thread, rows of whole 16-byte runs
    const int64_t per = cols / 8;
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < rows * per; i += int64_t(gridDim.x) * 256) {
      const int64_t r = i / per, c = (i % per) * 8;
      const float4 x = *reinterpret_cast<const float4*>(a + r * lda + c);
      const float4 y = *reinterpret_cast<const float4*>(a + r * lda + c + 4);
      __nv_bfloat162 b[4] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w),
                             __floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + r * sr + c) = *reinterpret_cast<uint4*>(b);
    }
    return;
  }
  for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < rows * cols; i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / cols, c = i % cols;
    const float x = a[r * lda + c];
    if (dtype == TPS_F32)
      static_cast<float*>(out)[r * sr + c * sc] = x;
    else
      static_cast<__nv_bfloat16*>(out)[r * sr + c * sc] = __float2bfloat16_rn(x);
  }
}

// ------------------------------------------------------------------ host

struct Call {  // what both directions check alike
  Mat h, w;
  int64_t T = 0, d = 0, V = 0, vreal = 0, w_in = 0, w_out = 0;
  int dt = 0;
  Labels lab = {};
  int reduction = TPS_REDUCE_NONE;
  double denominator = 0.0;
};

int check_call(const tps_tensor* h, const tps_tensor* Whead, const tps_tensor* labels, int32_t layout,
               const tps_ce_options* o, Call* c) {
  int rc;
  if ((rc = as_mat(h, "h", true, &c->h)) || (rc = as_mat(Whead, "Whead", false, &c->w))) return rc;
  if (layout != TPS_W_IN_OUT && layout != TPS_W_OUT_IN) return fail(TPS_ERR_ARG, "unknown weight layout %d", layout);
  const bool io = layout == TPS_W_IN_OUT;
  c->T = c->h.rows;
  c->d = c->h.cols;
  c->V = io ? c->w.cols : c->w.rows;
  if ((io ? c->w.rows : c->w.cols) != c->d)
    return fail(TPS_ERR_SHAPE, "Whead does not match h's width %lld", (long long)c->d);
  if (c->V < 1 || c->d < 1) return fail(TPS_ERR_SHAPE, "empty vocabulary or width");
  if (c->V >= (1ll << 31) || c->T >= (1ll << 31) || c->d >= (1ll << 31))
    return fail(TPS_ERR_SHAPE, "an extent of 2^31 or more");
  c->dt = c->h.dtype;
  if (c->dt == TPS_F32 && (c->T >= (1 << 29) || c->d >= (1 << 29) || c->V >= (1 << 29)))
    return fail(TPS_ERR_SHAPE, "an fp32 extent of 2^29 or more");  // three planes side by side stay below 2^31
  if ((c->dt != TPS_F32 && c->dt != TPS_BF16) || c->w.dtype != c->dt)
    return fail(TPS_ERR_DTYPE, "h and Whead must share f32 or bf16");
  if (labels == nullptr) return fail(TPS_ERR_ARG, "labels missing");
  if (labels->dtype != TPS_I64 && labels->dtype != TPS_I32) return fail(TPS_ERR_DTYPE, "labels must be i32 or i64");
  if ((rc = expect_vector(labels, "labels", labels->dtype, c->T))) return rc;
  weight_strides(c->w, layout, &c->w_in, &c->w_out);
  c->vreal = c->V;
  int64_t ignore = TPS_NO_IGNORE;
  if (o != nullptr) {
    if (o->vocab_size < 0 || o->vocab_size > c->V)
      return fail(TPS_ERR_SHAPE, "vocab_size %lld outside [0, %lld]", (long long)o->vocab_size, (long long)c->V);
    if (o->vocab_size > 0) c->vreal = o->vocab_size;
    if (o->reduction != TPS_REDUCE_NONE && o->reduction != TPS_REDUCE_SUM && o->reduction != TPS_REDUCE_MEAN)
      return fail(TPS_ERR_ARG, "unknown reduction %d", o->reduction);
    if (!(o->denominator >= 0.0) || !std::isfinite(o->denominator))
      return fail(TPS_ERR_ARG, "denominator must be finite and >= 0");
    if (o->reserved != 0) return fail(TPS_ERR_ARG, "reserved must be 0");
    ignore = o->ignore_index;
    c->reduction = o->reduction;
    c->denominator = o->denominator;
  }
  c->lab = Labels{labels->data, labels->dtype == TPS_I64 ? 1 : 0, ignore, c->vreal};
  return TPS_OK;
}

struct Layout {  // of all operands of a call
  bool direct = true;  // bf16 as TMA takes it
  int planes = 1;
};

Layout layout_of(const Call& c) {
  Layout l;
  l.planes = c.dt == TPS_F32 ? 3 : 1;
  GemmDesc g;  // the logits GEMM as it would be
  g.M = c.T; g.N = c.vreal; g.K = c.d; g.in_dtype = c.dt;
  g.a = c.h.data; g.a_sm = c.h.sr; g.a_sk = c.h.sc;
  g.b = c.w.data; g.b_sk = c.w_in; g.b_sn = c.w_out;
  l.direct = c.dt == TPS_BF16 && tma_can(g.a, g.a_sm, g.a_sk) && tma_can(g.b, g.b_sk, g.b_sn) && gemm_tc_supported(g);
  return l;
}
int launched(const char* what) {
  note_launch();
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? TPS_OK : fail(TPS_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(cudaGetLastError()));
}

int lay_out(const Call& c, const char* src, int64_t ni, int64_t nj, int64_t si, int64_t sj, char* dst, cudaStream_t s,
            Operand* o) {
  return lay_operand(c.dt, src, ni, nj, si, sj, dst, "lce", s, o);
}
// The piece [v0, v0 + n) of Whead as Operand(d, v).
int head_piece(const Call& c, const Layout& l, int64_t v0, int64_t n, char* room, cudaStream_t s, Operand* o) {
  const int64_t es = c.dt == TPS_F32 ? 4 : 2;
  const char* src = static_cast<const char*>(c.w.data) + v0 * c.w_out * es;
  if (!l.direct) return lay_out(c, src, c.d, n, c.w_in, c.w_out, room, s, o);
  *o = Operand{src, c.w_in, c.w_out, 0, 0};
  return TPS_OK;
}
int hidden(const Call& c, const Layout& l, char* room, cudaStream_t s, Operand* o) {
  if (!l.direct) return lay_out(c, static_cast<const char*>(c.h.data), c.T, c.d, c.h.sr, c.h.sc, room, s, o);
  *o = Operand{static_cast<const char*>(c.h.data), c.h.sr, c.h.sc, 0, 0};
  return TPS_OK;
}
GemmDesc gemm_of(const char* name, const Layout& l, int64_t M, int64_t N, int64_t K) {
  GemmDesc g;
  g.name = name;
  g.M = M; g.N = N; g.K = K; g.in_dtype = TPS_BF16;
  g.planes = l.planes;
  return g;
}

// Whether the few-token kernels take a forward call.
bool few_tokens(const Call& c) {
  const char* most = getenv("TPS_LCE_FEW");
  if (c.T < 1 || c.T > (c.dt == TPS_F32 ? kFewTokens : kFewTokensBf16) || (most != nullptr && c.T > atoi(most))) return false;
  const int64_t es = c.dt == TPS_F32 ? 4 : 2, pitch = c.w_out == 1 ? c.w_in : c.w_out;
  if ((reinterpret_cast<uintptr_t>(c.w.data) & 15u) != 0 || pitch * es % 16 != 0) return false;
  const int64_t tt = c.T <= 1 ? 1 : c.T <= 2 ? 2 : c.T <= 4 ? 4 : 8;
  return c.w_out == 1 || (c.w_in == 1 && tt * (c.d + 16) * es <= kFewShared);
}
template <class E, int TT>
int launch_few(const Call& c, const FewParams& p, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>((c.vreal + 127) / 128);
  ProfScope prof("ce_few", "lce", 2.0 * double(c.T) * double(c.d) * double(c.vreal), double(c.d) * double(c.vreal) * sizeof(E), s);
  if (c.w_out == 1) {
    ce_few_in_out_kernel<E, TT><<<blocks, 32 * kFewWarps, 0, s>>>(p);
  } else {
    static PerDevice<bool> ready;
    if (!allow_shared(ready, ce_few_out_in_kernel<E, TT>, kFewShared))
      return fail(TPS_ERR_CUDA, "ce_few: %s", cudaGetErrorString(cudaGetLastError()));
    const size_t n = 16 / sizeof(E);
    ce_few_out_in_kernel<E, TT><<<blocks, 32 * kFewWarps, TT * ((c.d + n - 1) / n * n) * sizeof(E), s>>>(p);
  }
  return launched("ce_few");
}
template <class E>
int few_of(const Call& c, const FewParams& p, cudaStream_t s) {
  if (c.T <= 1) return launch_few<E, 1>(c, p, s);
  if (c.T <= 2) return launch_few<E, 2>(c, p, s);
  if constexpr (sizeof(E) == 4) {
    if (c.T <= 4) return launch_few<E, 4>(c, p, s);
    return launch_few<E, 8>(c, p, s);
  }
  return fail(TPS_ERR_ARG, "ce_few: too many tokens");
}

// Columns of one piece that fit into `room` bytes at `column_bytes` per column.
int64_t piece_columns(int64_t V, int64_t room, int64_t column_bytes) {
  const int64_t most = round_up(V, kPieceStep);
  const int64_t fit = column_bytes > 0 ? room / column_bytes / kPieceStep * kPieceStep : most;
  return fit < most ? fit : most;
}
// Bytes of a piece's buffers per vocabulary column: dz, and Whead laid out.
int64_t column_bytes(int64_t T, int64_t d, bool direct, int planes, bool backward) {
  return (backward ? 2 * planes * T : 0) + (direct ? 0 : 2 * planes * round_up(d, 64));
}

struct Fixed {  // workspace before the pieces
  size_t pairs, zy, rows, alpha, flags, acc, h, pieces;
};
Fixed fixed_layout(int64_t T, int64_t d, int64_t V, bool direct, int planes, bool backward) {
  Fixed f = {};
  size_t at = 0;
  auto take = [&at](int64_t bytes) {
    const size_t p = at;
    at += align256(static_cast<size_t>(bytes));
    return p;
  };
  if (!backward) {
    f.pairs = take(8 * ((V + kStatsTileN - 1) / kStatsTileN) * (T < kRowBlock ? T : kRowBlock));
    f.zy = take(4 * T);
  } else {
    f.rows = take(16 * T);
    f.alpha = take(4);
    f.flags = take(4 * pair_tile_count(T, d));
    f.acc = take(4 * T * round_up(d, 4));
  }
  if (!direct) f.h = take(laid_bytes(T, d, planes));
  f.pieces = at;
  return f;
}
// Where a piece's columns are laid out: behind its dz.
size_t head_room(const Fixed& f, int64_t T, int planes, bool backward, int64_t cols) {
  return f.pieces + (backward ? align256(static_cast<size_t>(2 * planes * T * cols)) : 0);
}

// Tiles and K split of the dh GEMM over a piece of k_tiles K tiles: 256 x 512
// (wide) or 256 x 256 pair tiles, and the runs whose partial sums are added in
// order.  Its time follows waves of (tile, run) units, a K tile costing 0.555
// or 0.31 us, and some 8 us for each run's addition, which waits for the run
// before it.  Measured (us): T = 1000, d = 2048, 501 K tiles: wide with 1, 2,
// 4, 5, 9 runs 278, 156, 107, 159, 133, narrow with 1, 2, 4, 9 runs 156, 94,
// 100, 106; T = 8192, d = 4096, 512 K tiles: wide with 1, 2, 3, 4 runs 1286,
// 1190, 1251, 1243.  (fp32 planes are narrow and go by the same figures.)
// TPS_LCE_SPLIT=wr forces wide (w = 0, 1) and the runs r, for tests: small
// shapes would take neither wide tiles nor runs.
struct Split {
  bool wide = false;
  int runs = 1;
};
Split choose_split(int64_t T, int64_t d, int64_t k_tiles, bool may_wide) {
  Split best;
  const char* forced = getenv("TPS_LCE_SPLIT");
  if (forced != nullptr && (forced[0] == '0' || forced[0] == '1') && atoi(forced + 1) >= 1) {
    best.wide = forced[0] == '1' && may_wide;
    best.runs = static_cast<int>(atoi(forced + 1) < k_tiles ? atoi(forced + 1) : k_tiles);
    return best;
  }
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 2)
    return best;
  const int64_t pairs = sms / 2;
  double least = 0.0;
  for (int wide = 0; wide <= (may_wide ? 1 : 0); ++wide) {
    const int64_t tiles = wide ? wide_tile_count(T, d) : pair_tile_count(T, d);
    for (int runs = 1; runs <= 16 && (runs == 1 || k_tiles / runs >= 16); ++runs) {
      const int64_t waves = (tiles * runs + pairs - 1) / pairs, steps = (k_tiles + runs - 1) / runs;
      const double us = double(waves) * double(steps) * (wide ? 0.555 : 0.31) + (runs > 1 ? 8.0 * runs : 0.0);
      if (least == 0.0 || us < least) {
        least = us;
        best.wide = wide != 0;
        best.runs = runs;
      }
    }
  }
  return best;
}

}  // namespace

}  // namespace tps

using namespace tps;

extern "C" size_t tps_linear_ce_workspace_bytes(int64_t T, int64_t d, int64_t V, int32_t dtype, int32_t backward,
                                                int64_t piece) {
  if (T < 0 || d < 1 || V < 1 || piece < 0 || (dtype != TPS_F32 && dtype != TPS_BF16)) return 0;
  // The bytes for fp32 also serve bf16 operands that have to be laid out.
  const bool direct = dtype == TPS_BF16;
  const int planes = direct ? 1 : 3;
  const int64_t per = column_bytes(T, d, direct, planes, backward != 0);
  const int64_t cols = piece > 0 ? round_up(piece < V ? piece : V, kPieceStep)
                                 : piece_columns(V, kPieceBytes > kPieceStep * per ? kPieceBytes : kPieceStep * per, per);
  return fixed_layout(T, d, V, direct, planes, backward != 0).pieces + align256(static_cast<size_t>(per) * cols) + 512;
}

extern "C" int tps_linear_ce_fwd(const tps_tensor* h, const tps_tensor* Whead, const tps_tensor* labels,
                                 int32_t weight_layout, const tps_ce_options* options, const tps_tensor* loss,
                                 const tps_tensor* loss_reduced, const tps_tensor* lse, void* workspace,
                                 size_t workspace_bytes, void* cuda_stream) {
  clear_detail();
  Call c;
  int rc;
  if ((rc = check_call(h, Whead, labels, weight_layout, options, &c))) return rc;
  if ((rc = expect_vector(loss, "loss", TPS_F32, c.T)) || (rc = expect_vector(lse, "lse", TPS_F32, c.T))) return rc;
  float* total = nullptr;
  if (loss_reduced != nullptr && loss_reduced->data != nullptr) {
    if ((rc = expect_vector(loss_reduced, "loss_reduced", TPS_F32, 1))) return rc;
    total = static_cast<float*>(loss_reduced->data);
  }
  if (c.reduction == TPS_REDUCE_NONE) total = nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (c.T == 0) {
    if (total != nullptr && cudaMemsetAsync(total, 0, sizeof(float), s) != cudaSuccess)
      return fail(TPS_ERR_CUDA, "memset failed");
    return TPS_OK;
  }
  const Layout l = layout_of(c);
  const Fixed f = fixed_layout(c.T, c.d, c.V, l.direct, l.planes, false);
  const int64_t per = column_bytes(c.T, c.d, l.direct, l.planes, false);
  const size_t least = f.pieces + static_cast<size_t>(kPieceStep * per) + 256;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < least)
    return fail(TPS_ERR_WORKSPACE, "workspace needs at least %zu bytes, 256-byte aligned", least);
  uint32_t* err = device_error_word();
  if (err == nullptr) return fail(TPS_ERR_CUDA, "cannot resolve the device error word");
  char* ws = static_cast<char*>(workspace);
  float2* pairs = reinterpret_cast<float2*>(ws + f.pairs);
  float* zy = reinterpret_cast<float*>(ws + f.zy);
  float* loss_p = static_cast<float*>(loss->data);
  float* lse_p = static_cast<float*>(lse->data);
  const int64_t cols = piece_columns(c.vreal, static_cast<int64_t>(workspace_bytes - f.pieces) - 256, per);
  const int64_t tiles = (c.vreal + kStatsTileN - 1) / kStatsTileN, label_bytes = c.lab.i64 ? 8 : 4;
  Operand x, w;
  const bool few = few_tokens(c);
  if (few) {
    const FewParams p = {c.h.data, c.h.sr, c.h.sc, c.w.data, c.w_out == 1 ? c.w_in : c.w_out, c.T, c.d, c.V, c.vreal,
                         c.lab, pairs, zy};
    rc = c.dt == TPS_F32 ? few_of<float>(c, p, s) : few_of<__nv_bfloat16>(c, p, s);
  } else {
    rc = hidden(c, l, ws + f.h, s, &x);
  }
  if (rc) return rc;
  for (int64_t r0 = 0; r0 < c.T; r0 += kRowBlock) {
    const int64_t rows = c.T - r0 < kRowBlock ? c.T - r0 : kRowBlock;
    for (int64_t v0 = 0; !few && v0 < c.vreal; v0 += cols) {
      const int64_t n = c.vreal - v0 < cols ? c.vreal - v0 : cols;
      if ((rc = head_piece(c, l, v0, n, ws + f.pieces, s, &w))) return rc;
      GemmDesc g = gemm_of("lce_logits", l, rows, n, c.d);
      set_a(&g, x, false);
      g.a = x.p + r0 * x.si * 2;
      if (g.a_cols > 0 && x.si == 1) g.a_cols -= r0;
      set_b(&g, w, false);
      g.epi.mode = EPI_CE_LSE;
      g.epi.stats = reinterpret_cast<float*>(pairs + v0 / kStatsTileN * rows);
      g.epi.stats_ld = rows;
      g.epi.ce_col0 = v0;
      g.epi.ce_labels = static_cast<const char*>(c.lab.p) + r0 * label_bytes;
      g.epi.ce_label_i64 = c.lab.i64;
      g.epi.ce_zy = zy + r0;
      if ((rc = run_gemm(g, n, 1, s))) return rc;
    }
    ProfScope prof("ce_join", "lce", 0.0, 8.0 * double(rows) * double(tiles), s);
    if (c.T < 152)  // fewer rows than would keep every SM busy 32 at a time
      ce_join_row_kernel<<<static_cast<unsigned>(rows), 32 * kJoinWarps, 0, s>>>(pairs, rows, tiles, zy, c.lab, loss_p,
                                                                                lse_p, err);
    else
      ce_join_kernel<<<static_cast<unsigned>((rows + 31) / 32), 32 * kJoinWarps, 0, s>>>(
          pairs, rows, tiles, rows, r0, zy + r0, c.lab, loss_p, lse_p, err);
    if ((rc = launched("ce_join"))) return rc;
  }
  if (total != nullptr) {
    ce_total_kernel<<<1, 1024, 0, s>>>(loss_p, c.T, c.lab, c.reduction, c.denominator, total);
    if ((rc = launched("ce_total"))) return rc;
  }
  return TPS_OK;
}

extern "C" int tps_linear_ce_bwd(const tps_tensor* h, const tps_tensor* Whead, const tps_tensor* labels,
                                 const tps_tensor* lse, const tps_tensor* grad_loss, int32_t weight_layout,
                                 const tps_ce_options* options, const tps_tensor* dHidden, const tps_tensor* dWhead,
                                 void* workspace, size_t workspace_bytes, void* cuda_stream) {
  clear_detail();
  Call c;
  int rc;
  if ((rc = check_call(h, Whead, labels, weight_layout, options, &c))) return rc;
  if ((rc = expect_vector(lse, "lse", TPS_F32, c.T))) return rc;
  const float* up = nullptr;
  int64_t up_step = 0;
  if (grad_loss != nullptr && grad_loss->data != nullptr) {
    const bool per_token = c.reduction == TPS_REDUCE_NONE;
    if ((rc = expect_vector(grad_loss, "grad_loss", TPS_F32, per_token ? c.T : 1))) return rc;
    up = static_cast<const float*>(grad_loss->data);
    up_step = per_token ? 1 : 0;
  }
  Mat dh, dw;
  const bool want_dh = dHidden != nullptr, want_dw = dWhead != nullptr;
  if (want_dh) {
    if ((rc = as_mat(dHidden, "dHidden", true, &dh)) || (rc = expect(dh, "dHidden", c.T, c.d))) return rc;
    if (dh.dtype != TPS_F32 && dh.dtype != TPS_BF16) return fail(TPS_ERR_DTYPE, "dHidden must be f32 or bf16");
  }
  int64_t dw_in = 0, dw_out = 0;
  if (want_dw) {
    if ((rc = as_mat(dWhead, "dWhead", false, &dw)) || (rc = expect(dw, "dWhead", c.w.rows, c.w.cols))) return rc;
    if (dw.dtype != TPS_F32 && dw.dtype != TPS_BF16) return fail(TPS_ERR_DTYPE, "dWhead must be f32 or bf16");
    weight_strides(dw, weight_layout, &dw_in, &dw_out);
  }
  if (!want_dh && !want_dw) return fail(TPS_ERR_ARG, "neither dHidden nor dWhead is wanted");
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const int64_t dw_es = dw.dtype == TPS_F32 ? 4 : 2;
  if (want_dw && (c.T == 0 || c.vreal < c.V)) {  // columns that no token reaches
    const int64_t v0 = c.T == 0 ? 0 : c.vreal;
    if ((rc = launch_fill(static_cast<char*>(dw.data) + v0 * dw_out * dw_es, dw.dtype, c.d, c.V - v0, dw_in, dw_out, s)))
      return rc;
  }
  if (c.T == 0) return TPS_OK;

  const Layout l = layout_of(c);
  const Fixed f = fixed_layout(c.T, c.d, c.V, l.direct, l.planes, true);
  const int64_t per = column_bytes(c.T, c.d, l.direct, l.planes, true);
  const size_t least = f.pieces + static_cast<size_t>(kPieceStep * per) + 256;  // 256: between a piece's two buffers
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < least)
    return fail(TPS_ERR_WORKSPACE, "workspace needs at least %zu bytes, 256-byte aligned", least);
  uint32_t* err = device_error_word();
  if (err == nullptr) return fail(TPS_ERR_CUDA, "cannot resolve the device error word");
  char* ws = static_cast<char*>(workspace);
  float4* rows = reinterpret_cast<float4*>(ws + f.rows);
  uint32_t* flags = reinterpret_cast<uint32_t*>(ws + f.flags);
  // without an upstream gradient each token's is 1, which dz holds exactly
  float* alpha = l.planes == 1 && (c.reduction != TPS_REDUCE_NONE || up != nullptr) ? reinterpret_cast<float*>(ws + f.alpha)
                                                                                    : nullptr;
  const int64_t cols = piece_columns(c.vreal, static_cast<int64_t>(workspace_bytes - f.pieces) - 256, per);

  {
    const bool count = (c.reduction == TPS_REDUCE_MEAN && c.denominator == 0.0) || (alpha != nullptr && up_step != 0);
    const int64_t blocks = count ? 1 : (c.T + 1023) / 1024;
    ce_rows_kernel<<<static_cast<unsigned>(blocks < 1024 ? blocks : 1024), 1024, 0, s>>>(
        c.T, c.lab, static_cast<const float*>(lse->data), up, up_step, c.reduction, c.denominator, rows, alpha, err);
    if ((rc = launched("ce_rows"))) return rc;
  }
  // dh is summed over the pieces in fp32: in the caller's buffer where that
  // is fp32 rows that TMA can add to, else in the workspace.
  float* acc = reinterpret_cast<float*>(ws + f.acc);
  int64_t ld_acc = round_up(c.d, 4);
  const bool direct = want_dh && dh.dtype == TPS_F32 && dh.sc == 1 &&
                      (reinterpret_cast<uintptr_t>(dh.data) & 15u) == 0 && dh.sr % 4 == 0 && dh.sr >= c.d;
  if (direct) {
    acc = static_cast<float*>(dh.data);
    ld_acc = dh.sr;
  }
  char* dz_p = ws + f.pieces;  // T x cols, or its planes side by side
  const Operand dz = {dz_p, l.planes * cols, 1, l.planes > 1 ? cols : 0, l.planes > 1 ? l.planes * cols : 0};
  char* w_room = ws + head_room(f, c.T, l.planes, true, cols);
  Operand x, w;
  if ((rc = hidden(c, l, ws + f.h, s, &x))) return rc;
  for (int64_t v0 = 0; v0 < c.vreal; v0 += cols) {
    const int64_t n = c.vreal - v0 < cols ? c.vreal - v0 : cols;
    if ((rc = head_piece(c, l, v0, n, w_room, s, &w))) return rc;
    GemmDesc g = gemm_of("lce_dlogits", l, c.T, n, c.d);
    set_a(&g, x, false);
    set_b(&g, w, false);
    g.epi.mode = EPI_CE_GRAD;
    g.epi.d = dz_p; g.epi.d_dtype = TPS_BF16;
    g.epi.ce_rows = rows;
    g.epi.ce_col0 = v0;
    g.d_plane = dz.plane;
    g.n_store = round_up(n, 64);
    if ((rc = run_gemm(g, dz.si, 1, s))) return rc;
    if (want_dh) {  // dh += dz W_piece^T
      GemmDesc q = gemm_of("lce_dhidden", l, c.T, c.d, n);
      set_a(&q, dz, false);
      set_b(&q, w, true);
      q.epi.d = acc; q.epi.ldd = ld_acc;
      q.epi.accumulate = v0 > 0;
      q.epi.alpha = alpha;
      q.wide = true;
      const Split split = choose_split(c.T, c.d, (n + 63) / 64 * (l.planes > 1 ? 6 : 1), gemm_wide_supported(q));
      q.wide = split.wide;
      q.ksplit = split.runs;
      if (q.ksplit > 1) {
        const int64_t tiles = q.wide ? wide_tile_count(c.T, c.d) : pair_tile_count(c.T, c.d);
        if (cudaMemsetAsync(flags, 0, static_cast<size_t>(tiles) * sizeof(uint32_t), s) != cudaSuccess)
          return fail(TPS_ERR_CUDA, "memset failed");
        q.kflags = flags;
        q.pair = true;
      }
      if ((rc = run_gemm(q, ld_acc, 1, s))) return rc;
    }
    if (want_dw) {  // dW_piece = h^T dz
      GemmDesc q = gemm_of("lce_dwhead", l, c.d, n, c.T);
      set_a(&q, x, true);
      set_b(&q, dz, false);
      q.epi.d = static_cast<char*>(dw.data) + v0 * dw_out * dw_es; q.epi.d_dtype = dw.dtype;
      q.epi.alpha = alpha;
      if ((rc = run_gemm(q, dw_in, dw_out, s))) return rc;
    }
  }
  if (want_dh && !direct) {
    const bool vec = dh.dtype == TPS_BF16 && dh.sc == 1 && c.d % 8 == 0 && dh.sr % 8 == 0 &&
                     (reinterpret_cast<uintptr_t>(dh.data) & 15u) == 0;
    const int64_t items = vec ? c.T * c.d / 8 : c.T * c.d;
    const int64_t blocks = (items + 255) / 256;
    ProfScope prof("ce_convert", "lce", 0.0, 6.0 * double(c.T) * double(c.d), s);
    ce_convert_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(
        acc, ld_acc, dh.data, dh.dtype, c.T, c.d, dh.sr, dh.sc, vec ? 1 : 0);
    if ((rc = launched("ce_convert"))) return rc;
  }
  return TPS_OK;
}
