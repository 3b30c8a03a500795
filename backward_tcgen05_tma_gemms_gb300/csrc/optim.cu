// optim.cu -- the AdamW step of many tensors in one launch, and the global
// norm of their gradients.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   w = w (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// g is the gradient times a device scalar (the clip coefficient of
// tps_grad_norm); where that scalar is not finite nothing is changed.
//
// Moments in 8 bits hold m and sqrt(v) as e4m3 numbers with one fp32 scale
// for every 256 elements (the largest magnitude / 448).  sqrt(v) rather than
// v halves the binades a block has to span; what is not zero is not rounded
// to zero there, or m / sqrt(v) of a small element would explode.  A step
// changes v by a factor of b2, far less than half a step of e4m3: rounded to
// nearest it would never move.  So values go up or down at random, with the
// probability that keeps their expectation, by 16 bits of a hash of the
// element's place and the step's seed (multiply-xorshift mixing with the
// multipliers of C. Wellons' search, "Prospecting for hash functions",
// 2018).  bf16 weights without an fp32 master copy are rounded the same way.
//
// Bound by memory: one warp takes 256 elements (a block of the 8-bit form),
// 2 x 4 a lane, so every load of a warp is consecutive, and the block's
// maxima are two warp reductions.  The tensors' table travels in the kernel
// parameters: no copy, no workspace, nothing to keep alive.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "api_common.cuh"

namespace tps {

namespace {

constexpr int kUnit = TPS_ADAMW_BLOCK;  // elements of a warp's unit
constexpr int kWarps = 8;               // warps of a block

struct Entry {
  void* p;
  const void* g;
  float* w;  // fp32 master copy
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n, place, first;  // elements, place of the first in the random stream, first unit
  int64_t wide;             // every pointer is 16-byte aligned
};

template <int N>
struct Table {
  int32_t count;
  int32_t stochastic;
  int64_t units;
  const float* coef;
  const tps_adamw_scalars* dev;  // read instead of `s` when given
  tps_adamw_scalars s;
  float b1, c1, b2, c2, eps;
  Entry e[N];
};

__device__ __forceinline__ uint32_t mix(uint64_t place, uint32_t seed) {
  uint32_t x = (static_cast<uint32_t>(place) * 0x9e3779b1u + static_cast<uint32_t>(place >> 32) * 0x85ebca77u) ^ seed;
  x = (x ^ (x >> 16)) * 0x2c1b3c6du;
  x = (x ^ (x >> 12)) * 0x297a2d39u;
  return x ^ (x >> 15);
}
// fp32 to the bf16 below or above by 16 random bits.
__device__ __forceinline__ __nv_bfloat16 bf16_by(float x, uint32_t rnd) {
  const uint32_t b = __float_as_uint(x);
  // infinities and NaN have no neighbour to go to
  const uint32_t r = (b & 0x7f800000u) == 0x7f800000u ? b : b + rnd;
  return __ushort_as_bfloat16(static_cast<unsigned short>(r >> 16));
}
// y in [0, 448] to e4m3 by 16 random bits: numbers of at least 2^-6 have 3
// mantissa bits, smaller ones lie on the grid of 2^-9.
__device__ __forceinline__ uint32_t e4m3_by(float y, uint32_t rnd) {
  const uint32_t big = ((__float_as_uint(y) + (rnd << 4)) >> 20) - 960u;
  const uint32_t small = static_cast<uint32_t>(__fadd_rn(y * 512.0f, static_cast<float>(rnd) * 0x1p-16f));
  return y >= 0x1p-6f ? big : small;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {  // sign, 4 exponent bits, 3 mantissa bits
  const uint32_t mag = code & 0x7fu;
  // a float whose exponent field is the code's times 2^120 is the number, subnormals included
  const float x = __uint_as_float(mag << 20) * 0x1p120f;
  return code & 0x80u ? -x : x;
}

// Four consecutive elements.
__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const float4 q = *reinterpret_cast<const float4*>(p);
  x[0] = q.x; x[1] = q.y; x[2] = q.z; x[3] = q.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(q.x << 16); x[1] = __uint_as_float(q.x & 0xffff0000u);
  x[2] = __uint_as_float(q.y << 16); x[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const __nv_bfloat16 (&x)[4]) {
  uint2 q;
  q.x = __bfloat16_as_ushort(x[0]) | static_cast<uint32_t>(__bfloat16_as_ushort(x[1])) << 16;
  q.y = __bfloat16_as_ushort(x[2]) | static_cast<uint32_t>(__bfloat16_as_ushort(x[3])) << 16;
  *reinterpret_cast<uint2*>(p) = q;
}

// The index of element i (0..3) of group j (0, 1) of a lane within a unit.
__device__ __forceinline__ int in_unit(int lane, int j) { return j * 128 + lane * 4; }

// The eight values of a lane, `n` of the unit's 256 being there.
template <class T>
__device__ __forceinline__ void read8(const T* p, int lane, bool full, int n, float (&x)[2][4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = in_unit(lane, j);
    if (full) {
      load4(p + at, x[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] = at + i < n ? load1(p + at + i) : 0.0f;
    }
  }
}
template <class T>
__device__ __forceinline__ void write8(T* p, int lane, bool full, int n, const T (&x)[2][4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = in_unit(lane, j);
    if (full) {
      store4(p + at, x[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i < n) p[at + i] = x[j][i];
    }
  }
}
__device__ __forceinline__ void read8_codes(const uint8_t* p, int lane, bool full, int n, float scale, float (&x)[2][4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = in_unit(lane, j);
    uint32_t q = 0;
    if (full) {
      q = *reinterpret_cast<const uint32_t*>(p + at);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i < n) q |= static_cast<uint32_t>(p[at + i]) << (8 * i);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[j][i] = __fmul_rn(e4m3_value((q >> (8 * i)) & 0xffu), scale);
  }
}
// x as e4m3 numbers with the block's scale.  SQRT: x >= 0 and nothing but 0 becomes 0.
template <bool SQRT>
__device__ __forceinline__ void write8_codes(uint8_t* p, float* scale, int lane, bool full, int n,
                                             const float (&x)[2][4], const uint32_t (&rnd)[2][4]) {
  uint32_t top = 0;  // as bits, so that a NaN is the largest
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(x[j][i]) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  float a = __uint_as_float(top);
  if (a < 1e-30f) a = 0.0f;
  const float inv = a > 0.0f ? __fdiv_rn(448.0f, a) : (a == 0.0f ? 0.0f : a);
  if (lane == 0) *scale = __fmul_rn(a, 1.0f / 448.0f);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t q = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y = fminf(__fmul_rn(fabsf(x[j][i]), inv), 448.0f);
      uint32_t c = e4m3_by(y, rnd[j][i]);
      if (SQRT) {
        if (c == 0 && y > 0.0f) c = 1;
      } else if (c != 0 && x[j][i] < 0.0f) {
        c |= 0x80u;
      }
      q |= c << (8 * i);
    }
    const int at = in_unit(lane, j);
    if (full) {
      *reinterpret_cast<uint32_t*>(p + at) = q;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i < n) p[at + i] = static_cast<uint8_t>(q >> (8 * i));
    }
  }
}

template <class PT, class GT, bool MASTER, bool E4M3, int N>
__global__ void __launch_bounds__(32 * kWarps) adamw_kernel(const __grid_constant__ Table<N> t) {
  const int lane = threadIdx.x & 31;
  const float coef = t.coef != nullptr ? *t.coef : 1.0f;
  if (!isfinite(coef)) return;  // the gradient is not finite: this step leaves everything as it is
  const tps_adamw_scalars s = t.dev != nullptr ? *t.dev : t.s;
  int k = 0;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < t.units;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    while (k + 1 < t.count && u >= t.e[k + 1].first) ++k;
    const Entry& e = t.e[k];
    const int64_t unit = u - e.first, at = unit * kUnit;
    const int n = static_cast<int>(e.n - at < kUnit ? e.n - at : kUnit);
    const bool full = e.wide && n == kUnit;
    float g[2][4], w[2][4], m[2][4], v[2][4];
    read8(static_cast<const GT*>(e.g) + at, lane, full, n, g);
    if (MASTER)
      read8(static_cast<const float*>(e.w) + at, lane, full, n, w);
    else
      read8(static_cast<const PT*>(e.p) + at, lane, full, n, w);
    if (E4M3) {
      read8_codes(static_cast<const uint8_t*>(e.m) + at, lane, full, n, e.ms[unit], m);
      read8_codes(static_cast<const uint8_t*>(e.v) + at, lane, full, n, e.vs[unit], v);
    } else {
      read8(static_cast<const float*>(e.m) + at, lane, full, n, m);
      read8(static_cast<const float*>(e.v) + at, lane, full, n, v);
    }
    float root[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float gg = g[j][i] * coef;
        if (E4M3) v[j][i] = __fmul_rn(v[j][i], v[j][i]);
        m[j][i] = __fadd_rn(__fmul_rn(m[j][i], t.b1), __fmul_rn(gg, t.c1));
        v[j][i] = __fadd_rn(__fmul_rn(v[j][i], t.b2), __fmul_rn(__fmul_rn(gg, gg), t.c2));
        root[j][i] = __fsqrt_rn(v[j][i]);
        const float step = __fdiv_rn(__fmul_rn(m[j][i], s.step_size), fmaf(root[j][i], s.root_scale, t.eps));
        w[j][i] = __fsub_rn(__fmul_rn(w[j][i], s.decay), step);
      }
    constexpr bool kRandom = E4M3 || (!MASTER && sizeof(PT) == 2);
    uint32_t rm[2][4], rv[2][4], rp[2][4];
    if (kRandom) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = mix(static_cast<uint64_t>(e.place + at + in_unit(lane, j) + i), s.seed);
          rm[j][i] = t.stochastic ? x & 0xffffu : 0x8000u;
          rv[j][i] = t.stochastic ? x >> 16 : 0x8000u;
          rp[j][i] = t.stochastic ? (x * 0x9e3779b1u) >> 16 : 0x8000u;
        }
    }
    if (sizeof(PT) == 2) {
      __nv_bfloat16 b[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          b[j][i] = MASTER || !t.stochastic ? __float2bfloat16_rn(w[j][i]) : bf16_by(w[j][i], rp[j][i]);
      write8(static_cast<__nv_bfloat16*>(e.p) + at, lane, full, n, b);
      if (MASTER) write8(e.w + at, lane, full, n, w);
    } else {
      write8(static_cast<float*>(e.p) + at, lane, full, n, w);
    }
    if (E4M3) {
      write8_codes<false>(static_cast<uint8_t*>(e.m) + at, e.ms + unit, lane, full, n, m, rm);
      write8_codes<true>(static_cast<uint8_t*>(e.v) + at, e.vs + unit, lane, full, n, root, rv);
    } else {
      write8(static_cast<float*>(e.m) + at, lane, full, n, m);
      write8(static_cast<float*>(e.v) + at, lane, full, n, v);
    }
  }
}

struct Span {
  const void* p;
  int64_t n, first;
  int32_t bf16, wide;
};
template <int N>
struct Spans {
  int32_t count;
  int64_t units;
  Span e[N];
};

constexpr int kNormBlocks = 152 * 8;

// Partial sums of squares, one for each block, of a fixed assignment of units.
template <int N>
__global__ void __launch_bounds__(32 * kWarps) norm_kernel(const __grid_constant__ Spans<N> t, float* part) {
  __shared__ float red[kWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int k = 0;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + w; u < t.units; u += static_cast<int64_t>(gridDim.x) * kWarps) {
    while (k + 1 < t.count && u >= t.e[k + 1].first) ++k;
    const Span& e = t.e[k];
    const int64_t at = (u - e.first) * kUnit;
    const int n = static_cast<int>(e.n - at < kUnit ? e.n - at : kUnit);
    const bool full = e.wide && n == kUnit;
    float x[2][4];
    if (e.bf16)
      read8(static_cast<const __nv_bfloat16*>(e.p) + at, lane, full, n, x);
    else
      read8(static_cast<const float*>(e.p) + at, lane, full, n, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(x[0][i], x[0][i], fmaf(x[1][i], x[1][i], acc[i]));
  }
  float a = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (lane == 0) red[w] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    a = 0.0f;
    for (int i = 0; i < kWarps; ++i) a += red[i];
    part[blockIdx.x] = a;
  }
}

// norm = sqrt of the sum of the partial sums (fp64, fixed order) and the
// coefficient that brings it to max_norm (max_norm <= 0: 1).
__global__ void __launch_bounds__(1024) norm_finish_kernel(const float* part, int n, double max_norm, float* out) {
  __shared__ double red[32];
  double a = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) a += part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x != 0) return;
  a = 0.0;
  for (int i = 0; i < 32; ++i) a += red[i];
  const float norm = static_cast<float>(sqrt(a));
  out[0] = norm;
  float c = 1.0f;
  if (!isfinite(norm))
    c = __int_as_float(0x7fc00000);  // NaN: tps_adamw_step then changes nothing
  else if (max_norm > 0.0)
    c = fminf(1.0f, static_cast<float>(max_norm / (static_cast<double>(norm) + 1e-6)));
  out[1] = c;
}

constexpr int kFew = 32, kMany = 320;  // table sizes: 2.9 KB and 28 KB of kernel parameters

int sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

bool is16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <class PT, class GT, bool MASTER, bool E4M3, int N>
int launch_adamw(const Table<kMany>& all, int64_t elements, int per_element, cudaStream_t s) {
  Table<N> t;
  memcpy(&t, &all, offsetof(Table<kMany>, e));
  memcpy(t.e, all.e, sizeof(Entry) * all.count);
  const int64_t blocks = (t.units + kWarps - 1) / kWarps, most = int64_t(sms()) * 8;
  ProfScope prof("adamw", E4M3 ? "e4m3" : "f32", 0.0, double(elements) * per_element, s);
  adamw_kernel<PT, GT, MASTER, E4M3, N><<<static_cast<unsigned>(blocks < most ? blocks : most), 32 * kWarps, 0, s>>>(t);
  note_launch();
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? TPS_OK : fail(TPS_ERR_CUDA, "adamw: launch failed: %s", cudaGetErrorString(cudaGetLastError()));
}

template <int N>
int launch_norm(const Spans<kMany>& all, float* part, int blocks, cudaStream_t s) {
  Spans<N> t;
  t.count = all.count;
  t.units = all.units;
  memcpy(t.e, all.e, sizeof(Span) * all.count);
  norm_kernel<N><<<blocks, 32 * kWarps, 0, s>>>(t, part);
  note_launch();
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? TPS_OK : fail(TPS_ERR_CUDA, "norm: launch failed: %s", cudaGetErrorString(cudaGetLastError()));
}

template <class PT, class GT, bool MASTER, bool E4M3>
int launch_sized(const Table<kMany>& t, int64_t elements, int per_element, cudaStream_t s) {
  return t.count <= kFew ? launch_adamw<PT, GT, MASTER, E4M3, kFew>(t, elements, per_element, s)
                         : launch_adamw<PT, GT, MASTER, E4M3, kMany>(t, elements, per_element, s);
}

// Kind of a tensor: its types and whether it has a master copy, 0..11.
int launch_kind(int kind, const Table<kMany>& t, int64_t elements, cudaStream_t s) {
  using B = __nv_bfloat16;
  switch (kind) {
    case 0: return launch_sized<float, float, false, false>(t, elements, 28, s);
    case 1: return launch_sized<float, B, false, false>(t, elements, 26, s);
    case 2: return launch_sized<B, float, false, false>(t, elements, 24, s);
    case 3: return launch_sized<B, B, false, false>(t, elements, 22, s);
    case 4: return launch_sized<B, float, true, false>(t, elements, 30, s);
    case 5: return launch_sized<B, B, true, false>(t, elements, 28, s);
    case 6: return launch_sized<float, float, false, true>(t, elements, 16, s);
    case 7: return launch_sized<float, B, false, true>(t, elements, 14, s);
    case 8: return launch_sized<B, float, false, true>(t, elements, 12, s);
    case 9: return launch_sized<B, B, false, true>(t, elements, 10, s);
    case 10: return launch_sized<B, float, true, true>(t, elements, 18, s);
    default: return launch_sized<B, B, true, true>(t, elements, 16, s);
  }
}

int check_hyper(const tps_adamw_hyper* h) {
  if (h == nullptr) return fail(TPS_ERR_ARG, "missing hyperparameters");
  if (!(h->lr >= 0) || !std::isfinite(h->lr) || !(h->weight_decay >= 0) || !std::isfinite(h->weight_decay))
    return fail(TPS_ERR_ARG, "lr and weight_decay must be finite and >= 0");
  if (!(h->beta1 >= 0 && h->beta1 < 1) || !(h->beta2 >= 0 && h->beta2 < 1))
    return fail(TPS_ERR_ARG, "beta1 and beta2 must be in [0, 1)");
  if (!(h->eps >= 0) || !std::isfinite(h->eps)) return fail(TPS_ERR_ARG, "eps must be finite and >= 0");
  if (h->step < 1) return fail(TPS_ERR_ARG, "step counts from 1");
  return TPS_OK;
}

}  // namespace

}  // namespace tps

using namespace tps;

extern "C" int tps_adamw_prepare(const tps_adamw_hyper* h, tps_adamw_scalars* out) {
  clear_detail();
  int rc;
  if ((rc = check_hyper(h))) return rc;
  if (out == nullptr) return fail(TPS_ERR_ARG, "missing output");
  out->step_size = static_cast<float>(h->lr / (1.0 - std::pow(h->beta1, static_cast<double>(h->step))));
  out->root_scale = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(h->beta2, static_cast<double>(h->step))));
  out->decay = static_cast<float>(1.0 - h->lr * h->weight_decay);
  out->seed = h->seed;
  return TPS_OK;
}

extern "C" int tps_adamw_step(const tps_adamw_tensor* tensors, int32_t n, const tps_adamw_hyper* h,
                              const float* grad_scale, const tps_adamw_scalars* device_scalars, void* cuda_stream) {
  clear_detail();
  if (n < 0 || (n > 0 && tensors == nullptr)) return fail(TPS_ERR_ARG, "missing tensors");
  tps_adamw_scalars sc;
  int rc;
  if ((rc = tps_adamw_prepare(h, &sc))) return rc;
  if (reinterpret_cast<uintptr_t>(grad_scale) % 4 != 0 || reinterpret_cast<uintptr_t>(device_scalars) % 16 != 0)
    return fail(TPS_ERR_LAYOUT, "misaligned grad_scale or device_scalars");
  auto kind_of = [](const tps_adamw_tensor& t) {
    const int pg = t.param_dtype == TPS_F32 ? (t.grad_dtype == TPS_BF16) : 2 + (t.grad_dtype == TPS_BF16);
    return (t.state_dtype == TPS_E4M3 ? 6 : 0) + pg + (t.master != nullptr ? 2 : 0);
  };
  unsigned kinds = 0;
  for (int32_t i = 0; i < n; ++i) {  // everything is checked before anything is launched
    const tps_adamw_tensor& t = tensors[i];
    if (t.numel < 0) return fail(TPS_ERR_SHAPE, "tensor %d: negative numel", i);
    const int pd = t.param_dtype, gd = t.grad_dtype, sd = t.state_dtype;
    if ((pd != TPS_F32 && pd != TPS_BF16) || (gd != TPS_F32 && gd != TPS_BF16) || (sd != TPS_F32 && sd != TPS_E4M3))
      return fail(TPS_ERR_DTYPE, "tensor %d: weights and gradients are f32 or bf16, moments f32 or e4m3", i);
    if (t.master != nullptr && pd != TPS_BF16) return fail(TPS_ERR_DTYPE, "tensor %d: a master copy is for bf16 weights", i);
    if (t.numel == 0) continue;
    if (t.param == nullptr || t.grad == nullptr || t.m == nullptr || t.v == nullptr)
      return fail(TPS_ERR_ARG, "tensor %d: missing data", i);
    if ((sd == TPS_E4M3) != (t.m_scale != nullptr) || (sd == TPS_E4M3) != (t.v_scale != nullptr))
      return fail(TPS_ERR_ARG, "tensor %d: scales go with e4m3 moments", i);
    auto off = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
    const uintptr_t se = sd == TPS_F32 ? 4 : 1;
    if (off(t.param, pd == TPS_F32 ? 4 : 2) || off(t.grad, gd == TPS_F32 ? 4 : 2) || off(t.m, se) || off(t.v, se) ||
        off(t.master, 4) || off(t.m_scale, 4) || off(t.v_scale, 4))
      return fail(TPS_ERR_LAYOUT, "tensor %d: misaligned data", i);
    kinds |= 1u << kind_of(t);
  }
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  for (int kind = 0; kind < 12; ++kind) {
    if (!(kinds >> kind & 1u)) continue;
    Table<kMany> tab = {};
    tab.stochastic = h->stochastic != 0;
    tab.coef = grad_scale;
    tab.dev = device_scalars;
    tab.s = sc;
    tab.b1 = static_cast<float>(h->beta1);
    tab.c1 = static_cast<float>(1.0 - h->beta1);
    tab.b2 = static_cast<float>(h->beta2);
    tab.c2 = static_cast<float>(1.0 - h->beta2);
    tab.eps = static_cast<float>(h->eps);
    int64_t elements = 0;
    for (int32_t i = 0; i <= n; ++i) {
      const bool end = i == n;
      if (!end && (tensors[i].numel == 0 || kind_of(tensors[i]) != kind)) continue;
      if ((end || tab.count == kMany) && tab.count > 0) {
        if ((rc = launch_kind(kind, tab, elements, s))) return rc;
        tab.count = 0;
        tab.units = 0;
        elements = 0;
      }
      if (end) break;
      const tps_adamw_tensor& t = tensors[i];
      const bool wide = is16(t.param) && is16(t.grad) && is16(t.m) && is16(t.v) && is16(t.master);
      tab.e[tab.count++] = Entry{t.param, t.grad, t.master, t.m, t.v, t.m_scale, t.v_scale, t.numel, t.place,
                                 tab.units, wide ? 1 : 0};
      tab.units += (t.numel + kUnit - 1) / kUnit;
      elements += t.numel;
    }
  }
  return TPS_OK;
}

extern "C" size_t tps_grad_norm_workspace_bytes(int32_t n) {
  return n < 0 ? 0 : align256(static_cast<size_t>(kNormBlocks) * ((n + kMany - 1) / kMany + 1) * sizeof(float));
}

extern "C" int tps_grad_norm(const tps_span* grads, int32_t n, double max_norm, float* out, void* workspace,
                             size_t workspace_bytes, void* cuda_stream) {
  clear_detail();
  if (n < 0 || (n > 0 && grads == nullptr)) return fail(TPS_ERR_ARG, "missing gradients");
  if (out == nullptr || reinterpret_cast<uintptr_t>(out) % 4 != 0) return fail(TPS_ERR_ARG, "missing or misaligned output");
  if (std::isnan(max_norm)) return fail(TPS_ERR_ARG, "max_norm is not a number");
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
      workspace_bytes < tps_grad_norm_workspace_bytes(n))
    return fail(TPS_ERR_WORKSPACE, "workspace needs %zu bytes, 256-byte aligned", tps_grad_norm_workspace_bytes(n));
  for (int32_t i = 0; i < n; ++i) {
    if (grads[i].numel < 0) return fail(TPS_ERR_SHAPE, "gradient %d: negative numel", i);
    if (grads[i].dtype != TPS_F32 && grads[i].dtype != TPS_BF16)
      return fail(TPS_ERR_DTYPE, "gradient %d must be f32 or bf16", i);
    if (grads[i].numel > 0 && grads[i].data == nullptr) return fail(TPS_ERR_ARG, "gradient %d: missing data", i);
    if (reinterpret_cast<uintptr_t>(grads[i].data) % (grads[i].dtype == TPS_F32 ? 4 : 2) != 0)
      return fail(TPS_ERR_LAYOUT, "gradient %d: misaligned data", i);
  }
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  float* part = static_cast<float*>(workspace);
  Spans<kMany> t = {};
  int parts = 0, rc;
  double bytes = 0.0;
  for (int32_t i = 0; i <= n; ++i) {
    const bool end = i == n;
    if (!end && grads[i].numel == 0) continue;
    if ((end || t.count == kMany) && t.count > 0) {
      const int64_t want = (t.units + kWarps - 1) / kWarps;
      const int blocks = static_cast<int>(want < kNormBlocks ? want : kNormBlocks);
      {
        ProfScope prof("grad_norm", "partial", 0.0, bytes, s);
        rc = t.count <= kFew ? launch_norm<kFew>(t, part + parts, blocks, s) : launch_norm<kMany>(t, part + parts, blocks, s);
      }
      if (rc) return rc;
      parts += blocks;
      t.count = 0;
      t.units = 0;
      bytes = 0.0;
    }
    if (end) break;
    t.e[t.count++] = Span{grads[i].data, grads[i].numel, t.units, grads[i].dtype == TPS_BF16, is16(grads[i].data)};
    t.units += (grads[i].numel + kUnit - 1) / kUnit;
    bytes += double(grads[i].numel) * (grads[i].dtype == TPS_F32 ? 4 : 2);
  }
  norm_finish_kernel<<<1, 1024, 0, s>>>(part, parts, max_norm, out);
  note_launch();
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? TPS_OK : fail(TPS_ERR_CUDA, "norm: launch failed: %s", cudaGetErrorString(cudaGetLastError()));
}
