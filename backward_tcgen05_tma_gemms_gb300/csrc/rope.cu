// rope.cu -- rotary positions of query and key heads.
//
// Pair i of a head's first rotary_dim elements, (a, b), turns by the angle
// p f_i of its position p:
//   forward  (a c - b s, b c + a s),  backward  (a c + b s, b c - a s),
// c and s being amplitude times cosine and sine.  The pairs are (x_i,
// x_{i + r/2}) or, interleaved, (x_{2i}, x_{2i+1}); the rest of the head is
// copied.
//
// Angles without a table: the plan keeps f_i / 2 pi, the turns a position, as a
// 64-bit binary fraction, so p times it modulo 2^64 is the fraction of a turn,
// without a rounding; its upper 32 bits, as a signed number of half turns /
// 2^31, go through sincospif.  The fraction comes from a double and is good to
// 2^-55, which leaves an angle |p| 2^-55 of a turn off (2^-25 at p = 2^30, as
// much as the conversion to a float).
//
// A block takes a few tokens: each thread forms the cosine and sine of one
// (token, pair), which all heads of the token share through shared memory,
// and streams its items -- 16 bytes of either run of a head's pairs -- with
// the loads of the first ones issued before the angles are formed.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "api_common.cuh"

namespace tps {

namespace {

constexpr int kThreads = 256;
constexpr int kTokenPairs = 256;  // (token, pair)s of a block
static_assert(kTokenPairs >= TPS_ROPE_MAX_PAIRS, "one token's pairs fit");

struct View {
  char* p;
  int64_t sb, ss, sh;  // bytes between batches, tokens and heads
};

struct RopeParams {
  View qi, qo, ki, ko;
  int heads_q, heads;      // query heads, query and key heads
  int64_t rows, S;         // tokens, tokens of one batch entry
  int D, rot;              // elements of a head, those that turn
  int units, rot_units;    // thread units of a head, those that turn
  int tokens, block_heads; // of one block
  uint32_t inv_units, inv_units_heads[2];  // 2^32 / units, and / (units heads) of a block and of the last one
  const void* pos;
  int pos_i64, pos_shared; // int64 positions; one row of positions for all batches
  float amp, sign;
};
struct Turns {
  uint64_t t[TPS_ROPE_MAX_PAIRS];
};

template <class T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

// N consecutive elements as one load or store (16 bytes when N > 1).
template <class T, int N>
struct __align__(sizeof(T) * N) Run {
  T v[N];
};

// A block's items are (token, head, unit), unit fastest; item i of a thread
// is threadIdx.x + i * kThreads.
template <class T, int N, bool INTER, bool VEC_TAIL>
__global__ void __launch_bounds__(kThreads, 6) rope_kernel(const __grid_constant__ Turns turns, const RopeParams p) {
  __shared__ __align__(16) float2 cs[kTokenPairs];  // (cosine, sine) of each (token, pair)
  __shared__ int64_t base[4][kTokenPairs];           // byte offsets of each token in q, k and the outputs
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int tokens = static_cast<int>(p.rows - row0 < p.tokens ? p.rows - row0 : p.tokens);
  const int h0 = blockIdx.y * p.block_heads, heads = min(p.block_heads, p.heads - h0);
  const int per_token = heads * p.units, items = tokens * per_token, half = p.rot / 2;
  using R = Run<T, N>;
  for (int i = threadIdx.x; i < tokens; i += kThreads) {
    const int64_t b = (row0 + i) / p.S, t = row0 + i - b * p.S;
    base[0][i] = b * p.qi.sb + t * p.qi.ss;
    base[1][i] = b * p.qo.sb + t * p.qo.ss;
    base[2][i] = b * p.ki.sb + t * p.ki.ss;
    base[3][i] = b * p.ko.sb + t * p.ko.ss;
  }
  __syncthreads();
  struct Item {
    const char* src;
    char* dst;
    int e1;    // second run, relative to the first, in elements
    int at;    // token and unit in `cs` (slot), or -1 outside the turned part
    bool two;  // the second run is there
  };
  // Where pair i of unit u of a token lies in `cs`: two pairs (16 bytes) of
  // neighbouring units side by side, so that a warp reads without conflicts.
  constexpr int kPairRun = N > 1 ? 2 : 1;
  auto slot = [&](int tok, int u, int i) { return tok * half + (i / kPairRun * p.rot_units + u) * kPairRun + i % kPairRun; };
  // Quotients by 32-bit reciprocals: exact while i times the divisor is below 2^32.
  const uint32_t by_token = p.inv_units_heads[blockIdx.y + 1 == gridDim.y], by_units = p.inv_units;
  auto quotient = [](int i, int d, uint32_t inv) { return d == 1 ? i : static_cast<int>(__umulhi(i, inv)); };
  auto item = [&](int i) {
    Item it;
    const int tok = quotient(i, per_token, by_token), in = i - tok * per_token;
    const int hh = quotient(in, p.units, by_units), u = in - hh * p.units, h = h0 + hh;
    int e0;
    if (u >= p.rot_units) {
      e0 = p.rot + (u - p.rot_units) * 2 * N;
      it.e1 = N;
      it.at = -1;
    } else {
      e0 = INTER ? u * 2 * N : u * N;
      it.e1 = INTER ? N : half;
      it.at = slot(tok, u, 0);
    }
    it.two = VEC_TAIL || e0 + it.e1 + N <= p.D;  // a tail may end with a single run
    const bool q = h < p.heads_q;
    const int hr = q ? h : h - p.heads_q, bytes = e0 * static_cast<int>(sizeof(T));
    it.src = (q ? p.qi.p : p.ki.p) + base[q ? 0 : 2][tok] + hr * (q ? p.qi.sh : p.ki.sh) + bytes;
    it.dst = (q ? p.qo.p : p.ko.p) + base[q ? 1 : 3][tok] + hr * (q ? p.qo.sh : p.ko.sh) + bytes;
    return it;
  };
  // One item in flight a thread and six blocks an SM: 8192 tokens of 40 heads
  // of 128 in 32.8 us (5.1 TB/s); two to five items in flight at the registers
  // they take, 37 to 51 us.
  R x, y;
  Item it;
  auto load = [&](int i) {
    it = item(i);
    x = *reinterpret_cast<const R*>(it.src);
    if (it.two) y = *reinterpret_cast<const R*>(it.src + it.e1 * int(sizeof(T)));
  };
  if (static_cast<int>(threadIdx.x) < items) load(threadIdx.x);
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const int tok = i / half;
    const int64_t row = row0 + tok, at_pos = p.pos_shared ? row % p.S : row;
    const int64_t pos = p.pos_i64 ? static_cast<const int64_t*>(p.pos)[at_pos]
                                  : static_cast<int64_t>(static_cast<const int32_t*>(p.pos)[at_pos]);
    const uint64_t f = static_cast<uint64_t>(pos) * turns.t[i - tok * half];
    float c, n;
    sincospif(static_cast<float>(static_cast<int32_t>(f >> 32)) * 0x1p-31f, &n, &c);
    const int pair = i - tok * half;
    cs[slot(tok, pair / N, pair % N)] = make_float2(c * p.amp, n * p.amp * p.sign);
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < items; i0 += kThreads) {
    if (i0 != static_cast<int>(threadIdx.x)) load(i0);
    if (it.at >= 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 t = cs[it.at + i / kPairRun * p.rot_units * kPairRun + i % kPairRun];
        // the unit's 2 N elements: pair i is (x_i, y_i), or elements 2i and 2i+1 of x followed by y
        T& ra = INTER ? (2 * i < N ? x.v[2 * i < N ? 2 * i : 0] : y.v[2 * i < N ? 0 : 2 * i - N]) : x.v[i];
        T& rb = INTER ? (2 * i + 1 < N ? x.v[2 * i + 1 < N ? 2 * i + 1 : 0] : y.v[2 * i + 1 < N ? 0 : 2 * i + 1 - N])
                      : y.v[i];
        const float a = to_f(ra), d = to_f(rb);
        ra = from_f<T>(fmaf(a, t.x, -d * t.y));
        rb = from_f<T>(fmaf(d, t.x, a * t.y));
      }
    }
    *reinterpret_cast<R*>(it.dst) = x;
    if (it.two) *reinterpret_cast<R*>(it.dst + it.e1 * int(sizeof(T))) = y;
  }
}

// A (B, S, H, D) or (T, H, D) view with unit stride along D.
int heads_view(const tps_tensor* t, const char* name, View* v, int64_t* B, int64_t* S, int64_t* H, int64_t* D,
               int* dtype) {
  if (t == nullptr) return fail(TPS_ERR_ARG, "%s: missing tensor", name);
  if (t->ndim != 3 && t->ndim != 4) return fail(TPS_ERR_SHAPE, "%s: expected (T, H, D) or (B, S, H, D)", name);
  if (t->dtype != TPS_F32 && t->dtype != TPS_BF16) return fail(TPS_ERR_DTYPE, "%s must be f32 or bf16", name);
  const int o = t->ndim - 3;
  int64_t n = 1;
  for (int i = 0; i < t->ndim; ++i) {
    if (t->shape[i] < 0) return fail(TPS_ERR_SHAPE, "%s: negative extent", name);
    n *= t->shape[i];
  }
  if (t->data == nullptr && n > 0) return fail(TPS_ERR_ARG, "%s: missing data", name);
  const int64_t es = t->dtype == TPS_F32 ? 4 : 2;
  if (t->shape[o + 2] > 1 && t->stride[o + 2] != 1) return fail(TPS_ERR_LAYOUT, "%s: heads must be contiguous", name);
  if (reinterpret_cast<uintptr_t>(t->data) % es != 0) return fail(TPS_ERR_LAYOUT, "%s: misaligned data", name);
  *B = o ? t->shape[0] : 1;
  *S = t->shape[o];
  *H = t->shape[o + 1];
  *D = t->shape[o + 2];
  *dtype = t->dtype;
  v->p = static_cast<char*>(t->data);
  v->sb = o ? t->stride[0] * es : 0;
  v->ss = t->stride[o] * es;
  v->sh = t->stride[o + 1] * es;
  return TPS_OK;
}

bool aligned16(const View& v) {
  return (reinterpret_cast<uintptr_t>(v.p) | static_cast<uintptr_t>(v.sb) | static_cast<uintptr_t>(v.ss) |
          static_cast<uintptr_t>(v.sh)) % 16 == 0;
}

template <class T, int N, bool VEC_TAIL>
void launch_rope(const Turns& t, const RopeParams& p, bool inter, dim3 grid, cudaStream_t s) {
  if (inter)
    rope_kernel<T, N, true, VEC_TAIL><<<grid, kThreads, 0, s>>>(t, p);
  else
    rope_kernel<T, N, false, VEC_TAIL><<<grid, kThreads, 0, s>>>(t, p);
}

int rope(const tps_rope_plan* plan, const tps_tensor* Q, const tps_tensor* K, const tps_tensor* positions,
         const tps_tensor* Qo, const tps_tensor* Ko, float sign, void* cuda_stream) {
  clear_detail();
  if (plan == nullptr) return fail(TPS_ERR_ARG, "missing plan");
  if (plan->rotary_dim < 2 || plan->rotary_dim % 2 != 0 || plan->rotary_dim / 2 > TPS_ROPE_MAX_PAIRS)
    return fail(TPS_ERR_ARG, "the plan is not one that tps_rope_plan_init made");
  RopeParams p = {};
  int64_t B, S, H, D, b2, s2, h2, d2;
  int dt, dt2, rc;
  if ((rc = heads_view(Q, "Q", &p.qi, &B, &S, &H, &D, &dt))) return rc;
  if ((rc = heads_view(Qo, "Q out", &p.qo, &b2, &s2, &h2, &d2, &dt2))) return rc;
  if (b2 != B || s2 != S || h2 != H || d2 != D) return fail(TPS_ERR_SHAPE, "Q out: another shape than Q");
  if (dt2 != dt) return fail(TPS_ERR_DTYPE, "Q out: another type than Q");
  int64_t Hk = 0;
  if ((K == nullptr) != (Ko == nullptr)) return fail(TPS_ERR_ARG, "K and K out go together");
  if (K != nullptr) {
    if ((rc = heads_view(K, "K", &p.ki, &b2, &s2, &Hk, &d2, &dt2))) return rc;
    if (b2 != B || s2 != S || d2 != D) return fail(TPS_ERR_SHAPE, "K: other tokens or head width than Q");
    if (dt2 != dt) return fail(TPS_ERR_DTYPE, "K: another type than Q");
    if ((rc = heads_view(Ko, "K out", &p.ko, &b2, &s2, &h2, &d2, &dt2))) return rc;
    if (b2 != B || s2 != S || h2 != Hk || d2 != D) return fail(TPS_ERR_SHAPE, "K out: another shape than K");
    if (dt2 != dt) return fail(TPS_ERR_DTYPE, "K out: another type than K");
  }
  if (D < plan->rotary_dim) return fail(TPS_ERR_SHAPE, "heads of %lld elements turn %d", (long long)D, plan->rotary_dim);
  if (D > (1 << 20) || H + Hk > (1 << 20)) return fail(TPS_ERR_SHAPE, "too many heads, or too wide");
  if (positions == nullptr) return fail(TPS_ERR_ARG, "positions missing");
  if (positions->dtype != TPS_I32 && positions->dtype != TPS_I64)
    return fail(TPS_ERR_DTYPE, "positions must be i32 or i64");
  int64_t np = 1;
  for (int i = 0; i < positions->ndim && i < 4; ++i) np *= positions->shape[i];
  p.pos_shared = np != B * S && np == S;
  if ((rc = expect_vector(positions, "positions", positions->dtype, p.pos_shared ? S : B * S))) return rc;
  p.rows = B * S;
  p.S = S;
  p.heads_q = static_cast<int>(H);
  p.heads = static_cast<int>(H + Hk);
  if (p.rows == 0 || p.heads == 0) return TPS_OK;
  p.D = static_cast<int>(D);
  p.rot = plan->rotary_dim;
  p.pos = positions->data;
  p.pos_i64 = positions->dtype == TPS_I64;
  p.amp = plan->amplitude;
  p.sign = sign;
  // 16-byte runs where every row of every head starts on one and both the
  // pairs and the rest are whole runs; else one pair a thread.
  const int es = dt == TPS_F32 ? 4 : 2, wide = 16 / es;
  const bool vec = p.rot % (2 * wide) == 0 && p.D % wide == 0 && aligned16(p.qi) && aligned16(p.qo) &&
                   (K == nullptr || (aligned16(p.ki) && aligned16(p.ko)));
  const int N = vec ? wide : 1;
  auto same = [](const View& a, const View& b) { return a.p == b.p && a.sb == b.sb && a.ss == b.ss && a.sh == b.sh; };
  const bool in_place = same(p.qi, p.qo) && (K == nullptr || same(p.ki, p.ko));
  const int tail = in_place ? 0 : p.D - p.rot;  // in place the rest of the head is there already
  p.rot_units = p.rot / (2 * N);
  p.units = p.rot_units + (tail + 2 * N - 1) / (2 * N);
  const bool vec_tail = tail % (2 * N) == 0;
  // Tokens of one block: as many as leave every SM eight blocks, up to what
  // `cs` holds; with few tokens, their heads are spread over blocks as well,
  // down to one round of items each.
  const int64_t sms = 152;
  p.tokens = kTokenPairs / (p.rot / 2);
  while (p.tokens > 1 && (p.rows + p.tokens - 1) / p.tokens < 8 * sms) p.tokens /= 2;
  const int64_t blocks = (p.rows + p.tokens - 1) / p.tokens;
  p.block_heads = p.heads;
  while (p.block_heads > 1 && blocks * ((p.heads + p.block_heads - 1) / p.block_heads) < 2 * sms &&
         int64_t(p.tokens) * p.block_heads * p.units > kThreads)
    p.block_heads = (p.block_heads + 1) / 2;
  while (p.block_heads > 1 && int64_t(p.tokens) * p.block_heads * p.units > 32768) p.block_heads = (p.block_heads + 1) / 2;
  const int64_t groups = (p.heads + p.block_heads - 1) / p.block_heads;
  const int64_t items = int64_t(p.tokens) * p.block_heads * p.units, last_heads = p.heads - (groups - 1) * p.block_heads;
  auto inverse = [](int64_t d) { return static_cast<uint32_t>(((int64_t(1) << 32) + d - 1) / d); };
  p.inv_units = inverse(p.units);
  p.inv_units_heads[0] = inverse(int64_t(p.units) * p.block_heads);
  p.inv_units_heads[1] = inverse(int64_t(p.units) * last_heads);
  if (blocks > 0x7fffffff || groups > 65535 || items * p.units * p.block_heads >= (int64_t(1) << 32))
    return fail(TPS_ERR_SHAPE, "too many tokens or heads for one launch");
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(groups));
  Turns t;
  memcpy(t.t, plan->turns, sizeof(t.t));
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  {
    ProfScope prof("rope", sign > 0 ? "fwd" : "bwd", 0.0, 2.0 * es * double(p.rows) * p.heads * p.D, s);
    const bool inter = plan->interleaved != 0;
    if (dt == TPS_BF16) {
      if (!vec) launch_rope<__nv_bfloat16, 1, false>(t, p, inter, grid, s);
      else if (vec_tail) launch_rope<__nv_bfloat16, 8, true>(t, p, inter, grid, s);
      else launch_rope<__nv_bfloat16, 8, false>(t, p, inter, grid, s);
    } else {
      if (!vec) launch_rope<float, 1, false>(t, p, inter, grid, s);
      else if (vec_tail) launch_rope<float, 4, true>(t, p, inter, grid, s);
      else launch_rope<float, 4, false>(t, p, inter, grid, s);
    }
  }
  note_launch();
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? TPS_OK : fail(TPS_ERR_CUDA, "rope: launch failed: %s", cudaGetErrorString(cudaGetLastError()));
}

}  // namespace

}  // namespace tps

using namespace tps;

extern "C" int tps_rope_plan_init(const tps_rope_options* o, tps_rope_plan* plan) {
  clear_detail();
  if (o == nullptr || plan == nullptr) return fail(TPS_ERR_ARG, "missing options or plan");
  if (o->rotary_dim < 2 || o->rotary_dim % 2 != 0 || o->rotary_dim / 2 > TPS_ROPE_MAX_PAIRS)
    return fail(TPS_ERR_SHAPE, "rotary_dim %d: even, 2 to %d", o->rotary_dim, 2 * TPS_ROPE_MAX_PAIRS);
  if (o->reserved != 0) return fail(TPS_ERR_ARG, "reserved must be 0");
  if (!(o->base > 1.0) || !std::isfinite(o->base)) return fail(TPS_ERR_ARG, "base must be finite and above 1");
  if (o->scaling < TPS_ROPE_NONE || o->scaling > TPS_ROPE_YARN) return fail(TPS_ERR_ARG, "unknown scaling %d", o->scaling);
  const double r = o->rotary_dim, factor = o->scaling == TPS_ROPE_NONE ? 1.0 : o->factor;
  if (!(factor >= 1.0) || !std::isfinite(factor)) return fail(TPS_ERR_ARG, "factor must be finite and at least 1");
  const double two_pi = 6.283185307179586476925286766559;
  double base = o->base, lo = 0.0, hi = 0.0;
  if (o->scaling == TPS_ROPE_NTK) {
    if (o->rotary_dim < 4) return fail(TPS_ERR_SHAPE, "this scaling needs a rotary_dim of 4 or more");
    base *= std::pow(factor, r / (r - 2.0));
    if (!std::isfinite(base)) return fail(TPS_ERR_ARG, "base times the factor's power is not finite");
  }
  if (std::isinf(o->attention_factor) || std::isnan(o->attention_factor))
    return fail(TPS_ERR_ARG, "attention_factor must be finite");
  if (o->scaling == TPS_ROPE_YARN) {
    const double fast = o->beta_fast > 0 ? o->beta_fast : 32.0, slow = o->beta_slow > 0 ? o->beta_slow : 1.0;
    if (!(o->original_context > 0) || !std::isfinite(o->original_context) || !(fast >= slow) || !std::isfinite(fast))
      return fail(TPS_ERR_ARG, "original_context must be finite and positive, beta_fast at least beta_slow");
    // the pair index whose frequency makes `turns` turns within the original context
    auto at = [&](double turns) { return r * std::log(o->original_context / (turns * two_pi)) / (2.0 * std::log(base)); };
    lo = std::fmax(std::floor(at(fast)), 0.0);
    hi = std::fmin(std::ceil(at(slow)), r - 1.0);
  }
  memset(plan, 0, sizeof(*plan));
  plan->rotary_dim = o->rotary_dim;
  plan->interleaved = o->interleaved != 0;
  plan->amplitude = static_cast<float>(o->attention_factor > 0 ? o->attention_factor
                                       : o->scaling == TPS_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0);
  for (int i = 0; i < o->rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (o->scaling == TPS_ROPE_LINEAR) f /= factor;
    if (o->scaling == TPS_ROPE_YARN) {
      const double ramp = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 1e-3)));
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    plan->turns[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64));  // f <= 1: under 0.16 of a turn
  }
  return TPS_OK;
}

extern "C" int tps_rope_fwd(const tps_rope_plan* plan, const tps_tensor* Q, const tps_tensor* K,
                            const tps_tensor* positions, const tps_tensor* Qo, const tps_tensor* Ko, void* cuda_stream) {
  return rope(plan, Q, K, positions, Qo, Ko, 1.0f, cuda_stream);
}

extern "C" int tps_rope_bwd(const tps_rope_plan* plan, const tps_tensor* dQo, const tps_tensor* dKo,
                            const tps_tensor* positions, const tps_tensor* dQ, const tps_tensor* dK, void* cuda_stream) {
  return rope(plan, dQo, dKo, positions, dQ, dK, -1.0f, cuda_stream);
}
