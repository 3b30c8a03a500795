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
// With fp32 moments the root and the quotient of the step are the hardware's
// approximations, to two units each; the state holds neither.  With e4m3
// moments the root is state, and correctly rounded.
//
// 218 M weights: fp32 moments with a master copy 0.92 ms (6.6 TB/s, memory),
// e4m3 moments 0.51 ms (4.3 TB/s; 80 instructions a weight bound it, about
// fourteen of them for the random bits); the norm reads bf16 gradients at
// 5.6 TB/s one call behind the other, 4.8 TB/s after other work.
//
// One warp takes 256 elements (a block of the 8-bit form),
// 2 x 4 a lane, so every load of a warp is consecutive, and the block's
// maxima are two warp reductions.  The tensors' table travels in the kernel
// parameters: no copy, no workspace, nothing to keep alive.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <type_traits>

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
  int32_t chunk;             // consecutive units of a warp
  uint32_t random, nearest;  // of 32 random bits: those kept, and those set (two halves) to round to nearest
  int64_t units;
  const float* coef;
  const tps_adamw_scalars* dev;  // read instead of `s` when given
  tps_adamw_scalars s;
  float b1, c1, b2, c2, eps;  // beta, 1 - beta
  float minus_zero;
  Entry e[N];
};

constexpr uint32_t kPlaceMul = 0x9e3779b1u;
// 32 random bits of a place: `x` is place * kPlaceMul plus its upper half's
// share.  seed2 = seed ^ seed >> 16: what x ^= seed leaves after the first
// shift, folded into one operation.
__device__ __forceinline__ uint32_t mix(uint32_t x, uint32_t seed2) {
  x = (x ^ (x >> 16) ^ seed2) * 0x2c1b3c6du;
  x = (x ^ (x >> 12)) * 0x297a2d39u;
  return x ^ (x >> 15);
}
// fp32 (not a NaN) to the bf16 below or above by 16 random bits, in the upper
// half; infinity has no bits to carry from.
__device__ __forceinline__ uint32_t bf16_by(float x, uint32_t rnd) { return __float_as_uint(x) + rnd; }
// The e4m3 code below or above |x| 448 / a by 16 random bits, in the low
// byte; s = 448 / a * 2^-120.  That product has the code's exponent in a
// float's exponent field and its mantissa on top of the float's, and e4m3
// subnormals are float subnormals there, so that one addition and one shift
// do it for all of them.  (The product may pass 448 by its rounding; 16 units
// of that stay below the last random bit.)
__device__ __forceinline__ uint32_t e4m3_by(float x, float s, uint32_t rnd) {
  return (rnd * 16u + __float_as_uint(fabsf(x) * s)) >> 20;
}
// And back: the code's bits in place of a float's are the number times 2^-120;
// s = scale * 2^120.
__device__ __forceinline__ float e4m3_float(uint32_t bits, float s) { return __uint_as_float(bits) * s; }
// Blocks whose scale times 2^120 may overflow are read 2^-120 smaller: a code's
// bits times the scale itself, which for a scale above 64 is a normal number,
// then times 2^120.  Blocks whose 448 / a 2^-120 would lose bits are brought
// down by 2^-40, up to three times, before they are written.  Both are exact,
// and a whole warp agrees on them.
constexpr float kSmaller = 0x1p-40f, kLarger = 0x1p120f, kLargeScale = 64.0f;
// Bits of code i of four: exponent and mantissa from bit 26 down, and the sign
// in bit 31.  (Shifts to the left are products here: they run beside the
// logical operations, which this kernel has most of.)
__device__ __forceinline__ uint32_t unsigned_code(uint32_t q, int i) {
  return (i < 3 ? q * (1u << (20 - 8 * (i < 3 ? i : 0))) : q >> 4) & 0x07f00000u;
}
__device__ __forceinline__ uint32_t signed_code(uint32_t q, int i) {
  return ((q * (1u << (24 - 8 * i))) & 0x80000000u) | unsigned_code(q, i);
}

// The index of a lane's first element of group j (0, 1) of four within a unit.
__device__ __forceinline__ int in_unit(int lane, int j) { return j * 128 + lane * 4; }

// Four consecutive elements as they come from memory.
template <class T> struct Four { uint2 q; };
template <> struct Four<float> { float4 q; };
__device__ __forceinline__ void unpack(const Four<float>& f, float (&x)[4]) {
  x[0] = f.q.x; x[1] = f.q.y; x[2] = f.q.z; x[3] = f.q.w;
}
__device__ __forceinline__ void unpack(const Four<__nv_bfloat16>& f, float (&x)[4]) {
  x[0] = __uint_as_float(f.q.x << 16); x[1] = __uint_as_float(f.q.x & 0xffff0000u);
  x[2] = __uint_as_float(f.q.y << 16); x[3] = __uint_as_float(f.q.y & 0xffff0000u);
}
// FULL, here and below: all 256 elements of the unit are there and every
// pointer is aligned; else `n` of them are, and they go one by one.
template <bool FULL, class T>
__device__ __forceinline__ void fetch(const T* p, int lane, int n, Four<T> (&f)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = in_unit(lane, j);
    if (FULL) {
      f[j].q = *reinterpret_cast<const decltype(f[j].q)*>(p + at);
    } else {
      T x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = T(0.0f);
        if (at + i < n) x[i] = p[at + i];
      }
      memcpy(&f[j], x, sizeof(x));
    }
  }
}
template <bool FULL>
__device__ __forceinline__ void fetch_codes(const uint8_t* p, int lane, int n, uint32_t (&q)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = in_unit(lane, j);
    q[j] = 0;
    if (FULL) {
      q[j] = *reinterpret_cast<const uint32_t*>(p + at);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i < n) q[j] |= static_cast<uint32_t>(p[at + i]) << (8 * i);
    }
  }
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
// bf16 values in the upper halves of words.
__device__ __forceinline__ void store4(__nv_bfloat16* p, const uint32_t (&x)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(__byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, uint32_t x) {
  *p = __ushort_as_bfloat16(static_cast<unsigned short>(x >> 16));
}
template <bool FULL, class T, class V>
__device__ __forceinline__ void write8(T* p, int lane, int n, const V (&x)[2][4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = in_unit(lane, j);
    if (FULL) {
      store4(p + at, x[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i < n) store1(p + at + i, x[j][i]);
    }
  }
}
// The largest magnitude of the warp's block, 0 where it is next to nothing.
__device__ __forceinline__ float block_top(const float (&x)[2][4]) {
  float part = 0.0f;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; i += 2) part = max_nan(part, fabsf(x[j][i]), fabsf(x[j][i + 1]));
  const float a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(part)));  // a NaN has the largest bits
  return a < 1e-30f ? 0.0f : a;
}
// x with its block's largest magnitude a brought to where 448 / a keeps all its bits.
__device__ __forceinline__ float bring_down(float a, float (&x)[2][4]) {
  for (int k = 0; k < 3 && a > kLargeScale * 256.0f; ++k) {
    a *= kSmaller;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] *= kSmaller;
  }
  return a;
}
// x as e4m3 numbers, inv = 448 (1 / a) 2^-120.  SQRT: x >= 0 and nothing but 0 becomes 0.
template <bool FULL, bool SQRT>
__device__ __forceinline__ void write8_codes(uint8_t* p, float inv, int lane, int n, const float (&x)[2][4],
                                             const uint32_t (&rnd)[2][4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3_by(x[j][i], inv, rnd[j][i]);
    uint32_t q = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    if (SQRT) {
      if ((q - 0x01010101u) & ~q & 0x80808080u) {  // a code is 0 (this test may name too many): is its element?
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((q >> (8 * i) & 0xffu) == 0 && x[j][i] > 0.0f) q |= 1u << (8 * i);
      }
    } else {  // the signs; a zero may keep its own
      const uint32_t s01 = __byte_perm(__float_as_uint(x[j][0]), __float_as_uint(x[j][1]), 0x0073);
      const uint32_t s23 = __byte_perm(__float_as_uint(x[j][2]), __float_as_uint(x[j][3]), 0x0073);
      q |= __byte_perm(s01, s23, 0x5410) & 0x80808080u;
    }
    const int at = in_unit(lane, j);
    if (FULL) {
      *reinterpret_cast<uint32_t*>(p + at) = q;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i < n) p[at + i] = static_cast<uint8_t>(q >> (8 * i));
    }
  }
}

// Smallest of three.
__device__ __forceinline__ float min_of(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Pairs of fp32 operations as one instruction, each rounded on its own.
__device__ __forceinline__ uint64_t two(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void both(uint64_t x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Square roots of a pair that go into the state, correctly rounded (so the
// codes are those of the rounded root): Markstein's correction, P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990 -- with y near 1 / sqrt(x), r = x y is off by little and
// r + (x - r^2) y / 2 by that squared before its one rounding.  For x of at
// least kRootLeast, where x - r^2, some 2^-22 x, is a normal number; smaller
// ones and zeros (whose y would be infinite) are for small_roots.
constexpr float kRootLeast = 0x1p-100f;
__device__ __forceinline__ uint64_t root2(uint64_t x) {
  float a, b;
  both(x, a, b);
  asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(b));
  const uint64_t y = two(a, b), r = mul2(x, y);
  return fma2(fma2(mul2(r, two(-1.0f, -1.0f)), r, x), mul2(y, two(0.5f, 0.5f)), r);
}
// root2's results r of x, in place, where a lane has an x below kRootLeast.
__device__ __forceinline__ void small_roots(const uint64_t (&x)[2][2], uint64_t (&r)[2][2]) {
  float v[8], least;
#pragma unroll
  for (int i = 0; i < 4; ++i) both(x[i / 2][i % 2], v[2 * i], v[2 * i + 1]);
  least = fminf(v[0], v[1]);
#pragma unroll
  for (int i = 2; i < 8; i += 2) least = min_of(least, v[i], v[i + 1]);
  if (!(least < kRootLeast)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    both(r[i / 2][i % 2], a, b);
    r[i / 2][i % 2] = two(v[2 * i] < kRootLeast ? __fsqrt_rn(v[2 * i]) : a,
                          v[2 * i + 1] < kRootLeast ? __fsqrt_rn(v[2 * i + 1]) : b);
  }
}
__device__ __forceinline__ float rcp_of(float x) {  // to one unit; subnormals count as 0
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Square root to two units, for a step only.
__device__ __forceinline__ float root_of(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The entry of unit u: the last that starts at or before it.
template <class E>
__device__ __forceinline__ int entry_of(const E* e, int count, int64_t u) {
  int lo = 0;
  for (int hi = count; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (u >= e[mid].first) lo = mid; else hi = mid;
  }
  return lo;
}

// What a lane reads of a unit, so that the next unit's loads can be in
// flight while this one is computed.
template <class GT, class WT, bool E4M3>
struct Raw {
  Four<GT> g[2];
  Four<WT> w[2];
  Four<float> m[2], v[2];  // fp32 moments
  uint32_t qm[2], qv[2];   // e4m3 moments and their scales
  float ms, vs;
};

template <bool FULL, class WT, class GT, bool MASTER, bool E4M3>
__device__ __forceinline__ void adamw_fetch(const Entry& e, int64_t unit, int n, int lane, Raw<GT, WT, E4M3>& r) {
  const int64_t at = unit * kUnit;
  fetch<FULL>(static_cast<const GT*>(e.g) + at, lane, n, r.g);
  fetch<FULL>((MASTER ? reinterpret_cast<const WT*>(e.w) : static_cast<const WT*>(e.p)) + at, lane, n, r.w);
  if (E4M3) {
    fetch_codes<FULL>(static_cast<const uint8_t*>(e.m) + at, lane, n, r.qm);
    fetch_codes<FULL>(static_cast<const uint8_t*>(e.v) + at, lane, n, r.qv);
    r.ms = e.ms[unit];
    r.vs = e.vs[unit];
  } else {
    fetch<FULL>(static_cast<const float*>(e.m) + at, lane, n, r.m);
    fetch<FULL>(static_cast<const float*>(e.v) + at, lane, n, r.v);
  }
}

template <bool FULL, class PT, class WT, class GT, bool MASTER, bool E4M3, int N>
__device__ __forceinline__ void adamw_unit(const Table<N>& t, const Entry& e, int64_t unit, int n, float coef,
                                           const tps_adamw_scalars& s, int lane, const Raw<GT, WT, E4M3>& r) {
  const int64_t at = unit * kUnit;
  float g[2][4], w[2][4], m[2][4], v[2][4], root[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    unpack(r.g[j], g[j]);
    unpack(r.w[j], w[j]);
    if (!E4M3) {
      unpack(r.m[j], m[j]);
      unpack(r.v[j], v[j]);
    }
  }
  if (E4M3) {
    const bool bm = r.ms > kLargeScale, bv = r.vs > kLargeScale;
    const float sm = bm ? r.ms : r.ms * 0x1p120f;
    const float sv = bv ? r.vs : r.vs * 0x1p120f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[j][i] = e4m3_float(signed_code(r.qm[j], i), sm);
        root[j][i] = e4m3_float(unsigned_code(r.qv[j], i), sv);
      }
    if (bm || bv) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (bm) m[j][i] *= kLarger;
          if (bv) root[j][i] *= kLarger;
        }
    }
  }
  if (E4M3) {
    // One rounding an operation, as any elementary implementation has it: a
    // last bit that differs here can move a code by a whole step.
    const uint64_t b1 = two(t.b1, t.b1), c1 = two(t.c1, t.c1), b2 = two(t.b2, t.b2), c2 = two(t.c2, t.c2);
    const uint64_t cc = two(coef, coef), ss = two(s.step_size, s.step_size), rs = two(s.root_scale, s.root_scale);
    // products that go into a sum are fma's with a -0 the compiler cannot see:
    // it would fuse a packed product and sum into one rounding
    const uint64_t zero = two(t.minus_zero, t.minus_zero);
    const uint64_t eps = two(t.eps, t.eps), dc = two(s.decay, s.decay), minus = two(-1.0f, -1.0f);
    uint64_t mm[2][2], vv[2][2], rr[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = 2 * k;
        const uint64_t gg = mul2(two(g[j][i], g[j][i + 1]), cc), r0 = two(root[j][i], root[j][i + 1]);
        mm[j][k] = add2(fma2(two(m[j][i], m[j][i + 1]), b1, zero), fma2(gg, c1, zero));
        vv[j][k] = add2(fma2(mul2(r0, r0), b2, zero), fma2(mul2(gg, gg), c2, zero));
        rr[j][k] = root2(vv[j][k]);
      }
    small_roots(vv, rr);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = 2 * k;
        float d0, d1;
        both(fma2(rr[j][k], rs, eps), d0, d1);
        const uint64_t step = mul2(mul2(mm[j][k], ss), two(rcp_of(d0), rcp_of(d1)));
        both(fma2(step, minus, mul2(two(w[j][i], w[j][i + 1]), dc)), w[j][i], w[j][i + 1]);
        both(mm[j][k], m[j][i], m[j][i + 1]);
        both(rr[j][k], root[j][i], root[j][i + 1]);
      }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float gg = g[j][i] * coef;
        m[j][i] = fmaf(m[j][i], t.b1, gg * t.c1);
        v[j][i] = fmaf(v[j][i], t.b2, gg * gg * t.c2);
        const float step = __fdividef(m[j][i] * s.step_size, fmaf(root_of(v[j][i]), s.root_scale, t.eps));
        w[j][i] = fmaf(w[j][i], s.decay, -step);
      }
  }
  constexpr bool kRandom = E4M3 || (!MASTER && sizeof(PT) == 2);
  uint32_t rm[2][4], rv[2][4], rp[2][4];
  if (kRandom) {
    // places of a unit share their upper half: both they and units start on multiples of 256
    const uint64_t place = static_cast<uint64_t>(e.place + at);
    const uint32_t seed2 = s.seed ^ s.seed >> 16;
    const uint32_t base = (static_cast<uint32_t>(place) + 4 * lane) * kPlaceMul + static_cast<uint32_t>(place >> 32) * 0x85ebca77u;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x = mix(base + static_cast<uint32_t>(128 * j + i) * kPlaceMul, seed2);
        rp[j][i] = (x * kPlaceMul) >> 16;
        x = (x & t.random) | t.nearest;
        rm[j][i] = x & 0xffffu;
        rv[j][i] = x >> 16;
      }
  }
  if (sizeof(PT) == 2) {
    uint32_t b[2][4];
    float probe = 0.0f;  // NaN if a weight is not finite
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) probe = fmaf(w[j][i], 0.0f, probe);
    if (MASTER || __any_sync(0xffffffffu, t.nearest || probe != 0.0f)) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t rn = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(w[j][i]))) << 16;
          b[j][i] = MASTER || t.nearest || probe != 0.0f ? rn : bf16_by(w[j][i], rp[j][i]);
        }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) b[j][i] = bf16_by(w[j][i], rp[j][i]);
    }
    write8<FULL>(static_cast<__nv_bfloat16*>(e.p) + at, lane, n, b);
    if (MASTER) write8<FULL>(e.w + at, lane, n, w);
  } else {
    write8<FULL>(static_cast<float*>(e.p) + at, lane, n, w);
  }
  if (E4M3) {
    // even lanes form the reciprocal for m, odd ones for sqrt(v)
    float am = block_top(m), av = block_top(root);
    if (lane < 2) (lane ? e.vs : e.ms)[unit] = __fmul_rn(lane ? av : am, 1.0f / 448.0f);
    am = bring_down(am, m);
    av = bring_down(av, root);
    const float a = (lane & 1) ? av : am;
    const float inv = (a > 0.0f ? __fmul_rn(__frcp_rn(a), 448.0f) : a) * 0x1p-120f;
    write8_codes<FULL, false>(static_cast<uint8_t*>(e.m) + at, __shfl_sync(0xffffffffu, inv, 0), lane, n, m, rm);
    write8_codes<FULL, true>(static_cast<uint8_t*>(e.v) + at, __shfl_sync(0xffffffffu, inv, 1), lane, n, root, rv);
  } else {
    write8<FULL>(static_cast<float*>(e.m) + at, lane, n, m);
    write8<FULL>(static_cast<float*>(e.v) + at, lane, n, v);
  }
}

template <class PT, class GT, bool MASTER, bool E4M3, int N>
__global__ void __launch_bounds__(32 * kWarps, E4M3 ? 3 : 4) adamw_kernel(const __grid_constant__ Table<N> t) {
  using WT = typename std::conditional<MASTER, float, PT>::type;
  const int lane = threadIdx.x & 31;
  const float coef = t.coef != nullptr ? *t.coef : 1.0f;
  if (!isfinite(coef)) return;  // the gradient is not finite: this step leaves everything as it is
  const tps_adamw_scalars s = t.dev != nullptr ? *t.dev : t.s;
  // Consecutive units of one tensor share its pointers: the table is read and
  // the addresses are formed once for `chunk` of them.
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * t.chunk;
  int64_t u = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * t.chunk;
  int k = entry_of(t.e, t.count, u);
  for (; u < t.units; u += step) {
    const int64_t end = u + t.chunk < t.units ? u + t.chunk : t.units;
    for (int64_t at = u; at < end;) {
      while (k + 1 < t.count && at >= t.e[k + 1].first) ++k;
      const Entry& e = t.e[k];
      int64_t unit = at - e.first;
      const int64_t whole = e.wide ? e.n / kUnit : 0;
      const int64_t stop = end - e.first < whole ? end - e.first : whole;
      if (unit < stop) {
        at += stop - unit;
        Raw<GT, WT, E4M3> now, next;
        if (E4M3) adamw_fetch<true, WT, GT, MASTER, E4M3>(e, unit, kUnit, lane, now);
        for (; unit < stop; ++unit) {
          if (!E4M3)
            adamw_fetch<true, WT, GT, MASTER, E4M3>(e, unit, kUnit, lane, now);
          else if (unit + 1 < stop)
            adamw_fetch<true, WT, GT, MASTER, E4M3>(e, unit + 1, kUnit, lane, next);
          adamw_unit<true, PT, WT, GT, MASTER, E4M3>(t, e, unit, kUnit, coef, s, lane, now);
          if (E4M3) now = next;
        }
      } else {
        const int64_t left = e.n - unit * kUnit;
        const int n = static_cast<int>(left < kUnit ? left : kUnit);
        Raw<GT, WT, E4M3> now;
        adamw_fetch<false, WT, GT, MASTER, E4M3>(e, unit, n, lane, now);
        adamw_unit<false, PT, WT, GT, MASTER, E4M3>(t, e, unit, n, coef, s, lane, now);
        ++at;
      }
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
constexpr int kAhead = 8;  // units of a warp in flight

// Whether a run's sum of squares is one: squares of fp32 numbers overflow from
// 2^64 on, and each of the run's 64 may be off by 2^-150, which is next to
// nothing of a sum above 2^-110.  `bits`: of all its values, signs apart.
__device__ __forceinline__ bool sum_holds(float s, uint32_t bits) {
  return (s >= 0x1p-110f && s < INFINITY) || bits == 0;
}
// What a warp of norm_kernel adds up, whatever the magnitudes: eight values of
// a lane at a time, over a power of two near the largest of them.
template <int N>
__device__ __noinline__ double scaled_squares(const Spans<N>& t, int64_t r, int64_t step, int lane) {
  double total = 0.0;
  for (int k = 0; r * kAhead < t.units; r += step) {
    for (int64_t u = r * kAhead; u < (r + 1) * kAhead && u < t.units; ++u) {
      while (k + 1 < t.count && u >= t.e[k + 1].first) ++k;
      const Span& e = t.e[k];
      float x[8], top = 0.0f, sum = 0.0f;
      for (int i = 0; i < 8; ++i) {
        const int64_t at = (u - e.first) * kUnit + lane * 8 + i;
        x[i] = 0.0f;
        if (at < e.n)
          x[i] = e.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.p)[at]) : static_cast<const float*>(e.p)[at];
        top = max_nan(top, fabsf(x[i]), 0.0f);
      }
      if (!(top > 0.0f && top < INFINITY)) {  // 0, infinity or NaN
        total += top;
        continue;
      }
      const uint32_t f = __float_as_uint(top) >> 23, E = f < 1 ? 1 : f > 253 ? 253 : f;
      const float down = __uint_as_float((254 - E) << 23), up = __uint_as_float(E << 23);  // 2^(127 - E), 2^(E - 127)
      for (int i = 0; i < 8; ++i) sum = fmaf(x[i] * down, x[i] * down, sum);
      total += static_cast<double>(sum) * up * up;
    }
  }
  return total;
}

// Partial sums of squares, one for each block, of a fixed assignment of units.
template <int N>
__global__ void __launch_bounds__(32 * kWarps) norm_kernel(const __grid_constant__ Spans<N> t, double* part) {
  __shared__ double red[kWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  double total = 0.0;
  bool holds = true;
  // kAhead consecutive units of a warp at a time: inside one tensor, all
  // their loads are in flight before the first sum
  const int64_t runs = (t.units + kAhead - 1) / kAhead;
  int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + w;
  int k = entry_of(t.e, t.count, r * kAhead);
  for (; r < runs; r += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t u0 = r * kAhead;
    // a run's 64 squares of a lane in fp32, runs in fp64: a long fp32 sum
    // would lose the small terms, always downwards
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t bits = 0;
    while (k + 1 < t.count && u0 >= t.e[k + 1].first) ++k;
    const int64_t at0 = (u0 - t.e[k].first) * kUnit;
    if (t.e[k].wide && t.e[k].n - at0 >= kAhead * kUnit) {
      if (t.e[k].bf16) {  // 16 bytes a lane and load
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(t.e[k].p) + at0) + lane;
        uint4 q[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) q[i] = p[32 * i];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint32_t v[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = __uint_as_float(v[j] << 16), hi = __uint_as_float(v[j] & 0xffff0000u);
            acc[j] = fmaf(lo, lo, fmaf(hi, hi, acc[j]));
            bits |= v[j] & 0x7fff7fffu;
          }
        }
      } else {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(t.e[k].p) + at0) + lane;
        float4 q[2 * kAhead];
#pragma unroll
        for (int i = 0; i < 2 * kAhead; ++i) q[i] = p[32 * i];
#pragma unroll
        for (int i = 0; i < 2 * kAhead; ++i) {
          acc[0] = fmaf(q[i].x, q[i].x, acc[0]);
          acc[1] = fmaf(q[i].y, q[i].y, acc[1]);
          acc[2] = fmaf(q[i].z, q[i].z, acc[2]);
          acc[3] = fmaf(q[i].w, q[i].w, acc[3]);
          bits |= (__float_as_uint(q[i].x) | __float_as_uint(q[i].y) | __float_as_uint(q[i].z) | __float_as_uint(q[i].w)) &
                  0x7fffffffu;
        }
      }
      const float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      holds = holds && sum_holds(sum, bits);
      total += sum;
      continue;
    }
    int kk = k;
    for (int64_t u = u0; u < u0 + kAhead && u < t.units; ++u) {
      while (kk + 1 < t.count && u >= t.e[kk + 1].first) ++kk;
      const Span& e = t.e[kk];
      const int64_t at = (u - e.first) * kUnit, left = e.n - at;
      const int n = static_cast<int>(left < kUnit ? left : kUnit);
      float x[2][4];
      if (e.bf16) {
        Four<__nv_bfloat16> f[2];
        fetch<false>(static_cast<const __nv_bfloat16*>(e.p) + at, lane, n, f);
        unpack(f[0], x[0]);
        unpack(f[1], x[1]);
      } else {
        Four<float> f[2];
        fetch<false>(static_cast<const float*>(e.p) + at, lane, n, f);
        unpack(f[0], x[0]);
        unpack(f[1], x[1]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[j] = fmaf(x[0][j], x[0][j], fmaf(x[1][j], x[1][j], acc[j]));
        bits |= (__float_as_uint(x[0][j]) | __float_as_uint(x[1][j])) & 0x7fffffffu;
      }
    }
    const float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    holds = holds && sum_holds(sum, bits);
    total += sum;
  }
  if (__any_sync(0xffffffffu, !holds))
    total = scaled_squares(t, static_cast<int64_t>(blockIdx.x) * kWarps + w, static_cast<int64_t>(gridDim.x) * kWarps, lane);
  double a = total;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (lane == 0) red[w] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    a = 0.0;
    for (int i = 0; i < kWarps; ++i) a += red[i];
    part[blockIdx.x] = a;
  }
}

// norm = sqrt of the sum of the partial sums (fp64, fixed order) and the
// coefficient that brings it to max_norm (max_norm <= 0: 1).
__global__ void __launch_bounds__(1024) norm_finish_kernel(const double* part, int n, double max_norm, float* out) {
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
    c = fminf(1.0f, __fdiv_rn(static_cast<float>(max_norm), __fadd_rn(norm, 1e-6f)));
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
  // e4m3: registers leave three blocks an SM; runs of 16 units a warp and
  // sixteen blocks an SM in the grid measured best (218 M elements: runs of
  // 4, 8, 16, 32, 128 units 604, 539, 510, 508, 567 us).  fp32: one wave.
  const int64_t warps = int64_t(sms()) * (E4M3 ? 3 : 4) * kWarps;  // resident
  t.chunk = t.units >= 64 * warps ? 16 : t.units >= 8 * warps ? 4 : 1;
  const int64_t blocks = (t.units + kWarps - 1) / kWarps, most = int64_t(sms()) * (E4M3 ? 16 : 4);
  ProfScope prof("adamw", E4M3 ? "e4m3" : "f32", 0.0, double(elements) * per_element, s);
  adamw_kernel<PT, GT, MASTER, E4M3, N><<<static_cast<unsigned>(blocks < most ? blocks : most), 32 * kWarps, 0, s>>>(t);
  note_launch();
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? TPS_OK : fail(TPS_ERR_CUDA, "adamw: launch failed: %s", cudaGetErrorString(cudaGetLastError()));
}

template <int N>
int launch_norm(const Spans<kMany>& all, double* part, int blocks, cudaStream_t s) {
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
    if (t.place < 0 || t.place % kUnit != 0)
      return fail(TPS_ERR_ARG, "tensor %d: place must be a multiple of %d, at least 0", i, kUnit);
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
    Table<kMany> tab;
    tab.count = 0;
    tab.units = 0;
    tab.random = h->stochastic ? 0xffffffffu : 0u;
    tab.nearest = h->stochastic ? 0u : 0x80008000u;
    tab.coef = grad_scale;
    tab.dev = device_scalars;
    tab.s = sc;
    tab.b1 = static_cast<float>(h->beta1);
    tab.c1 = static_cast<float>(1.0 - h->beta1);
    tab.b2 = static_cast<float>(h->beta2);
    tab.c2 = static_cast<float>(1.0 - h->beta2);
    tab.eps = static_cast<float>(h->eps);
    tab.minus_zero = -0.0f;
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
  return n < 0 ? 0 : align256(static_cast<size_t>(kNormBlocks) * ((n + kMany - 1) / kMany + 1) * sizeof(double));
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
  double* part = static_cast<double*>(workspace);
  Spans<kMany> t;
  t.count = 0;
  t.units = 0;
  int parts = 0, rc;
  double bytes = 0.0;
  for (int32_t i = 0; i <= n; ++i) {
    const bool end = i == n;
    if (!end && grads[i].numel == 0) continue;
    if ((end || t.count == kMany) && t.count > 0) {
      const int64_t want = (t.units + kAhead * kWarps - 1) / (kAhead * kWarps);
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
