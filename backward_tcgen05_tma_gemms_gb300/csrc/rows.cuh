// rows.cuh -- device pieces of the kernels that work on the rows of matrices:
// runs of N elements in f32 or bf16 (the type is known at run time), e4m3
// codes of a row under one scale, and the generator of the dropout mask.
#pragma once
#include <cuda_bf16.h>

#include "internal.cuh"

namespace tps {

// Rows of n elements, `ld` elements apart; dtype TPS_F32, TPS_BF16 or TPS_E4M3.
struct Rows {
  char* p;
  int64_t ld;
  int dtype;
  __device__ __forceinline__ char* at(int64_t row, int64_t col) const {
    const int64_t i = row * ld + col;
    return p + (dtype == TPS_F32 ? 4 * i : dtype == TPS_BF16 ? 2 * i : i);
  }
};

// A run of N consecutive elements as loaded, before its conversion: loads of
// several runs are in flight together whatever their types are.
template <int N>
struct Raw;
template <>
struct Raw<8> {
  uint4 a, b;
};
template <>
struct Raw<1> {
  uint32_t a;
};
// N = 8: 16-byte aligned.  Plain loads: an output may be one of the inputs.
__device__ __forceinline__ void raw_load(const char* p, int dtype, Raw<8>& r) {
  r.a = *reinterpret_cast<const uint4*>(p);
  if (dtype == TPS_F32) r.b = *(reinterpret_cast<const uint4*>(p) + 1);
}
__device__ __forceinline__ void raw_load(const char* p, int dtype, Raw<1>& r) {
  if (dtype == TPS_F32)
    r.a = *reinterpret_cast<const uint32_t*>(p);
  else
    r.a = *reinterpret_cast<const uint16_t*>(p);
}
__device__ __forceinline__ void raw_value(const Raw<8>& r, int dtype, float (&v)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  if (dtype == TPS_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void raw_value(const Raw<1>& r, int dtype, float (&v)[1]) {
  v[0] = __uint_as_float(dtype == TPS_F32 ? r.a : r.a << 16);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ void run_store(char* p, int dtype, const float (&v)[8]) {
  if (dtype == TPS_F32) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
}
__device__ __forceinline__ void run_store(char* p, int dtype, const float (&v)[1]) {
  if (dtype == TPS_F32)
    *reinterpret_cast<float*>(p) = v[0];
  else
    *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v[0]);
}
// v as `dtype` holds it.
template <int N>
__device__ __forceinline__ void run_round(int dtype, float (&v)[N]) {
  if (dtype == TPS_BF16) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __bfloat162float(__float2bfloat16_rn(v[i]));
  }
}

// The same with the type known at compile time.
template <class T, int N>
struct Typed {
  static constexpr int kWords = N * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 q = *(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = q.x;
      w[4 * i + 1] = q.y;
      w[4 * i + 2] = q.z;
      w[4 * i + 3] = q.w;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      *(reinterpret_cast<uint4*>(p) + i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[i]);
    else
      return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[N]) {  // rounds
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
  }
};
template <class T>
struct Typed<T, 1> {
  T x;
  __device__ __forceinline__ void load(const T* p) { x = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = x; }
  __device__ __forceinline__ float at(int) const {
    if constexpr (sizeof(T) == 4)
      return x;
    else
      return __bfloat162float(x);
  }
  __device__ __forceinline__ void set(const float (&v)[1]) {
    if constexpr (sizeof(T) == 4)
      x = v[0];
    else
      x = __float2bfloat16_rn(v[0]);
  }
};
// a + b of two bf16 runs, rounded once.
__device__ __forceinline__ void add_bf16(Typed<__nv_bfloat16, 8>& a, const Typed<__nv_bfloat16, 8>& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 x = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a.w[i]),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b.w[i]));
    a.w[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
}
template <class T>
constexpr int dtype_of() { return sizeof(T) == 4 ? TPS_F32 : TPS_BF16; }

// ---- e4m3 codes of a row under one scale -----------------------------------
// The row's largest magnitude `top` becomes 448.  448 v / top is formed as
// (7/8 v) / (top / 512), correctly rounded: a first quotient by the reciprocal
// and one step that adds the remainder's share (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  For
// bf16 values both terms are exact, so that ties between two codes are ties
// and go to the even one.  Rows whose largest magnitude is below 1e-30 are
// zeros with the scale 0; a NaN makes the scale NaN.
struct RowCodes {
  float top, t, r;  // top / 512 and its reciprocal, 0 for a row of zeros and for one with an infinity
  __device__ __forceinline__ explicit RowCodes(float x) {
    top = x < 1e-30f ? 0.0f : x;
    t = top * (1.0f / 512.0f);
    r = top == 0.0f ? 0.0f : __frcp_rn(t);
    if (r == 0.0f) t = 0.0f;
  }
  __device__ __forceinline__ float scale() const { return __fdiv_rn(top, 448.0f); }
  __device__ __forceinline__ float of(float v) const {
    const float a = v * 0.875f, q = a * r;
    return fmaf(fmaf(-q, t, a), r, q);
  }
};
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t x;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(x) : "f"(hi), "f"(lo));
  return x;
}
__device__ __forceinline__ void codes_store(char* p, const RowCodes& c, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_e4m3x2(c.of(v[2 * i]), c.of(v[2 * i + 1]));
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}
__device__ __forceinline__ void codes_store(char* p, const RowCodes& c, const float (&v)[1]) {
  *reinterpret_cast<uint8_t*>(p) = static_cast<uint8_t>(pack_e4m3x2(c.of(v[0]), 0.0f));
}

// ---- dropout ----------------------------------------------------------------
// Element i of a tensor (its place in row-major order) is kept where 16 bits
// of Philox 4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers:
// as easy as 1, 2, 3", 2011) are at least `step`, and multiplied by
// 65536 / (65536 - step).  The key is the seed, the counter (i / 8, site); the
// eight elements that share a counter take the low and high halves of its four
// words in turn.  16 bits an element and not 32: the generator's 20 wide
// products are then shared by eight elements, and a pass stays bound by memory;
// a probability in steps of 2^-16 is off by at most 2^-17, and the multiplier
// goes with the probability that is used.
constexpr uint32_t kPhiloxW0 = 0x9e3779b9u, kPhiloxW1 = 0xbb67ae85u;  // what a round adds to the key
struct Dropout {
  uint64_t seed;
  const int64_t* seed_ptr;  // when set, the seed is read from here
  uint64_t site;
  uint32_t step;   // 0: everything is kept
  uint32_t keys[20];  // of a seed that the host knows: the two words of each round
  uint32_t below;  // (step << 16) - 1: 16 bits in the upper half of a word are kept where the word is larger
  float scale;
  __device__ __forceinline__ uint64_t key() const { return seed_ptr != nullptr ? static_cast<uint64_t>(*seed_ptr) : seed; }
};

__device__ __forceinline__ uint4 philox(const Dropout& d, uint64_t key, uint64_t index) {
  uint32_t c0 = static_cast<uint32_t>(index), c1 = static_cast<uint32_t>(index >> 32);
  uint32_t c2 = static_cast<uint32_t>(d.site), c3 = static_cast<uint32_t>(d.site >> 32);
  auto round = [&](uint32_t k0, uint32_t k1) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xd2511f53u, b = static_cast<uint64_t>(c2) * 0xcd9e8d57u;
    const uint32_t n0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0, n2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    c0 = n0;
    c2 = n2;
  };
  if (d.seed_ptr == nullptr) {  // the words are operands from the parameters
#pragma unroll
    for (int i = 0; i < 10; ++i) round(d.keys[2 * i], d.keys[2 * i + 1]);
  } else {
    uint32_t k0 = static_cast<uint32_t>(key), k1 = static_cast<uint32_t>(key >> 32);
#pragma unroll 1
    for (int i = 0; i < 10; ++i) {
      round(k0, k1);
      k0 += kPhiloxW0;
      k1 += kPhiloxW1;
    }
  }
  return make_uint4(c0, c1, c2, c3);
}
// v times the mask of the elements from `index` on (N = 8: a multiple of 8).
// What is dropped is 0 whatever it held.
__device__ __forceinline__ void drop(const Dropout& d, uint64_t key, int64_t index, float (&v)[8]) {
  const uint4 u = philox(d, key, static_cast<uint64_t>(index) >> 3);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (w[i] << 16) > d.below ? v[2 * i] * d.scale : 0.0f;
    v[2 * i + 1] = w[i] > d.below ? v[2 * i + 1] * d.scale : 0.0f;
  }
}
__device__ __forceinline__ void drop(const Dropout& d, uint64_t key, int64_t index, float (&v)[1]) {
  const uint4 u = philox(d, key, static_cast<uint64_t>(index) >> 3);
  const int j = static_cast<int>(index & 7);
  const uint32_t w = j < 4 ? (j < 2 ? u.x : u.y) : (j < 6 ? u.z : u.w);
  v[0] = (j & 1 ? w : w << 16) > d.below ? v[0] * d.scale : 0.0f;
}

}  // namespace tps
