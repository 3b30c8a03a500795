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
// of threads once, and the group joins its sums by shuffles and one round
// through shared memory; blocks walk the rows, and bulk copies keep a ring of
// the next rows in shared memory full, whatever the threads wait for.  8192 x
// 4096 in bf16 with residual take 46 us (5.8 TB/s) where loads into registers,
// with those of the next row ahead of the sums, took 52, 64 rows 3.4 us and 5.9,
// and the backward pass of 9728 rows 55 us and 81.  The e4m3 output needs the
// largest |h w| of the row, which is reduced together with the sum of squares:
// the codes do not depend on r.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "api_common.cuh"
#include "ptx.cuh"
#include "rows.cuh"
#include "rows_host.cuh"

namespace tps {

namespace {

constexpr int kMaxGroup = 512;     // threads of a row at most
constexpr int kMaxWarps = kMaxGroup / 32;
constexpr int kRingThreads = 256;  // of a block with a ring at most
constexpr int kLongThreads = 256;  // of a row that does not fit into registers
static_assert(kLongThreads <= kMaxGroup, "the warps' sums fit");
constexpr int64_t kDwCols = 256;   // columns of a block of the long rows' weight gradient
constexpr int64_t kSplits = 152;   // and the runs of rows it is split into

struct NormParams {
  Rows x, res, h, y;  // p of res, h: nullptr when absent
  const char* w;      // nullptr: ones
  int w_dtype;
  float* rstd;        // nullptr: no norm (codes of x)
  float* scale;       // e4m3 output
  int64_t rows, d;
  float eps, inv_d;
  Dropout drop;
  int stages;         // of a ring
  uint32_t* err;
};

// Sums (and the NaN-keeping maximum of magnitudes) over the G threads of a
// row group.  `buf` alternates between two halves, so that one barrier a call
// is enough.
struct Joined {
  float sum, top;
};
template <bool TOP, bool SYNC = false>  // SYNC: a barrier of the block in any case
__device__ __forceinline__ Joined join_group(Joined v, int G, float2 (&buf)[kMaxWarps]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.sum += __shfl_xor_sync(0xffffffffu, v.sum, o);
    if (TOP) v.top = max_nan(v.top, __shfl_xor_sync(0xffffffffu, v.top, o), 0.0f);
  }
  if (G <= 32) {
    if (SYNC) __syncthreads();
    return v;
  }
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

struct NormBwdParams {
  Rows dy, h, dh, dsum, dx;  // p of dh, dsum, dx: nullptr when absent
  const char* w;
  int w_dtype;
  const float* rstd;
  float* part;               // partial weight gradients [block][d], nullptr: none
  int64_t rows, d;
  float inv_d;
  Dropout drop;
  int stages;
  uint32_t* err;
};

// ---- rows through a ring ----------------------------------------------------
// The next rows of up to three tensors in shared memory: a stage holds one row
// of each for every group of the block.  A stage is filled again once the whole
// block has taken its rows into registers.
constexpr int kMaxStages = 8;
struct RowRing {
  uint64_t full[kMaxStages];
  uint32_t abort;
};
struct RingSource {
  const char* p[3];
  int64_t pitch[3];  // bytes
  int bytes[3];      // of a row, a multiple of 16; 0: no such tensor
};
__device__ __forceinline__ int ring_row_bytes(const RingSource& s) { return s.bytes[0] + s.bytes[1] + s.bytes[2]; }
// By the first warp: the rows from row0 on into a stage.
__device__ __forceinline__ void ring_fill(const RingSource& s, RowRing* ring, char* at, int stage, int groups, int64_t row0,
                                          int64_t rows) {
  if (row0 >= rows) return;
  const int lane = threadIdx.x & 31, n = static_cast<int>(rows - row0 < groups ? rows - row0 : groups);
  const int one = ring_row_bytes(s);
  if (lane == 0) mbar_expect_tx(&ring->full[stage], static_cast<uint32_t>(n * one));
  __syncwarp();
  if (lane < n) {
    char* to = at + (stage * groups + lane) * one;
#pragma unroll
    for (int t = 0; t < 3; ++t)
      if (s.bytes[t] > 0) {
        bulk_load(to, s.p[t] + (row0 + lane) * s.pitch[t], static_cast<uint32_t>(s.bytes[t]), &ring->full[stage]);
        to += s.bytes[t];
      }
  }
}
__device__ __forceinline__ void ring_start(const RingSource& s, RowRing* ring, char* at, int stages, int groups, int64_t row0,
                                           int64_t step, int64_t rows) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&ring->full[i], 1);
    ring->abort = 0u;
    fence_mbar_init();
    fence_async_smem();
  }
  __syncthreads();
  if (threadIdx.x < 32)
    for (int i = 0; i < stages; ++i) ring_fill(s, ring, at, i, groups, row0 + i * step, rows);
}
// A stage whose copies did not arrive in time: what it holds is not used, but
// they must be over when the block ends.
__device__ __forceinline__ void ring_wait(RowRing* ring, int stage, uint32_t phase, uint32_t* err) {
  if (!mbar_wait(&ring->full[stage], phase, &ring->abort, err)) mbar_wait_drain(&ring->full[stage], phase, err);
}


// The weights of a thread's columns, as floats in registers: ones without weights and past the row.
template <int R>
__device__ __forceinline__ void ring_weights(const char* w, int dtype, int c0, int stride, int d, float (&v)[R][8]) {
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int c = c0 + k * stride;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = 1.0f;
    if (w != nullptr && c < d) {
      Raw<8> q;
      raw_load(w + c * (dtype == TPS_F32 ? 4 : 2), dtype, q);
      raw_value(q, dtype, v[k]);
    }
  }
}
// Blocks of kRingThreads threads on an SM that the registers are to allow, by
// the floats of a thread that live through a row.
constexpr int ring_blocks(int floats) { return floats <= 16 ? 4 : floats <= 32 ? 3 : floats <= 72 ? 2 : 1; }
constexpr int ring_fwd_blocks(int R, bool wide_h) { return ring_blocks(R * 8 + R * (wide_h ? 8 : 4)); }
constexpr int ring_bwd_blocks(int R) { return ring_blocks(2 * R * 8); }

// R runs of eight elements a thread, lane + k G in the row.  BARE: codes of x
// alone, without weights, norm and sum.
template <class TX, class TR, class TY, int R, bool BARE>
__global__ void __launch_bounds__(kRingThreads, BARE ? ring_blocks(R * (sizeof(TR) == 4 ? 8 : 4)) : ring_fwd_blocks(R, sizeof(TR) == 4))
    norm_fwd_ring_kernel(const NormParams p, const int G) {
  let_next_kernel_start();  // a product that reads the rows
  constexpr bool CODES = sizeof(TY) == 1;
  __shared__ float2 buf[2][kMaxWarps];
  __shared__ RowRing ring;
  extern __shared__ __align__(128) char stages_at[];
  const int groups = blockDim.x / G, group = threadIdx.x / G, lane = threadIdx.x & (G - 1), d = static_cast<int>(p.d);
  const bool normed = !BARE && p.rstd != nullptr, summed = !BARE && p.h.p != nullptr, joined = !BARE && p.res.p != nullptr;
  const bool drops = !BARE && p.drop.step != 0u;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups;
  const RingSource src = {{p.x.p, p.res.p, nullptr},
                          {p.x.ld * int(sizeof(TX)), p.res.ld * int(sizeof(TR)), 0},
                          {d * int(sizeof(TX)), joined ? d * int(sizeof(TR)) : 0, 0}};
  ring_start(src, &ring, stages_at, p.stages, groups, row0, step, p.rows);
  const int c0 = lane * 8, stride = G * 8;
  float w[R][8];
  if constexpr (!BARE) ring_weights(p.w, p.w_dtype, c0, stride, d, w);
  TR* hp = reinterpret_cast<TR*>(p.h.p) + (row0 + group) * p.h.ld + c0;
  TY* yp = reinterpret_cast<TY*>(p.y.p) + (row0 + group) * p.y.ld + c0;
  const uint64_t key = drops ? p.drop.key() : 0;
  int stage = 0, turn = 0;
  uint32_t phase = 0;
  for (; row0 < p.rows; row0 += step) {
    const bool live = row0 + group < p.rows;
    ring_wait(&ring, stage, phase, p.err);
    const char* at = stages_at + (stage * groups + group) * ring_row_bytes(src);
    const TX* xs = reinterpret_cast<const TX*>(at) + c0;
    const TR* rs = reinterpret_cast<const TR*>(at + src.bytes[0]) + c0;
    Typed<TR, 8> h[R];  // the row, as it is stored
    Joined own = {0.0f, 0.0f};
    if (live) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (c0 + k * stride >= d) continue;
        Typed<TX, 8> x;
        Typed<TR, 8> r;
        x.load(xs + k * stride);
        if (joined) r.load(rs + k * stride);
        bool have = false;
        if constexpr (sizeof(TX) == sizeof(TR)) {
          if (!drops && !joined) {
            h[k] = x;
            have = true;
          }
          if constexpr (sizeof(TX) == 2) {
            if (!drops && joined) {  // one rounding, two values an instruction
              h[k] = x;
              add_bf16(h[k], r);
              have = true;
            }
          }
        }
        if (!have) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = x.at(i);
          if (drops) drop(p.drop, key, (row0 + group) * d + c0 + k * stride, v);
          if (joined) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r.at(i);
          }
          h[k].set(v);
        }
        if (summed) h[k].store(hp + k * stride);
        if constexpr (!BARE) {
#pragma unroll
          for (int i = 0; i < 8; ++i) own.sum = fmaf(h[k].at(i), h[k].at(i), own.sum);
        }
        if constexpr (CODES) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float u = h[k].at(i), v = h[k].at(i + 1);
            own.top = BARE ? max_nan(own.top, fabsf(u), fabsf(v))
                           : max_nan(own.top, fabsf(u * w[k][i]), fabsf(v * w[k][i + 1]));
          }
        }
      }
    }
    own = join_group<CODES, true>(own, G, buf[turn]);
    turn ^= 1;
    // everyone has the stage's rows
    if (threadIdx.x < 32) ring_fill(src, &ring, stages_at, stage, groups, row0 + p.stages * step, p.rows);
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1u;
    }
    if (live) {
      const float rstd = normed ? rsqrtf(fmaf(own.sum, p.inv_d, p.eps)) : 1.0f;
      const RowCodes codes(own.top);
      if (lane == 0) {
        if (normed) p.rstd[row0 + group] = rstd;
        if (CODES) p.scale[row0 + group] = codes.scale() * rstd;
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (c0 + k * stride >= d) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = BARE ? h[k].at(i) : h[k].at(i) * w[k][i];
        if constexpr (CODES) {
          codes_store(reinterpret_cast<char*>(yp + k * stride), codes, v);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= rstd;
          Typed<TY, 8> y;
          y.set(v);
          y.store(yp + k * stride);
        }
      }
    }
    hp += step * p.h.ld;
    yp += step * p.y.ld;
  }
}

// The rows are taken out of the stage twice, before and after the join, and the
// stage is filled again at the next row's join.
template <class TD, class TH, class TX, int R>
__global__ void __launch_bounds__(kRingThreads, ring_bwd_blocks(R)) norm_bwd_ring_kernel(const NormBwdParams p, const int G) {
  __shared__ float2 buf[2][kMaxWarps];
  __shared__ RowRing ring;
  extern __shared__ __align__(128) char stages_at[];  // at last [row group][d] sums of dw
  const int groups = blockDim.x / G, group = threadIdx.x / G, lane = threadIdx.x & (G - 1), d = static_cast<int>(p.d);
  const bool past = p.dh.p != nullptr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups;
  const RingSource src = {{p.dy.p, p.h.p, p.dh.p},
                          {p.dy.ld * int(sizeof(TD)), p.h.ld * int(sizeof(TH)), p.dh.ld * int(sizeof(TH))},
                          {d * int(sizeof(TD)), d * int(sizeof(TH)), past ? d * int(sizeof(TH)) : 0}};
  ring_start(src, &ring, stages_at, p.stages, groups, row0, step, p.rows);
  const int c0 = lane * 8, stride = G * 8;
  float w[R][8], dw[R][8];
  ring_weights(p.w, p.w_dtype, c0, stride, d, w);
#pragma unroll
  for (int k = 0; k < R; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = 0.0f;
  TH* dsp = reinterpret_cast<TH*>(p.dsum.p) + (row0 + group) * p.dsum.ld + c0;
  TX* dxp = reinterpret_cast<TX*>(p.dx.p) + (row0 + group) * p.dx.ld + c0;
  const uint64_t key = p.drop.step != 0u ? p.drop.key() : 0;
  int stage = 0, turn = 0;
  uint32_t phase = 0;
  bool first = true;
  for (; row0 < p.rows; row0 += step) {
    const bool live = row0 + group < p.rows;
    const float r = live ? __ldg(p.rstd + row0 + group) : 0.0f;
    ring_wait(&ring, stage, phase, p.err);
    const char* at = stages_at + (stage * groups + group) * ring_row_bytes(src);
    const TD* as = reinterpret_cast<const TD*>(at) + c0;
    const TH* bs = reinterpret_cast<const TH*>(at + src.bytes[0]) + c0;
    const TH* is = reinterpret_cast<const TH*>(at + src.bytes[0] + src.bytes[1]) + c0;
    Joined own = {0.0f, 0.0f};
    if (live) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (c0 + k * stride >= d) continue;
        Typed<TD, 8> a;
        Typed<TH, 8> b;
        a.load(as + k * stride);
        b.load(bs + k * stride);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = b.at(i) * r, g = a.at(i) * n;
          dw[k][i] += g;
          own.sum = fmaf(g, w[k][i], own.sum);
        }
      }
    }
    own = join_group<false, true>(own, G, buf[turn]);
    turn ^= 1;
    // everyone is done with the row before
    if (!first && threadIdx.x < 32)
      ring_fill(src, &ring, stages_at, (stage == 0 ? p.stages : stage) - 1, groups, row0 + (p.stages - 1) * step, p.rows);
    first = false;
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1u;
    }
    const float pull = -own.sum * p.inv_d * r;  // what h r is multiplied by
    if (live) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (c0 + k * stride >= d) continue;
        Typed<TD, 8> a;
        Typed<TH, 8> b, in;
        a.load(as + k * stride);
        b.load(bs + k * stride);
        if (past) in.load(is + k * stride);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = fmaf(a.at(i) * w[k][i], r, fmaf(b.at(i) * r, pull, past ? in.at(i) : 0.0f));
        if (p.dsum.p != nullptr) {
          Typed<TH, 8> o;
          o.set(v);
          o.store(dsp + k * stride);
        }
        if (p.dx.p != nullptr) {
          if (p.drop.step != 0u) drop(p.drop, key, (row0 + group) * d + c0 + k * stride, v);
          Typed<TX, 8> o;
          o.set(v);
          o.store(dxp + k * stride);
        }
      }
    }
    dsp += step * p.dsum.ld;
    dxp += step * p.dx.ld;
  }
  if (p.part == nullptr) return;
  let_next_kernel_start();
  float* sums = reinterpret_cast<float*>(stages_at);
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * d;
  __syncthreads();  // the rows are done with
#pragma unroll
  for (int k = 0; k < R; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + k * stride < d) sums[group * d + c0 + k * stride + i] = dw[k][i];
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float s = 0.0f;
    for (int q = 0; q < groups; ++q) s += sums[q * d + c];
    out[c] = s;
  }
}

// ---- rows of single elements -------------------------------------------------
// Rows that do not start on 16 bytes or do not hold whole runs of eight, up to
// kSingleRuns kMaxGroup columns: kSingleRuns elements a thread, lane + k G in the
// row, loaded into registers, the next row's ahead of the present one's sums;
// blockDim.x / G rows at a time.  TX: x; TR: the residual and h (x's type without
// a residual).
constexpr int kSingleRuns = 8;
template <class TX, class TR, class TY>
__global__ void __launch_bounds__(kMaxGroup, 2) norm_fwd_kernel(const NormParams p, const int G) {
  let_next_kernel_start();
  constexpr bool CODES = sizeof(TY) == 1;
  constexpr int R = kSingleRuns;
  __shared__ float2 buf[2][kMaxWarps];
  extern __shared__ __align__(16) float ws[];  // [d] weights, if there are any
  const int groups = blockDim.x / G, group = threadIdx.x / G, lane = threadIdx.x & (G - 1), d = static_cast<int>(p.d);
  const bool normed = p.rstd != nullptr, summed = p.h.p != nullptr, weighted = p.w != nullptr, joined = p.res.p != nullptr;
  // This thread's first column of the group's row, which moves on by `step` rows.
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group, row0 = row - group;
  const TX* xp = reinterpret_cast<const TX*>(p.x.p) + row * p.x.ld + lane;
  const TR* rp = reinterpret_cast<const TR*>(p.res.p) + row * p.res.ld + lane;
  TR* hp = reinterpret_cast<TR*>(p.h.p) + row * p.h.ld + lane;
  TY* yp = reinterpret_cast<TY*>(p.y.p) + row * p.y.ld + lane;
  Typed<TX, 1> x[R];
  Typed<TR, 1> r[R];
  auto fetch = [&] {
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (lane + k * G < d) {
        x[k].load(xp + k * G);
        if (joined) r[k].load(rp + k * G);
      }
    xp += step * p.x.ld;
    rp += step * p.res.ld;
  };
  if (row < p.rows) fetch();
  if (weighted) {
    for (int i = threadIdx.x; i < d; i += blockDim.x)
      ws[i] = p.w_dtype == TPS_F32 ? reinterpret_cast<const float*>(p.w)[i]
                                   : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.w)[i]);
    __syncthreads();
  }
  const uint64_t key = p.drop.step != 0u ? p.drop.key() : 0;
  int turn = 0;
  for (; row0 < p.rows; row0 += step, row += step) {
    const bool live = row < p.rows;
    float v[R];  // h, then w h
    Joined own = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < R; ++k) {
      v[k] = 0.0f;
      if (!live || lane + k * G >= d) continue;
      float q[1] = {x[k].at(0)};
      if (p.drop.step != 0u) drop(p.drop, key, row * d + lane + k * G, q);
      if (joined) q[0] += r[k].at(0);
      if (summed) {
        Typed<TR, 1> h;
        h.set(q);
        h.store(hp + k * G);
        q[0] = h.at(0);
      }
      v[k] = q[0];
      own.sum = fmaf(v[k], v[k], own.sum);
    }
    hp += step * p.h.ld;
    if (row + step < p.rows) fetch();
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (weighted && lane + k * G < d) v[k] *= ws[lane + k * G];
      if (CODES) own.top = max_nan(own.top, fabsf(v[k]), 0.0f);
    }
    own = join_group<CODES>(own, G, buf[turn]);
    turn ^= 1;
    const float rstd = normed ? rsqrtf(fmaf(own.sum, p.inv_d, p.eps)) : 1.0f;
    if (live) {
      const RowCodes codes(own.top);
      if (lane == 0) {
        if (normed) p.rstd[row] = rstd;
        if (CODES) p.scale[row] = codes.scale() * rstd;
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (lane + k * G >= d) continue;
        if constexpr (CODES) {
          const float q[1] = {v[k]};
          codes_store(reinterpret_cast<char*>(yp + k * G), codes, q);
        } else {
          const float q[1] = {v[k] * rstd};
          Typed<TY, 1> y;
          y.set(q);
          y.store(yp + k * G);
        }
      }
    }
    yp += step * p.y.ld;
  }
}

// TD: dy; TH: h, dh and dsum; TX: dx.  The sums of dw stay in registers.
template <class TD, class TH, class TX>
__global__ void __launch_bounds__(kMaxGroup, 1) norm_bwd_kernel(const NormBwdParams p, const int G) {
  constexpr int R = kSingleRuns;
  __shared__ float2 buf[2][kMaxWarps];
  extern __shared__ __align__(16) float ws[];  // [d] weights, if there are any; at last [row group][d] sums of dw
  const int groups = blockDim.x / G, group = threadIdx.x / G, lane = threadIdx.x & (G - 1), d = static_cast<int>(p.d);
  const bool past = p.dh.p != nullptr, weighted = p.w != nullptr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group, row0 = row - group;
  if (weighted) {
    for (int i = threadIdx.x; i < d; i += blockDim.x)
      ws[i] = p.w_dtype == TPS_F32 ? reinterpret_cast<const float*>(p.w)[i]
                                   : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.w)[i]);
    __syncthreads();
  }
  const uint64_t key = p.drop.step != 0u ? p.drop.key() : 0;
  float w[R], dw[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    w[k] = weighted && lane + k * G < d ? ws[lane + k * G] : 1.0f;
    dw[k] = 0.0f;
  }
  Typed<TD, 1> a[R];
  Typed<TH, 1> b[R], in[R];
  auto fetch = [&](int64_t at) {
    const TD* dyp = reinterpret_cast<const TD*>(p.dy.p) + at * p.dy.ld + lane;
    const TH* hp = reinterpret_cast<const TH*>(p.h.p) + at * p.h.ld + lane;
    const TH* dhp = reinterpret_cast<const TH*>(p.dh.p) + at * p.dh.ld + lane;
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (lane + k * G < d) {
        a[k].load(dyp + k * G);
        b[k].load(hp + k * G);
        if (past) in[k].load(dhp + k * G);
      }
  };
  if (row < p.rows) fetch(row);
  int turn = 0;
  for (; row0 < p.rows; row0 += step, row += step) {
    const bool live = row < p.rows;
    const float r = live ? __ldg(p.rstd + row) : 0.0f;
    float g[R], n[R], up[R];  // dy w, h r and dh
    Joined own = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < R; ++k) {
      g[k] = n[k] = up[k] = 0.0f;
      if (!live || lane + k * G >= d) continue;
      g[k] = a[k].at(0) * w[k];
      n[k] = b[k].at(0) * r;
      if (past) up[k] = in[k].at(0);
      dw[k] = fmaf(a[k].at(0), n[k], dw[k]);
      own.sum = fmaf(g[k], n[k], own.sum);
    }
    if (row + step < p.rows) fetch(row + step);
    own = join_group<false>(own, G, buf[turn]);
    turn ^= 1;
    const float pull = -own.sum * p.inv_d * r;  // what h r is multiplied by
    if (live) {
      TH* dsp = reinterpret_cast<TH*>(p.dsum.p) + row * p.dsum.ld + lane;
      TX* dxp = reinterpret_cast<TX*>(p.dx.p) + row * p.dx.ld + lane;
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (lane + k * G >= d) continue;
        float v[1] = {fmaf(g[k], r, fmaf(n[k], pull, up[k]))};
        if (p.dsum.p != nullptr) {
          Typed<TH, 1> o;
          o.set(v);
          o.store(dsp + k * G);
        }
        if (p.dx.p != nullptr) {
          if (p.drop.step != 0u) drop(p.drop, key, row * d + lane + k * G, v);
          Typed<TX, 1> o;
          o.set(v);
          o.store(dxp + k * G);
        }
      }
    }
  }
  if (p.part == nullptr) return;
  let_next_kernel_start();
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * d;
  __syncthreads();  // the weights are done with
#pragma unroll
  for (int k = 0; k < R; ++k)
    if (lane + k * G < d) ws[group * d + lane + k * G] = dw[k];
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float s = 0.0f;
    for (int q = 0; q < groups; ++q) s += ws[q * d + c];
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
  const float rstd = normed ? rsqrtf(fmaf(own.sum, p.inv_d, p.eps)) : 1.0f;
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
// How a call is run: runs of N elements, R of them a thread, G threads a row,
// blocks of `threads`, `per_sm` of them an SM walking the rows.
// N = 8: through a ring of `ring` stages, where every row of every tensor starts
// on 16 bytes and holds whole runs of eight, up to 16384 columns.  Four runs a
// thread in bf16, two where fp32 is among the types (as many bytes), more for more
// than kRingThreads threads' worth.
// N = 1: single elements, where the types agree.  N = 0: the kernels of long rows.
constexpr int64_t kSms = 152, kMostBlocks = kSms * 16;
constexpr int kRingShared = 216 << 10;  // of an SM
struct Spread {
  int N, R, G, threads, ring, per_sm;
};
// row_bytes: of one row of all tensors that are read.
enum Pass { FORWARD, BACKWARD, CODES_ONLY };
Spread spread_of(int64_t rows, int64_t d, bool wide, bool fp32, bool mixed, int64_t row_bytes, Pass kind) {
  Spread s = {0, 0, 0, 0, 0, 0};
  if (wide) {
    const int64_t runs = (d + 7) / 8;
    Spread r = {8, fp32 ? 2 : 4, 0, 0, 0, 0};
    while (runs > int64_t(r.R) * kRingThreads && r.R < 8) r.R *= 2;
    if (runs <= int64_t(r.R) * kRingThreads) {
      const int64_t need = (runs + r.R - 1) / r.R;
      r.G = need <= 32 ? 32 : round_pow2(need);
      r.threads = r.G < 128 ? 128 : r.G;
      const int64_t stage = row_bytes * (r.threads / r.G);
      // registers: floats of a thread that live through a row
      const int floats = (kind == BACKWARD ? 16 : kind == FORWARD ? 8 : 0) * r.R + (kind == BACKWARD ? 0 : r.R * (fp32 ? 8 : 4));
      const int most = ring_blocks(floats) * kRingThreads / r.threads;
      for (int per = most; per >= 1 && r.ring == 0; --per) {
        const int64_t n = (kRingShared / per - 2048) / stage;
        if (n >= 2) {
          r.ring = static_cast<int>(n < kMaxStages ? n : kMaxStages);
          r.per_sm = per;
        }
      }
      if (r.ring > 0) return r;
    }
  }
  if (mixed || d > kSingleRuns * kMaxGroup) return s;
  s.N = 1;
  s.R = kSingleRuns;
  const int64_t need = (d + s.R - 1) / s.R;
  s.G = need <= 32 ? 32 : round_pow2(need);
  s.threads = s.G < 256 ? 256 : s.G;
  while (s.threads > s.G && (rows * s.G + s.threads - 1) / s.threads < 2 * kSms) s.threads /= 2;  // few rows: a block each
  s.per_sm = (kind == BACKWARD ? 512 : 1024) / s.threads;
  return s;
}

// Blocks of `f`, and its shared memory: the most that any call of it may have,
// for another host thread may be launching it with more than this call needs.
template <class F>
int prepare_launch(F f, const Spread& sp, int64_t rows, size_t shared, int64_t* blocks) {
  if (shared > (40u << 10) &&  // with the static part, beyond 48 KB
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingShared) != cudaSuccess)
    return fail(TPS_ERR_CUDA, "norm: %s", cudaGetErrorString(cudaGetLastError()));
  int64_t per = sp.per_sm;
  if (sp.ring == 0 && per * (int64_t(shared) + 2048) > kRingShared) per = kRingShared / (int64_t(shared) + 2048);
  const int64_t groups = sp.threads / sp.G, need = (rows + groups - 1) / groups, most = kSms * (per < 1 ? 1 : per);
  *blocks = need < most ? need : most;
  return TPS_OK;
}
int ring_ready(const Spread& sp, int* stages, uint32_t** err) {
  *stages = sp.ring;
  *err = device_error_word();
  return *err != nullptr ? TPS_OK : fail(TPS_ERR_CUDA, "cannot resolve the device error word");
}

template <class TX, class TR, class TY, int R, bool RING>
int launch_fwd(NormParams p, const Spread& sp, cudaStream_t s) {
  int64_t blocks = 0;
  int rc;
  if constexpr (RING) {
    const size_t shared = static_cast<size_t>(sp.ring) * (sp.threads / sp.G) * p.d * (sizeof(TX) + (p.res.p ? sizeof(TR) : 0));
    if ((rc = ring_ready(sp, &p.stages, &p.err))) return rc;
    if constexpr (sizeof(TY) == 1 && sizeof(TX) == sizeof(TR)) {
      if (p.rstd == nullptr) {
        if ((rc = prepare_launch(norm_fwd_ring_kernel<TX, TR, TY, R, true>, sp, p.rows, shared, &blocks))) return rc;
        norm_fwd_ring_kernel<TX, TR, TY, R, true><<<static_cast<unsigned>(blocks), sp.threads, shared, s>>>(p, sp.G);
        return launched("quantize");
      }
    }
    if ((rc = prepare_launch(norm_fwd_ring_kernel<TX, TR, TY, R, false>, sp, p.rows, shared, &blocks))) return rc;
    norm_fwd_ring_kernel<TX, TR, TY, R, false><<<static_cast<unsigned>(blocks), sp.threads, shared, s>>>(p, sp.G);
  } else {
    const size_t shared = p.w != nullptr ? sizeof(float) * p.d : 0;
    if ((rc = prepare_launch(norm_fwd_kernel<TX, TR, TY>, sp, p.rows, shared, &blocks))) return rc;
    norm_fwd_kernel<TX, TR, TY><<<static_cast<unsigned>(blocks), sp.threads, shared, s>>>(p, sp.G);
  }
  return launched("norm");
}
template <class TX, class TR, class TY>
int launch_fwd_typed(const NormParams& p, const Spread& sp, cudaStream_t s) {
  constexpr bool kBf16 = sizeof(TX) == 2 && sizeof(TR) == 2;
  if (sp.N == 1) {
    if constexpr (sizeof(TX) == sizeof(TR)) return launch_fwd<TX, TR, TY, 1, false>(p, sp, s);
    return fail(TPS_ERR_DTYPE, "norm: single elements of two types");
  }
  if constexpr (!kBf16)
    if (sp.R == 2) return launch_fwd<TX, TR, TY, 2, true>(p, sp, s);
  if (sp.R == 4) return launch_fwd<TX, TR, TY, 4, true>(p, sp, s);
  return launch_fwd<TX, TR, TY, 8, true>(p, sp, s);
}
template <class TX, class TR>
int launch_fwd_out(const NormParams& p, const Spread& sp, cudaStream_t s) {
  if (p.y.dtype == TPS_E4M3) return launch_fwd_typed<TX, TR, uint8_t>(p, sp, s);
  return p.y.dtype == TPS_F32 ? launch_fwd_typed<TX, TR, float>(p, sp, s) : launch_fwd_typed<TX, TR, __nv_bfloat16>(p, sp, s);
}

int launch_norm_fwd(const NormParams& p, const char* label, cudaStream_t s) {
  const bool wide = p.d % 8 == 0 && starts_runs(p.x, p.rows) && starts_runs(p.res, p.rows) && starts_runs(p.h, p.rows) &&
                    starts_runs(p.y, p.rows) && (p.w == nullptr || starts_runs(p.w, 0, p.w_dtype, 1));
  const int tx = p.x.dtype, tr = p.res.p != nullptr ? p.res.dtype : tx;
  const bool codes = p.y.dtype == TPS_E4M3;
  const int64_t row_bytes = p.d * (es_of(tx) + (p.res.p != nullptr ? es_of(tr) : 0));
  const Spread sp = spread_of(p.rows, p.d, wide, tx == TPS_F32 || tr == TPS_F32, tx != tr, row_bytes, p.rstd == nullptr ? CODES_ONLY : FORWARD);
  const double bytes = double(p.rows) * double(p.d) *
                       (es_of(p.x.dtype) + (p.res.p ? es_of(p.res.dtype) : 0) + (p.h.p ? es_of(p.h.dtype) : 0) + es_of(p.y.dtype));
  ProfScope prof("norm", label, 0.0, bytes, s);
  using bf16 = __nv_bfloat16;
  if (sp.N != 0)
    return tx == TPS_F32 ? (tr == TPS_F32 ? launch_fwd_out<float, float>(p, sp, s) : launch_fwd_out<float, bf16>(p, sp, s))
                         : (tr == TPS_F32 ? launch_fwd_out<bf16, float>(p, sp, s) : launch_fwd_out<bf16, bf16>(p, sp, s));
  const unsigned grid = static_cast<unsigned>(p.rows);
  if (wide)
    codes ? norm_fwd_long_kernel<8, true><<<grid, kLongThreads, 0, s>>>(p) : norm_fwd_long_kernel<8, false><<<grid, kLongThreads, 0, s>>>(p);
  else
    codes ? norm_fwd_long_kernel<1, true><<<grid, kLongThreads, 0, s>>>(p) : norm_fwd_long_kernel<1, false><<<grid, kLongThreads, 0, s>>>(p);
  return launched("norm_long");
}

template <class TD, class TH, class TX, int R, bool RING>
int launch_bwd(NormBwdParams p, const Spread& sp, int64_t* parts, cudaStream_t s) {
  const int64_t per = sp.threads / sp.G;
  const size_t sums = p.part != nullptr ? sizeof(float) * p.d * per : 0;
  int rc;
  if constexpr (RING) {
    size_t shared = static_cast<size_t>(sp.ring) * per * p.d * (sizeof(TD) + sizeof(TH) * (p.dh.p ? 2 : 1));
    if (shared < sums) shared = sums;
    if ((rc = ring_ready(sp, &p.stages, &p.err)) ||
        (rc = prepare_launch(norm_bwd_ring_kernel<TD, TH, TX, R>, sp, p.rows, shared, parts)))
      return rc;
    norm_bwd_ring_kernel<TD, TH, TX, R><<<static_cast<unsigned>(*parts), sp.threads, shared, s>>>(p, sp.G);
  } else {
    size_t shared = p.w != nullptr ? sizeof(float) * p.d : 0;
    if (shared < sums) shared = sums;
    if ((rc = prepare_launch(norm_bwd_kernel<TD, TH, TX>, sp, p.rows, shared, parts))) return rc;
    norm_bwd_kernel<TD, TH, TX><<<static_cast<unsigned>(*parts), sp.threads, shared, s>>>(p, sp.G);
  }
  return launched("norm_bwd");
}
template <class TD, class TH, class TX>
int launch_bwd_typed(const NormBwdParams& p, const Spread& sp, int64_t* parts, cudaStream_t s) {
  constexpr bool kBf16 = sizeof(TD) == 2 && sizeof(TH) == 2;
  if (sp.N == 1) {
    if constexpr (sizeof(TD) == sizeof(TH)) return launch_bwd<TD, TH, TX, 1, false>(p, sp, parts, s);
    return fail(TPS_ERR_DTYPE, "norm: single elements of two types");
  }
  if constexpr (!kBf16)
    if (sp.R == 2) return launch_bwd<TD, TH, TX, 2, true>(p, sp, parts, s);
  if (sp.R == 4) return launch_bwd<TD, TH, TX, 4, true>(p, sp, parts, s);
  return launch_bwd<TD, TH, TX, 8, true>(p, sp, parts, s);
}
template <class TD, class TH>
int launch_bwd_out(const NormBwdParams& p, const Spread& sp, int64_t* parts, cudaStream_t s) {
  return p.dx.dtype == TPS_F32 ? launch_bwd_typed<TD, TH, float>(p, sp, parts, s)
                               : launch_bwd_typed<TD, TH, __nv_bfloat16>(p, sp, parts, s);
}

}  // namespace

// Sum of `n` rows of d floats to out (f32 or bf16), in row order.
__global__ void __launch_bounds__(1024) sum_rows_kernel(const float* part, int64_t n, int64_t d, void* out, int dtype) {
  __shared__ float s[32][33];
  wait_for_prior_kernel();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float acc = 0.0f;
  if (c < d) {
    constexpr int U = 8;  // loads in flight
    for (int64_t i = w; i < n; i += U * warps) {
      float x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] = i + u * warps < n ? part[(i + u * warps) * d + c] : 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) acc += x[u];
    }
  }
  s[w][lane] = acc;
  __syncthreads();
  if (w != 0 || c >= d) return;
  acc = 0.0f;
  for (int i = 0; i < warps; ++i) acc += s[i][lane];
  if (dtype == TPS_F32)
    static_cast<float*>(out)[c] = acc;
  else
    static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(acc);
}

int launch_sum_rows(const float* part, int64_t n, int64_t d, void* out, int dtype, bool early, cudaStream_t s) {
  ProfScope prof("sum_rows", "dw", 0.0, 4.0 * double(n) * double(d), s);
  const int64_t warps = (n + 7) / 8 < 32 ? (n + 7) / 8 : 32;  // eight rows a warp at a time
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = early_attribute();
  cfg.gridDim = dim3(static_cast<unsigned>((d + 31) / 32), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps), 1, 1);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, sum_rows_kernel, part, n, d, out, dtype);
  note_launch();
  return e == cudaSuccess ? TPS_OK : fail(TPS_ERR_CUDA, "sum_rows: launch failed: %s", cudaGetErrorString(cudaGetLastError()));
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
  if (scale != nullptr && (rc = aligned_vector(scale, "scale", TPS_F32, rows))) return rc;
  if ((rc = aligned_vector(rstd, "rstd", TPS_F32, rows))) return rc;
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
  if ((rc = aligned_vector(scale, "scale", TPS_F32, rows))) return rc;
  if (rows == 0) return TPS_OK;
  if (d == 0) return fail(TPS_ERR_SHAPE, "rows without elements");
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
  if ((rc = aligned_vector(rstd, "rstd", TPS_F32, rows))) return rc;
  if (dH != nullptr && (rc = float_rows(dH, "dH", false, rows, d, &p.dh))) return rc;
  if ((rc = dropout_of(dropout, &p.drop))) return rc;
  if (dSum != nullptr && (rc = float_rows(dSum, "dSum", true, rows, d, &p.dsum))) return rc;
  for (const Rows* g : {&p.dh, &p.dsum})
    if (g->p != nullptr && g->dtype != p.h.dtype) return fail(TPS_ERR_DTYPE, "dH and dSum must have H's type");
  if (dX != nullptr && (rc = float_rows(dX, "dX", true, rows, d, &p.dx))) return rc;
  // One tensor for both holds both where they are one number.
  if (rows > 0 && d > 0 && p.dsum.p != nullptr && p.dsum.p == p.dx.p &&
      (p.drop.step != 0u || p.dx.dtype != p.dsum.dtype || (rows > 1 && p.dx.ld != p.dsum.ld)))
    return fail(TPS_ERR_ARG, "dSum and dX are one tensor, but differ by the dropout, their types or pitches");
  if (dweight != nullptr && (rc = aligned_vector(dweight, "dweight", TPS_F32, d))) return rc;
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
  if (dX == nullptr) p.dx.dtype = th;
  const int64_t row_bytes = d * (es_of(td) + es_of(th) * (p.dh.p != nullptr ? 2 : 1));
  const Spread sp = spread_of(rows, d, wide, td == TPS_F32 || th == TPS_F32, td != th, row_bytes, BACKWARD);
  int64_t parts = rows < kSplits ? rows : kSplits;
  if (p.part != nullptr || p.dsum.p != nullptr || p.dx.p != nullptr) {
    using bf16 = __nv_bfloat16;
    const double bytes = double(rows) * double(d) *
                         (es_of(p.dy.dtype) + es_of(p.h.dtype) + (p.dh.p ? es_of(p.dh.dtype) : 0) +
                          (p.dsum.p ? es_of(p.dsum.dtype) : 0) + (p.dx.p ? es_of(p.dx.dtype) : 0));
    ProfScope prof("norm", "bwd", 0.0, bytes, s);
    if (sp.N != 0) {
      rc = td == TPS_F32 ? (th == TPS_F32 ? launch_bwd_out<float, float>(p, sp, &parts, s) : launch_bwd_out<float, bf16>(p, sp, &parts, s))
                         : (th == TPS_F32 ? launch_bwd_out<bf16, float>(p, sp, &parts, s) : launch_bwd_out<bf16, bf16>(p, sp, &parts, s));
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
  // Launched early behind a short pass: backward norms of 64 x 4096, 600 x 2048 and
  // 8192 x 4096 in bf16 take 9.1, 9.2 and 47.8 us so, else 9.7, 9.8 and 47.1.
  const bool early = rows < (1ll << 24) / d;
  return p.part != nullptr ? launch_sum_rows(p.part, parts, d, dweight->data, TPS_F32, early, s) : TPS_OK;
}
