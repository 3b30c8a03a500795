// gemm_rows.cu -- Y = X W for a few rows of X (tokens), with the linear
// epilogue: the weights are read once, and that bounds it.
//
//   z = x w row_scale col_scale + bias,  y = act(z) + residual
//
// The roles of the operands are swapped: 128 output features are the rows of
// the tensor core's tile and up to 256 tokens its columns, so that the 128
// lanes of tensor memory are full of features however few tokens there are
// (tiles of tokens x features would leave all but a few of their rows empty).
// W is the A operand in either layout, X the B operand; the accumulator holds Y
// transposed.  X is K-major, or, for a weight gradient, has its unit stride
// along the rows, as W then has along the features.
//
// The 128-feature tiles alone are too few for the SMs and for the bytes in
// flight that memory wants, so a cluster of up to eight CTAs splits K: each
// accumulates its run, writes its partial tile to shared memory as [token][feature],
// and the CTAs of the cluster add up the eight partials of their share of the
// tokens in rank order, out of each other's shared memory, with the epilogue
// on the sums.  No workspace, no flags, results do not depend on timing.
//
// fp32 operands come as three bf16 planes (GemmDesc::planes): every CTA runs the
// six products over its part of K, the five that hold remainders into one
// accumulator and the product of the planes 0 into another, which alone
// decides about infinities and NaN (T2Drains in gemm_tc2.cu).
//
// It is launched early: its barriers and tensor memory are set up while the
// kernel in front (a norm, a quantisation or the laying out of the operands) ends.
// A norm and the product of 64 rows, 14336 to 4096, 30.1 -> 29.0 us in bf16, 20.7 ->
// 19.1 us in e4m3.  Fetching W into L2 before the wait as well gave these 27.7 and
// 17.8 us, but cost a product that follows none of them up to 1 us: left out.
//
// Warp roles (192 to 576 threads): warp 0 loads (TMA), warp 1 issues the MMAs, the
// others drain tensor memory, four at a time; all of them add and store.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdlib>
#include <cstring>

#include "api_common.cuh"
#include "tc_common.cuh"

namespace tps {

namespace {

constexpr int GR_THREADS = 192, GR_MOST_THREADS = 576;  // see threads_of
constexpr int GR_FEATURES = 128;
constexpr int GR_W_BYTES = GR_FEATURES * 128;  // 128 bytes of K for each feature
constexpr int GR_MAX_STAGES = 8, GR_MAX_SPLIT = 8;
constexpr int GR_TOKENS = 256;                 // columns of a tile at most

struct GrBarriers {
  uint64_t full[GR_MAX_STAGES];
  uint64_t empty[GR_MAX_STAGES];
  uint64_t done;
  uint32_t tmem_slot;
  uint32_t abort;
};

struct GrParams {
  int T, N;
  int k_tiles, bn, t_tiles, stages, splits;
  uint32_t tmem_cols;
  int x_plane, w_plane;  // PLANES: elements between planes
  Epilogue epi;
  uint32_t* err;
};

// Epilogue of four columns of one row.
__device__ __forceinline__ void rows_store4(void* base, int dtype, int64_t idx, int n, const float (&v)[4]) {
  if (dtype == TPS_F32) {
    float* p = static_cast<float*>(base) + idx;
    if (n == 4 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = v[i];
    }
  } else {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + idx;
    if (n == 4 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
      *reinterpret_cast<uint2*>(p) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = __float2bfloat16_rn(v[i]);
    }
  }
}
__device__ __forceinline__ void rows_load4(const void* base, int dtype, int64_t idx, int n, float (&a)[4]) {
  if (dtype == TPS_F32) {
    const float* p = static_cast<const float*>(base) + idx;
    if (n == 4 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
      const float4 q = *reinterpret_cast<const float4*>(p);
      a[0] = q.x, a[1] = q.y, a[2] = q.z, a[3] = q.w;
      return;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + idx;
    if (n == 4 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      a[0] = __uint_as_float(q.x << 16), a[1] = __uint_as_float(q.x & 0xffff0000u);
      a[2] = __uint_as_float(q.y << 16), a[3] = __uint_as_float(q.y & 0xffff0000u);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = i < n ? any_elem(base, dtype, idx + i) : 0.0f;
}

// Adds up the cluster's S partial tiles [token][128] (at the same shared-memory
// address in every CTA) and stores this CTA's share of the tokens.  A load from
// another CTA takes about a microsecond: the loads of U items of a thread are
// in flight together.  (Bulk copies of each share to its CTA, which then adds
// up out of its own shared memory, took 1 us more at every size.)
template <int S>
__device__ __forceinline__ void rows_join_of(const Epilogue& e, uint32_t part, uint32_t rank, int t0, int tokens, int64_t n0,
                                             int64_t N) {
  constexpr int U = S <= 2 ? 4 : 2;
  const int first = tokens * static_cast<int>(rank) / S * 32, last = tokens * (static_cast<int>(rank) + 1) / S * 32;
  uint32_t from[S];
#pragma unroll
  for (int s = 0; s < S; ++s) from[s] = cluster_map(part, s);
  for (int i0 = first + threadIdx.x; i0 < last; i0 += U * blockDim.x) {
    float4 q[U][S];
    float res[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * blockDim.x, t = i / 32, f = i % 32 * 4;
      const int64_t row = t0 + t, col = n0 + f;
      if (i >= last || col >= N) continue;
#pragma unroll
      for (int s = 0; s < S; ++s) q[u][s] = ld_cluster_f32x4(from[s] + static_cast<uint32_t>((t * GR_FEATURES + f) * 4));
      if (e.res != nullptr) rows_load4(e.res, e.res_dtype, row * e.ld_res + col, N - col < 4 ? static_cast<int>(N - col) : 4, res[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * blockDim.x, t = i / 32, f = i % 32 * 4;
      const int64_t row = t0 + t, col = n0 + f;
      if (i >= last || col >= N) continue;
      const int n = N - col < 4 ? static_cast<int>(N - col) : 4;
      float v[4] = {q[u][0].x, q[u][0].y, q[u][0].z, q[u][0].w};
#pragma unroll
      for (int s = 1; s < S; ++s) {
        v[0] += q[u][s].x;
        v[1] += q[u][s].y;
        v[2] += q[u][s].z;
        v[3] += q[u][s].w;
      }
      if (!dbg_store_ok(e, row, col, n)) continue;
      if (e.mode == EPI_LINEAR) {
        linear_pre(e, row, col, n, v);
        if (e.d2 != nullptr) rows_store4(e.d2, e.d2_dtype, row * e.ldd2 + col, n, v);
        linear_acted(e, v);
        if (e.res != nullptr) {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] += res[u][k];
        }
      }
      rows_store4(e.d, e.d_dtype, row * e.ldd + col, n, v);
    }
  }
}
__device__ __forceinline__ void rows_join(const Epilogue& e, uint32_t part, uint32_t rank, int splits, int t0, int tokens,
                                          int64_t n0, int64_t N) {
  switch (splits) {
    case 1: rows_join_of<1>(e, part, rank, t0, tokens, n0, N); break;
    case 2: rows_join_of<2>(e, part, rank, t0, tokens, n0, N); break;
    case 4: rows_join_of<4>(e, part, rank, t0, tokens, n0, N); break;
    default: rows_join_of<8>(e, part, rank, t0, tokens, n0, N); break;
  }
}

enum GrKind : int { GR_BF16 = 0, GR_CODES = 1, GR_PLANES = 2 };  // e4m3 operands; fp32 as bf16 planes
// Planes of X and of W in product i, two bits each: 2 1 0 1 0 0 and 0 1 2 0 1 0.
__device__ __forceinline__ int gr_x_plane(int i) { return (0x046 >> (2 * i)) & 3; }
__device__ __forceinline__ int gr_w_plane(int i) { return (0x124 >> (2 * i)) & 3; }

// W_MN: W's unit stride is along the features.  X_MN: X's along the rows.
template <bool W_MN, bool X_MN, int KIND>
__global__ void __launch_bounds__(GR_MOST_THREADS)
    gemm_rows_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx, const GrParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const int stage_bytes = GR_W_BYTES + p.bn * 128;
  GrBarriers* bars = reinterpret_cast<GrBarriers*>(smem + p.stages * stage_bytes);
  volatile uint32_t* abort_flag = &bars->abort;
  constexpr bool CODES = KIND == GR_CODES, PLANES = KIND == GR_PLANES;
  constexpr int kBK = CODES ? 128 : 64, kProducts = PLANES ? 6 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = p.splits > 1 ? cluster_ctarank() : 0;
  const int tile = static_cast<int>(blockIdx.x) / p.splits;
  const int n0 = tile / p.t_tiles * GR_FEATURES, t0 = tile % p.t_tiles * p.bn;
  const int tokens = min(p.bn, p.T - t0);
  const int kt_begin = static_cast<int>(static_cast<int64_t>(p.k_tiles) * rank / p.splits);
  const int kt_end = static_cast<int>(static_cast<int64_t>(p.k_tiles) * (rank + 1) / p.splits);

  const int run = kt_end - kt_begin, total = run * kProducts;  // K tiles of a product, and of all
  auto load = [&](int i) {  // K tile i of this CTA into its stage
    const int stage = i % p.stages, prod = PLANES ? i / run : 0;
    const int k0 = (kt_begin + (PLANES ? i - prod * run : i)) * kBK;
    const int xa = PLANES ? gr_x_plane(prod) * p.x_plane : 0, wa = PLANES ? gr_w_plane(prod) * p.w_plane : 0;
    uint8_t* sw = smem + stage * stage_bytes;
    mbar_expect_tx(&bars->full[stage], stage_bytes);
    if (W_MN) {
#pragma unroll
      for (int j = 0; j < GR_FEATURES / 64; ++j)
        tma_load_2d(sw + j * TC_MN_BOX_BYTES, &tw, &bars->full[stage], n0 + wa + 64 * j, k0);
    } else {
      tma_load_2d(sw, &tw, &bars->full[stage], k0 + wa, n0);
    }
    if (X_MN) {  // boxes of 64 rows of X
      for (int j = 0; j < p.bn / 64; ++j)
        tma_load_2d(sw + GR_W_BYTES + j * TC_MN_BOX_BYTES, &tx, &bars->full[stage], t0 + xa + 64 * j, k0);
    } else {
      tma_load_2d(sw + GR_W_BYTES, &tx, &bars->full[stage], k0 + xa, t0);
    }
  };
  int issued = 0;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tw);
    tma_prefetch_desc(&tx);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->done, 1);
    bars->abort = 0u;
    fence_mbar_init();
    fence_async_smem();  // this thread's copies count on them at once
    wait_for_prior_kernel();
    // the first loads do not wait for tensor memory
    for (; issued < total && issued < p.stages; ++issued) load(issued);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  wait_for_prior_kernel();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;
  const uint32_t main_at = PLANES ? p.tmem_cols / 2 : 0;  // the accumulator of the planes 0

  if (warp == 0) {
    if (lane == 0) {
      for (; issued < total; ++issued) {
        if (!mbar_wait(&bars->empty[issued % p.stages], ((issued / p.stages) & 1) ^ 1u, abort_flag, p.err)) break;
        load(issued);
      }
      // Copies in flight finish before the block ends, whatever the MMA thread did.
      for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
        mbar_wait_drain(&bars->full[i % p.stages], static_cast<uint32_t>((i / p.stages) & 1), p.err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = CODES ? idesc_e4m3_f32(GR_FEATURES, p.bn) : idesc_bf16_f32(GR_FEATURES, p.bn, W_MN, X_MN);
      for (int i = 0; i < total; ++i) {
        const int stage = i % p.stages;
        if (!mbar_wait(&bars->full[stage], (i / p.stages) & 1, abort_flag, p.err)) break;
        tc_fence_after();
        const bool last = PLANES && i >= 5 * run;  // the product of the planes 0
        const bool first = i == 0 || (PLANES && i == 5 * run);
        const uint32_t acc = tmem + (last ? main_at : 0);
        const uint32_t sw = smem_u32(smem + stage * stage_bytes), sx = sw + GR_W_BYTES;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t ad = W_MN ? smem_desc_sw128(sw + kk * 2048, TC_MN_BOX_BYTES, 1024)
                                   : smem_desc_sw128(sw + kk * 32, 16, 1024);
          const uint64_t bd = X_MN ? smem_desc_sw128(sx + kk * 2048, TC_MN_BOX_BYTES, 1024)
                                   : smem_desc_sw128(sx + kk * 32, 16, 1024);
          if (CODES)
            tc_mma_f8(acc, ad, bd, idesc, (!first || kk != 0) ? 1u : 0u);
          else
            tc_mma_f16(acc, ad, bd, idesc, (!first || kk != 0) ? 1u : 0u);
        }
        tc_commit(&bars->empty[stage]);
      }
      tc_commit(&bars->done);
      mbar_wait_drain(&bars->done, 0, p.err);
    }
  }
  __syncwarp();
  __syncthreads();  // the MMAs have completed: nothing reads or writes the stages any more
  tc_fence_after();
  if (warp >= 2) {
    const int q = warp & 3;
    float* part = reinterpret_cast<float*>(smem) + q * 32 + lane;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16);
    for (int c = (warp - 2) / 4 * 16; c < tokens; c += (blockDim.x / 32 - 2) / 4 * 16) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(t_row + c, r);
      tmem_ld_wait();
      if constexpr (PLANES) {  // remainders that are not finite are left out
        uint32_t m[16];
        tmem_ld_32x32b_x16(t_row + main_at + c, m);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float rest = __uint_as_float(r[i]);
          r[i] = __float_as_uint(__uint_as_float(m[i]) + (fabsf(rest) < INFINITY ? rest : 0.0f));
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < tokens) part[(c + i) * GR_FEATURES] = __uint_as_float(r[i]);
    }
    tc_fence_before();
  }
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  if (!*abort_flag)
    rows_join(p.epi, smem_u32(smem), rank, p.splits, t0, tokens, n0, p.N);
  if (p.splits > 1) cluster_sync();  // the others have read this CTA's partial tile
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// ---- fp32, up to eight rows ---------------------------------------------------
// The fp32 pipes do it: 2 T operations a weight of four bytes.  A block takes
// 128 features of the cluster's run of K, with that run of X in shared memory.
// One token through 14336 x 4096, (N, K), takes 39.5 us, 0.88 of the copy's rate.
constexpr int GF_ROWS = 8, GF_WARPS = 8;
constexpr int GF_SHARED = 96 << 10;  // of X

struct GfParams {
  const float* x;
  int64_t ldx;
  const float* w;
  int64_t ldw;
  int64_t T, N, K;
  int splits;
  Epilogue epi;
};

// OUT_IN: W's unit stride is along K, a warp takes four features at a time with its
// lanes along K; else lanes are along the features and warps along K.
template <int TT, bool OUT_IN>
__global__ void __launch_bounds__(32 * GF_WARPS) gemm_few_kernel(const GfParams p) {
  extern __shared__ __align__(16) float part[];  // [t][128] sums (else [warp][t][128]), then X: OUT_IN [t][kn], else [k][t]
  wait_for_prior_kernel();
  float* xs = part + (OUT_IN ? 1 : GF_WARPS) * TT * GR_FEATURES;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = p.splits > 1 ? cluster_ctarank() : 0;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) / p.splits * GR_FEATURES;
  const int64_t quads = (p.K + 3) / 4;  // runs of K start on 16 bytes
  const int64_t k0 = quads * rank / p.splits * 4, k1 = quads * (rank + 1) / p.splits * 4;
  const int kn = static_cast<int>((k1 < p.K ? k1 : p.K) - k0), kp = (kn + 3) & ~3;
  for (int i = threadIdx.x; i < TT * kp; i += 32 * GF_WARPS) {
    const int t = i / kp, k = i - t * kp;
    xs[OUT_IN ? i : k * TT + t] = t < p.T && k < kn ? p.x[t * p.ldx + k0 + k] : 0.0f;
  }
  __syncthreads();
  if constexpr (OUT_IN) {
    constexpr int F = 4, kWarpFeatures = GR_FEATURES / GF_WARPS;
    for (int g = 0; g < kWarpFeatures / F; ++g) {
      const int64_t n = n0 + w * kWarpFeatures + g * F;
      const float* src[F];  // features past N read the last one
#pragma unroll
      for (int f = 0; f < F; ++f) src[f] = p.w + (n + f < p.N ? n + f : p.N - 1) * p.ldw + k0;
      float acc[F][TT];
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[f][t] = 0.0f;
      auto add = [&](const float4(&q)[F], int k) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const float4 y = *reinterpret_cast<const float4*>(xs + t * kp + k);
#pragma unroll
          for (int f = 0; f < F; ++f)
            acc[f][t] = fmaf(q[f].x, y.x, fmaf(q[f].y, y.y, fmaf(q[f].z, y.z, fmaf(q[f].w, y.w, acc[f][t]))));
        }
      };
      int k = lane * 4;
      for (; k + 128 + 4 <= kn; k += 256) {  // two runs of each feature in flight
        float4 q[2][F];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int f = 0; f < F; ++f) q[u][f] = *reinterpret_cast<const float4*>(src[f] + k + u * 128);
        add(q[0], k);
        add(q[1], k + 128);
      }
      for (; k < kn; k += 128) {
        float4 q[F];
#pragma unroll
        for (int f = 0; f < F; ++f) {
          if (k + 4 <= kn) {
            q[f] = *reinterpret_cast<const float4*>(src[f] + k);
          } else {  // the end of K
            q[f].x = src[f][k];
            q[f].y = k + 1 < kn ? src[f][k + 1] : 0.0f;
            q[f].z = k + 2 < kn ? src[f][k + 2] : 0.0f;
            q[f].w = 0.0f;
          }
        }
        add(q, k);
      }
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) acc[f][t] += __shfl_xor_sync(0xffffffffu, acc[f][t], o);
          if (lane == 0) part[t * GR_FEATURES + w * kWarpFeatures + g * F + f] = acc[f][t];
        }
    }
  } else {
    constexpr int U = 8;  // loads in flight
    const int64_t col = n0 + lane * 4;
    float acc[TT][4];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
    const float* src = p.w + k0 * p.ldw + col;
    for (int k = w; k < kn && col < p.N; k += GF_WARPS * U) {
      float4 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kk = k + u * GF_WARPS;
        const float* a = src + kk * p.ldw;
        if (kk < kn) {
          if (col + 4 <= p.N) {
            q[u] = *reinterpret_cast<const float4*>(a);
          } else {
            q[u].x = a[0];
            q[u].y = col + 1 < p.N ? a[1] : 0.0f;
            q[u].z = col + 2 < p.N ? a[2] : 0.0f;
            q[u].w = 0.0f;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kk = k + u * GF_WARPS;
        if (kk >= kn) continue;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const float x = xs[kk * TT + t];
          acc[t][0] = fmaf(q[u].x, x, acc[t][0]);
          acc[t][1] = fmaf(q[u].y, x, acc[t][1]);
          acc[t][2] = fmaf(q[u].z, x, acc[t][2]);
          acc[t][3] = fmaf(q[u].w, x, acc[t][3]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
      *reinterpret_cast<float4*>(part + (w * TT + t) * GR_FEATURES + lane * 4) =
          make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
    for (int i = threadIdx.x; i < TT * GR_FEATURES; i += 32 * GF_WARPS) {
      float a = 0.0f;
#pragma unroll
      for (int q = 0; q < GF_WARPS; ++q) a += part[q * TT * GR_FEATURES + i];
      part[i] = a;  // warp 0's part, read and written by this thread alone
    }
  }
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  rows_join(p.epi, smem_u32(part), rank, p.splits, 0, static_cast<int>(p.T), n0, p.N);
  if (p.splits > 1) cluster_sync();
}

// ------------------------------------------------------------------ host

struct GrPlan {
  int bn, t_tiles, n_tiles, k_tiles, splits, stages;
  size_t shared;
  double cost;  // microseconds
};
constexpr int64_t kSms = 152;
constexpr int GR_SHARED_TWO = 106 << 10, GR_SHARED_ONE = 212 << 10;  // of a CTA, two or one on an SM
constexpr int GR_SHARED_MOST = 227 << 10;

// The tile's tokens, the split of K and the stages.  Tiles of up to 64 tokens
// leave room for two CTAs on an SM.  The split (powers of two, up to a portable
// cluster) is the one whose time, in microseconds, is least:
//   start and join of a CTA, its K tiles in turn or the reading of W at the
//   copy's rate, whichever is longer, and what further waves of clusters add.
// Fitted to calls of 1 to 512 tokens with K and N from 1024 to 14336, which it
// gives within about 20 %.  With (K, N) = (14336, 4096), (4096, 14336) and
// (4096, 1024), 1 token takes 78, 27, 25 us with one run, 42, 23, 15 with 2, 25, 26, 10 with 4 and
// 23, 32, 7.5 with 8, where reading W takes 17.3, 17.3 and 1.2 us.
double tile_us(int bn) { return 0.32 + 0.0003 * bn; }
double start_us(int bn, int s) { return 5.5 + 0.005 * bn + 0.012 * bn / s; }
// More warps drain and add up a wider tile: with 192, 320 and 576 threads 256
// tokens through 4096 x 4096 take 18.6, 17.4 and 16.8 us in bf16 and 16.1, 14.8 and 13.6 in
// e4m3; 64 tokens through 4096 x 14336 26.0 and 25.4, one token 22.9 and 23.1 (two
// CTAs an SM have registers for 320 each).
int threads_of(int bn) { return bn > 64 ? GR_MOST_THREADS : bn > 32 ? 320 : GR_THREADS; }
constexpr double kWaveUs = 3.0;        // a further wave where memory bounds the call
constexpr double kBytesPerUs = 6.776e6;
// K tiles of one accumulator of planes: the tensor cores cut each partial sum
// where fp32 would round it, so that chains stay as short as the drains of
// gemm_tc2.cu (T2_SUB).
constexpr int64_t kPlaneRun = 8;
// Clusters of s CTAs that the device holds at once with one CTA on an SM, by
// what CUDA says of the kernel: an SM group holds whole clusters only (on
// a GB300 76, 36 and 15 of 2, 4 and 8).  Where CUDA does not say it, the SMs
// divided by s, for this call.
int64_t clusters_at_once(int s) {
  static PerDevice<bool> ready;
  static PerDevice<int> known[GR_MAX_SPLIT + 1];
  int n = 0;
  if (on_this_device(known[s], &n, [s](int* m) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(s), 1, 1);
        cfg.blockDim = dim3(GR_THREADS, 1, 1);
        cfg.dynamicSmemBytes = GR_SHARED_ONE;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(s);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return allow_shared(ready, gemm_rows_kernel<false, false, GR_BF16>, GR_SHARED_MOST) &&
               cudaOccupancyMaxActiveClusters(m, gemm_rows_kernel<false, false, GR_BF16>, &cfg) == cudaSuccess && *m > 0;
      }))
    return n;
  cudaGetLastError();
  return kSms / s;
}
GrPlan plan_of(const GemmDesc& g) {
  GrPlan r;
  r.t_tiles = static_cast<int>((g.M + GR_TOKENS - 1) / GR_TOKENS);
  const int64_t unit = g.a_sk == 1 ? 16 : 64;  // boxes of 64 rows where X's unit stride is along them
  r.bn = static_cast<int>(((g.M + r.t_tiles - 1) / r.t_tiles + unit - 1) / unit * unit);
  r.n_tiles = static_cast<int>((g.N + GR_FEATURES - 1) / GR_FEATURES);
  const int bk = g.in_dtype == TPS_E4M3 ? 128 : 64;
  r.k_tiles = static_cast<int>((g.K + bk - 1) / bk);
  const int64_t products = g.planes > 1 ? 6 : 1;
  const int64_t per_sm = r.bn <= 64 ? 2 : 1, tiles = int64_t(r.t_tiles) * r.n_tiles;
  r.splits = 1;
  r.cost = -1.0;
  for (int s = 1; s <= GR_MAX_SPLIT && s <= r.k_tiles; s *= 2) {
    const int64_t run = (r.k_tiles + s - 1) / s;
    if (products > 1 && run > kPlaneRun && 2 * s <= GR_MAX_SPLIT && 2 * s <= r.k_tiles) continue;
    const int64_t clusters = clusters_at_once(s) * per_sm;
    const double w_us = double(g.N) * double(g.K) * (g.in_dtype == TPS_E4M3 ? 1.0 : 2.0 * double(g.planes)) / kBytesPerUs;
    const double own = double(run * products) * tile_us(r.bn);
    double cost;
    if (per_sm > 1) {  // two CTAs share an SM: waves run into each other
      const double waves = tiles > clusters ? double(tiles) / double(clusters) : 1.0;
      cost = start_us(r.bn, s) + (waves * own > w_us ? waves * own : w_us) + (waves - 1.0) * kWaveUs;
    } else {
      const double waves = double((tiles + clusters - 1) / clusters), all = waves * (start_us(r.bn, s) + own);
      cost = all > w_us ? all : w_us;
    }
    if (r.cost < 0.0 || cost < r.cost) {
      r.cost = cost;
      r.splits = s;
    }
  }
  const int stage = GR_W_BYTES + r.bn * 128;
  const int budget = (per_sm == 2 ? GR_SHARED_TWO : GR_SHARED_ONE) - 2048;
  r.stages = budget / stage < GR_MAX_STAGES ? budget / stage : GR_MAX_STAGES;
  r.shared = 1024 + static_cast<size_t>(r.stages) * stage + sizeof(GrBarriers);
  return r;
}

template <bool W_MN, bool X_MN, int KIND>
int launch_typed(const GemmDesc& g, const CUtensorMap& tw, const CUtensorMap& tx, const GrParams& p, const GrPlan& plan,
                 cudaStream_t stream) {
  static PerDevice<bool> ready;
  if (!allow_shared(ready, gemm_rows_kernel<W_MN, X_MN, KIND>, GR_SHARED_MOST)) return TPS_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.t_tiles * plan.n_tiles * plan.splits), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads_of(plan.bn)), 1, 1);
  cfg.dynamicSmemBytes = plan.shared;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(plan.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = early_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ProfScope prof("gemm_rows", g.name, 2.0 * double(g.M) * double(g.N) * double(g.K) * (KIND == GR_PLANES ? 6.0 : 1.0),
                 double(g.K) * double(g.N) * (KIND == GR_CODES ? 1.0 : 2.0), stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_rows_kernel<W_MN, X_MN, KIND>, tw, tx, p);
  note_launch();
  return e == cudaSuccess ? TPS_OK : TPS_ERR_CUDA;
}

}  // namespace

// fp32 rows of X and W's rows in either layout, 16-byte aligned.
bool gemm_few_supported(const GemmDesc& g) {
  if (g.in_dtype != TPS_F32 || g.M < 1 || g.M > GF_ROWS || g.N < 1 || g.K < 1) return false;
  if (g.epi.mode != EPI_LINEAR && g.epi.mode != EPI_STORE) return false;
  if (g.epi.accumulate || g.epi.alpha != nullptr || g.kparts > 1 || g.n_segs > 1 || g.K2 > 0 || g.K3 > 0 || g.planes > 1)
    return false;
  const int64_t ldw = g.b_sk == 1 ? g.b_sn : g.b_sk;
  if (g.a_sk != 1 || (g.b_sk != 1 && g.b_sn != 1) || ldw % 4 != 0 || (reinterpret_cast<uintptr_t>(g.b) & 15u) != 0) return false;
  const int64_t tt = g.M <= 1 ? 1 : g.M <= 2 ? 2 : g.M <= 4 ? 4 : 8;
  return tt * ((g.K + GR_MAX_SPLIT - 1) / GR_MAX_SPLIT + 8) * 4 <= GF_SHARED;
}

template <int TT, bool OUT_IN>
static int launch_few(const GemmDesc& g, const GfParams& p, cudaStream_t stream) {
  static PerDevice<bool> ready;
  if (!allow_shared(ready, gemm_few_kernel<TT, OUT_IN>, GF_SHARED + 4 * GF_WARPS * GF_ROWS * GR_FEATURES)) return TPS_ERR_CUDA;
  const int64_t run = ((p.K + 3) / 4 + p.splits - 1) / p.splits * 4;
  const int64_t floats = TT * run + (OUT_IN ? 1 : GF_WARPS) * TT * GR_FEATURES;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + GR_FEATURES - 1) / GR_FEATURES * p.splits), 1, 1);
  cfg.blockDim = dim3(32 * GF_WARPS, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(4 * floats);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = early_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ProfScope prof("gemm_few", g.name, 2.0 * double(p.T) * double(p.N) * double(p.K), 4.0 * double(p.K) * double(p.N), stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_few_kernel<TT, OUT_IN>, p);
  note_launch();
  return e == cudaSuccess ? TPS_OK : TPS_ERR_CUDA;
}

int launch_gemm_few(const GemmDesc& g, cudaStream_t stream) {
  GfParams p;
  p.x = static_cast<const float*>(g.a);
  p.ldx = g.a_sm;
  p.w = static_cast<const float*>(g.b);
  const bool out_in = g.b_sk == 1;
  p.ldw = out_in ? g.b_sn : g.b_sk;
  p.T = g.M;
  p.N = g.N;
  p.K = g.K;
  p.epi = g.epi;
  // Enough blocks for four on every SM, as far as a cluster goes; every run holds some of K.
  const int64_t tiles = (g.N + GR_FEATURES - 1) / GR_FEATURES;
  p.splits = 1;
  while (p.splits < GR_MAX_SPLIT && tiles * p.splits < 4 * kSms && (g.K + 3) / 4 >= 2 * p.splits) p.splits *= 2;
  const int64_t tt = g.M <= 1 ? 1 : g.M <= 2 ? 2 : g.M <= 4 ? 4 : 8;
  while (p.splits < GR_MAX_SPLIT && tt * (((g.K + 3) / 4 + p.splits - 1) / p.splits * 4) * 4 > GF_SHARED) p.splits *= 2;
  if (tiles * p.splits >= (1ll << 31)) return TPS_ERR_SHAPE;
  if (g.M <= 1) return out_in ? launch_few<1, true>(g, p, stream) : launch_few<1, false>(g, p, stream);
  if (g.M <= 2) return out_in ? launch_few<2, true>(g, p, stream) : launch_few<2, false>(g, p, stream);
  if (g.M <= 4) return out_in ? launch_few<4, true>(g, p, stream) : launch_few<4, false>(g, p, stream);
  return out_in ? launch_few<8, true>(g, p, stream) : launch_few<8, false>(g, p, stream);
}

// X K-major, or both operands the other way; everything else as the CTA-pair kernel wants it.
bool gemm_rows_supported(const GemmDesc& g) {
  if (g.epi.mode != EPI_LINEAR && g.epi.mode != EPI_STORE) return false;
  if (g.n_segs > 1 || g.K2 > 0 || g.K3 > 0 || g.epi.accumulate || g.epi.alpha != nullptr || g.kparts > 1) return false;
  if (g.a_sk != 1 && (g.a_sm != 1 || g.b_sk == 1)) return false;
  if (g.planes == 1 && (g.a_cols > 0 || g.b_cols > 0)) return false;
  if (g.in_dtype == TPS_E4M3 && g.epi.mode != EPI_LINEAR) return false;
  if (!gemm_tc_supported(g)) return false;
  const GrPlan r = plan_of(g);
  if (g.planes > 1 && (r.k_tiles + r.splits - 1) / r.splits > kPlaneRun) return false;
  return int64_t(r.t_tiles) * r.n_tiles * r.splits < (1ll << 31);
}

// By what either kernel takes: a pair tile's K tile costs 0.31 us, whatever
// fills its 256 x 256.  Measured (us, this kernel / pairs, bf16, 256, 512 and 1024
// tokens): K = 14336, N = 4096: 33 / 72, 51 / 72, 88 / 74; K = 4096, N = 4096: 17 / 26, 22 / 26,
// 33 / 27; K = 4096, N = 14336: 37 / 31, 65 / 48, 99 / 70; K = 1024, N = 4096: 11.4 / 11.9, 13.4 /
// 12.1, 16.9 / 12.6.
// TPS_LINEAR_ROWS=n takes this kernel for up to n rows and no others.
bool gemm_rows_preferred(const GemmDesc& g) {
  const char* most = getenv("TPS_LINEAR_ROWS");
  if (most != nullptr) return g.M <= atoll(most);
  const GrPlan r = plan_of(g);
  const int64_t waves = (pair_tile_count(g.M, g.N) + kSms / 2 - 1) / (kSms / 2);
  return r.cost < 6.0 + 0.31 * double(waves) * double(r.k_tiles) * (g.planes > 1 ? 6.0 : 1.0);
}

int launch_gemm_rows(const GemmDesc& g, uint32_t* dev_err, cudaStream_t stream) {
  const bool w_mn = g.b_sk != 1, x_mn = g.a_sk != 1, codes = g.in_dtype == TPS_E4M3, planes = g.planes > 1;
  const GrPlan plan = plan_of(g);
  CUtensorMap tw, tx;
  bool ok;
  if (codes) {
    ok = !w_mn && tc_make_map8(&tw, g.b, g.N, g.K, g.b_sn, 128, GR_FEATURES) &&
         tc_make_map8(&tx, g.a, g.M, g.K, g.a_sm, 128, plan.bn);
  } else {
    const int64_t w_cols = planes ? g.b_cols : w_mn ? g.N : g.K, x_cols = planes ? g.a_cols : x_mn ? g.M : g.K;
    ok = (w_mn ? tc_make_map(&tw, g.b, g.K, w_cols, g.b_sk, 64, TC_BK)
               : tc_make_map(&tw, g.b, g.N, w_cols, g.b_sn, TC_BK, GR_FEATURES)) &&
         (x_mn ? tc_make_map(&tx, g.a, g.K, x_cols, g.a_sk, 64, TC_BK) : tc_make_map(&tx, g.a, g.M, x_cols, g.a_sm, TC_BK, plan.bn));
  }
  if (!ok) return TPS_ERR_CUDA;
  GrParams p;
  p.T = static_cast<int>(g.M);
  p.N = static_cast<int>(g.N);
  p.k_tiles = plan.k_tiles;
  p.bn = plan.bn;
  p.t_tiles = plan.t_tiles;
  p.stages = plan.stages;
  p.splits = plan.splits;
  p.x_plane = static_cast<int>(g.a_plane);
  p.w_plane = static_cast<int>(g.b_plane);
  p.tmem_cols = 32;
  while (p.tmem_cols < static_cast<uint32_t>(plan.bn)) p.tmem_cols *= 2;
  if (planes) p.tmem_cols *= 2;
  p.epi = g.epi;
  p.err = dev_err;
  if (codes) return launch_typed<false, false, GR_CODES>(g, tw, tx, p, plan, stream);
  if (planes)
    return x_mn   ? launch_typed<true, true, GR_PLANES>(g, tw, tx, p, plan, stream)
           : w_mn ? launch_typed<true, false, GR_PLANES>(g, tw, tx, p, plan, stream)
                  : launch_typed<false, false, GR_PLANES>(g, tw, tx, p, plan, stream);
  return x_mn   ? launch_typed<true, true, GR_BF16>(g, tw, tx, p, plan, stream)
         : w_mn ? launch_typed<true, false, GR_BF16>(g, tw, tx, p, plan, stream)
                : launch_typed<false, false, GR_BF16>(g, tw, tx, p, plan, stream);
}

}  // namespace tps
