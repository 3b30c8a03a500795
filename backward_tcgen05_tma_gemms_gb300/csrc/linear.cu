// linear.cu -- matrix product with bias, activation and residual in its
// epilogue, and its gradients.
//
//   z = x W + b,  y = act(z) + residual          (e4m3: z = s_x s_w (x W) + b)
//   dz = dy act'(z),  dx = dz W^T,  dW = x^T dz,  db = sum over the rows of dz
//
// Forward.  bf16 and e4m3: CTA pairs on 256 x 256 tiles (T2_LIN, T2_LIN8 of
// gemm_tc2.cu), or, for few rows, the split over K of gemm_rows.cu.  fp32: up to
// eight rows on the fp32 pipes (gemm_rows.cu), else as three bf16 planes a
// value on the tensor cores (T2_PLANES_LIN).  The epilogue works on the fp32
// accumulator: z is rounded once, where it is kept, and y once.
//
// Backward.  One pass over dy and z forms dz in the operands' type and the
// sums of its columns (fp32, of dz before its rounding); the two products then
// read dz.  Without an activation dz is dy itself, where it has the operands'
// type, and only the sums are formed.  For bf16 operands dz is bf16, whatever
// the types of dy and of the gradients, for the tensor cores take both operands
// of one type and a second plane of dz would double the products.  Each term is
// off by up to 2^-8 of itself, with either sign: 8192 x 4096 x 14336 gives bf16
// gradients 2.3e-3 off where an fp32 dz gives 1.7e-3, which is their own
// rounding.  fp32 operands have an fp32 dz.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "api_common.cuh"
#include "epilogue.cuh"
#include "operand.cuh"
#include "ptx.cuh"
#include "rows.cuh"
#include "rows_host.cuh"

namespace tps {

namespace {

constexpr int64_t kParts = 256;  // partial sums of a column of dz at most
constexpr int kDzRows = 8;       // rows of a block at a time

struct DzParams {
  Rows dy, z, dz;  // p of z: nullptr without activation; p of dz: nullptr when dy serves
  float* part;     // [gridDim.y][N], or nullptr
  int64_t T, N;
  int act;
};

// A run of N elements in flight, of type T or (void) of the type that the tensor
// has at run time.
template <class T, int N>
struct DzRun {
  Typed<T, N> t;
  __device__ __forceinline__ void load(const Rows& m, int64_t r, int64_t c) { t.load(reinterpret_cast<const T*>(m.p) + r * m.ld + c); }
  __device__ __forceinline__ void value(const Rows&, float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = t.at(i);
  }
};
template <int N>
struct DzRun<void, N> {
  Raw<N> t;
  __device__ __forceinline__ void load(const Rows& m, int64_t r, int64_t c) { raw_load(m.at(r, c), m.dtype, t); }
  __device__ __forceinline__ void value(const Rows& m, float (&v)[N]) const { raw_value(t, m.dtype, v); }
};

// A warp takes 32 runs of N elements of a row, a block eight rows at a time, every
// gridDim.y-th group of eight; the columns' sums stay in registers.  Some 25
// instructions an element with an activation (two of them on the special function
// unit), nearly the time that memory takes: the activation is a type, and so is
// that of the tensors where they share one; four blocks an SM leave loads in
// flight.
template <class T, int N, int ACT>
__global__ void __launch_bounds__(32 * kDzRows, 4) linear_dz_kernel(const DzParams p) {
  __shared__ float sums[kDzRows][32 * N + 1];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 32 * N, c = c0 + lane * N;
  float s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0.0f;
  constexpr int U = 2;  // rows whose loads are in flight
  const int64_t step = static_cast<int64_t>(gridDim.y) * kDzRows;
  if (c < p.N) {
    for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * kDzRows + w; r0 < p.T; r0 += U * step) {
      DzRun<T, N> a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u * step;
        if (r < p.T) {
          a[u].load(p.dy, r, c);
          if (ACT != kActNone) b[u].load(p.z, r, c);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u * step;
        if (r >= p.T) continue;
        float v[N];
        a[u].value(p.dy, v);
        if constexpr (ACT != kActNone) {
          float z[N];
          b[u].value(p.z, z);
#pragma unroll
          for (int i = 0; i < N; ++i) v[i] *= linear_slope_c<ACT>(z[i]);
        }
        if (p.dz.p != nullptr) {
          if constexpr (std::is_void_v<T>) {
            run_store(p.dz.at(r, c), p.dz.dtype, v);
          } else {
            Typed<T, N> o;
            o.set(v);
            o.store(reinterpret_cast<T*>(p.dz.p) + r * p.dz.ld + c);
          }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += v[i];
      }
    }
  }
  if (p.part == nullptr) return;
  let_next_kernel_start();
#pragma unroll
  for (int i = 0; i < N; ++i) sums[w][lane * N + i] = s[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * N; i += 32 * kDzRows) {
    if (c0 + i >= p.N) continue;
    float t = 0.0f;
#pragma unroll
    for (int q = 0; q < kDzRows; ++q) t += sums[q][i];
    p.part[static_cast<int64_t>(blockIdx.y) * p.N + c0 + i] = t;
  }
}
template <class T, int N>
void launch_dz_act(const DzParams& p, dim3 grid, cudaStream_t s) {
  switch (p.act) {
    case TPS_ACT_GELU_ERF: linear_dz_kernel<T, N, TPS_ACT_GELU_ERF><<<grid, 32 * kDzRows, 0, s>>>(p); break;
    case TPS_ACT_GELU_TANH: linear_dz_kernel<T, N, TPS_ACT_GELU_TANH><<<grid, 32 * kDzRows, 0, s>>>(p); break;
    case TPS_ACT_TANH: linear_dz_kernel<T, N, TPS_ACT_TANH><<<grid, 32 * kDzRows, 0, s>>>(p); break;
    case TPS_ACT_SILU: linear_dz_kernel<T, N, TPS_ACT_SILU><<<grid, 32 * kDzRows, 0, s>>>(p); break;
    default: linear_dz_kernel<T, N, kActNone><<<grid, 32 * kDzRows, 0, s>>>(p); break;
  }
}
template <int N>
void launch_dz(const DzParams& p, dim3 grid, cudaStream_t s) {
  const int t = p.dy.dtype;
  const bool one = (p.z.p == nullptr || p.z.dtype == t) && (p.dz.p == nullptr || p.dz.dtype == t);
  if (one && t == TPS_BF16)
    launch_dz_act<__nv_bfloat16, N>(p, grid, s);
  else if (one)
    launch_dz_act<float, N>(p, grid, s);
  else
    launch_dz_act<void, N>(p, grid, s);
}

// ------------------------------------------------------------------ host

struct Linear {  // what both directions check alike
  Mat x, w;
  int64_t T = 0, K = 0, N = 0, w_in = 0, w_out = 0;
  int dt = 0;
};

int check_linear(const tps_tensor* X, const tps_tensor* W, int32_t act, int32_t layout, bool codes, Linear* c) {
  int rc;
  if ((rc = as_mat(X, "X", true, &c->x)) || (rc = as_mat(W, "W", false, &c->w))) return rc;
  if (layout != TPS_W_IN_OUT && layout != TPS_W_OUT_IN) return fail(TPS_ERR_ARG, "unknown weight layout %d", layout);
  if (act != TPS_ACT_NONE && act != TPS_ACT_GELU_ERF && act != TPS_ACT_GELU_TANH && act != TPS_ACT_TANH && act != TPS_ACT_SILU)
    return fail(TPS_ERR_ARG, "unknown activation %d", act);
  const bool io = layout == TPS_W_IN_OUT;
  c->T = c->x.rows;
  c->K = c->x.cols;
  c->N = io ? c->w.cols : c->w.rows;
  if ((io ? c->w.rows : c->w.cols) != c->K) return fail(TPS_ERR_SHAPE, "W does not match X's width %lld", (long long)c->K);
  if (c->K < 1 || c->N < 1) return fail(TPS_ERR_SHAPE, "empty width");
  c->dt = c->x.dtype;
  if (c->w.dtype != c->dt) return fail(TPS_ERR_DTYPE, "X and W must share a type");
  if (c->dt != TPS_F32 && c->dt != TPS_BF16 && !(codes && c->dt == TPS_E4M3))
    return fail(TPS_ERR_DTYPE, codes ? "X and W must be f32, bf16 or e4m3" : "X and W must be f32 or bf16");
  const int64_t most = c->dt == TPS_F32 ? 1ll << 29 : 1ll << 31;  // three planes side by side stay below 2^31
  if (c->T >= most || c->K >= most || c->N >= most) return fail(TPS_ERR_SHAPE, "an extent of 2^%d or more", c->dt == TPS_F32 ? 29 : 31);
  for (const Mat* m : {&c->x, &c->w}) {
    if (reinterpret_cast<uintptr_t>(m->data) % es_of(m->dtype) != 0) return fail(TPS_ERR_LAYOUT, "misaligned data");
    if (m->sr < 0 || m->sc < 0) return fail(TPS_ERR_LAYOUT, "negative stride");
  }
  weight_strides(c->w, layout, &c->w_in, &c->w_out);
  return TPS_OK;
}

// Operands as the tensor cores take them.
struct Room {  // of a workspace
  char* p;
  size_t at;
  char* take(int64_t bytes) {
    char* q = p + at;
    at += align256(static_cast<size_t>(bytes));
    return q;
  }
};
// Operands that are laid out, all in one launch (fp32, 500 x 1024 by 1024 x 4100: the
// call takes 41.0 us, 44.7 with a launch for each; in a CUDA graph 38.6 and 40.7).
struct Lay {
  int dt;
  Room* room;
  LayJob jobs[kLayJobs];
  int n = 0;
  Operand operand(const void* p, int64_t ni, int64_t nj, int64_t si, int64_t sj, bool direct) {
    if (direct) return Operand{static_cast<const char*>(p), si, sj, 0, 0};
    Operand o;
    lay_job(dt, static_cast<const char*>(p), ni, nj, si, sj, room->take(laid_bytes(ni, nj, dt == TPS_F32 ? 3 : 1)), &jobs[n++], &o);
    if (dt != TPS_F32) o.plane = o.cols = 0;  // rows like any others
    return o;
  }
  int launch(cudaStream_t s) const { return launch_lay(dt, jobs, n, "linear", s); }
};
// bf16 that TMA can describe as it is (pitches as its maps want them).
bool direct_of(const void* p, int64_t ni, int64_t nj, int64_t si, int64_t sj) {
  if (!tma_can(p, si, sj)) return false;
  const int64_t outer = sj == 1 ? si : sj, inner = sj == 1 ? nj : ni;
  return outer >= inner && outer * 2 < (1ll << 40);
}
GemmDesc linear_gemm(const char* name, int dt, int64_t M, int64_t N, int64_t K) {
  GemmDesc g;
  g.name = name;
  g.M = M; g.N = N; g.K = K;
  g.in_dtype = dt == TPS_F32 ? TPS_BF16 : dt;
  g.planes = dt == TPS_F32 ? 3 : 1;
  return g;
}
int run_linear(const GemmDesc& g, int64_t d_sm, int64_t d_sn, cudaStream_t s) {
  if (d_sn == 1 && gemm_rows_supported(g) && gemm_rows_preferred(g)) {
    uint32_t* err = device_error_word();
    if (err == nullptr) return fail(TPS_ERR_CUDA, "cannot resolve the device error word");
    GemmDesc t = g;
    t.epi.ldd = d_sm;
    t.epi.dbg_rows = g.M;
    t.epi.dbg_cols = g.N;
    t.epi.dbg_err = err;
    const int rc = launch_gemm_rows(t, err, s);
    return rc == TPS_ERR_CUDA ? fail(rc, "%s: launch failed: %s", g.name, cudaGetErrorString(cudaGetLastError())) : rc;
  }
  return run_gemm(g, d_sm, d_sn, s);
}
int run_few(GemmDesc g, int64_t d_sm, cudaStream_t s) {
  g.in_dtype = TPS_F32;
  g.planes = 1;
  g.epi.ldd = d_sm;
  g.epi.dbg_rows = g.M;
  g.epi.dbg_cols = g.N;
  g.epi.dbg_err = device_error_word();
  const int rc = launch_gemm_few(g, s);
  return rc == TPS_ERR_CUDA ? fail(rc, "%s: launch failed: %s", g.name, cudaGetErrorString(cudaGetLastError())) : rc;
}

// The six products of fp32 planes go through one count of K tiles.
int contraction(int dt, int64_t K) {
  return dt == TPS_F32 && 6 * K >= (1ll << 31) ? fail(TPS_ERR_SHAPE, "a contraction over 2^31 / 6 or more in fp32") : TPS_OK;
}
int need_room(const void* workspace, size_t bytes, size_t need) {
  if (need > 0 && (workspace == nullptr || bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255)))
    return fail(TPS_ERR_WORKSPACE, "workspace needs %zu bytes, 256-byte aligned", need);
  return TPS_OK;
}

}  // namespace

}  // namespace tps

using namespace tps;

extern "C" size_t tps_linear_workspace_bytes(int64_t T, int64_t K, int64_t N, int32_t dtype, int32_t backward) {
  if (T < 0 || K < 1 || N < 1) return 0;
  const int planes = dtype == TPS_F32 ? 3 : 1, es = dtype == TPS_F32 ? 4 : 2;
  size_t n = 0;
  if (dtype == TPS_F32) {
    n += align256(laid_bytes(T, K, planes)) + align256(laid_bytes(K, N, planes));
    if (backward) n += align256(laid_bytes(T, N, planes));
  }
  if (backward) n += align256(es * T * round_up(N, 8)) + align256(4 * kParts * N);
  return n;
}

extern "C" int tps_linear_fwd(const tps_tensor* X, const tps_tensor* W, const tps_tensor* bias,
                              const tps_tensor* residual, int32_t act, int32_t weight_layout,
                              const tps_tensor* x_scale, const tps_tensor* w_scale, const tps_tensor* Z,
                              const tps_tensor* Y, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  clear_detail();
  Linear c;
  int rc;
  if ((rc = check_linear(X, W, act, weight_layout, true, &c))) return rc;
  const bool codes = c.dt == TPS_E4M3;
  if (codes && weight_layout != TPS_W_OUT_IN) return fail(TPS_ERR_LAYOUT, "e4m3 weights are (out, in)");
  if (codes != (x_scale != nullptr) || codes != (w_scale != nullptr))
    return fail(TPS_ERR_ARG, "x_scale and w_scale go with e4m3 operands");
  if (codes && ((rc = aligned_vector(x_scale, "x_scale", TPS_F32, c.T)) || (rc = aligned_vector(w_scale, "w_scale", TPS_F32, c.N))))
    return rc;
  GemmDesc g = linear_gemm("linear", c.dt, c.T, c.N, c.K);
  g.epi.mode = EPI_LINEAR;
  g.epi.act = act;
  if (bias != nullptr) {
    const char* p;
    if ((rc = weight_vector(bias, c.N, &p, &g.epi.bias_dtype))) return rc;
    g.epi.bias = p;
  }
  Rows res = {}, y = {}, z = {};
  if (residual != nullptr && (rc = float_rows(residual, "residual", false, c.T, c.N, &res))) return rc;
  if ((rc = float_rows(Y, "Y", true, c.T, c.N, &y))) return rc;
  if (Z != nullptr && (rc = float_rows(Z, "Z", true, c.T, c.N, &z))) return rc;
  if (c.T == 0) return TPS_OK;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (codes) {
    g.epi.row_scale = static_cast<const float*>(x_scale->data);
    g.epi.col_scale = static_cast<const float*>(w_scale->data);
  }
  g.epi.res = res.p;
  g.epi.ld_res = res.ld;
  g.epi.res_dtype = res.dtype;
  g.epi.d = y.p;
  g.epi.d_dtype = y.dtype;
  g.epi.d2 = z.p;
  g.epi.ldd2 = z.ld;
  g.epi.d2_dtype = z.dtype;
  g.a = c.x.data; g.a_sm = c.x.sr; g.a_sk = c.x.sc;
  g.b = c.w.data; g.b_sk = c.w_in; g.b_sn = c.w_out;
  if (codes) {
    g.epi.ldd = y.ld;
    // a single row has no pitch: any that TMA can describe
    if (c.T == 1 && c.x.sc == 1) g.a_sm = round_up(c.K, 16);
    if (c.N == 1 && c.w.sc == 1) g.b_sn = round_up(c.K, 16);
    if (!gemm_tc_supported(g)) return fail(TPS_ERR_LAYOUT, "e4m3 operands need rows that start on 16 bytes and do not overlap");
    return run_linear(g, y.ld, 1, s);
  }
  if (c.dt == TPS_F32) {
    GemmDesc f = g;
    f.in_dtype = TPS_F32;
    f.planes = 1;
    if (gemm_few_supported(f)) return run_few(f, y.ld, s);
  }
  if ((rc = contraction(c.dt, c.K))) return rc;
  const bool bf16 = c.dt == TPS_BF16;
  const bool x_ok = bf16 && direct_of(g.a, c.T, c.K, c.x.sr, c.x.sc), w_ok = bf16 && direct_of(g.b, c.K, c.N, c.w_in, c.w_out);
  const int planes = bf16 ? 1 : 3;
  const size_t need = (x_ok ? 0 : align256(laid_bytes(c.T, c.K, planes))) + (w_ok ? 0 : align256(laid_bytes(c.K, c.N, planes)));
  if ((rc = need_room(workspace, workspace_bytes, need))) return rc;
  Room room{static_cast<char*>(workspace), 0};
  Lay lay{c.dt, &room};
  const Operand x = lay.operand(g.a, c.T, c.K, c.x.sr, c.x.sc, x_ok), w = lay.operand(g.b, c.K, c.N, c.w_in, c.w_out, w_ok);
  if ((rc = lay.launch(s))) return rc;
  set_a(&g, x, false);
  set_b(&g, w, false);
  return run_linear(g, y.ld, 1, s);
}

extern "C" int tps_linear_bwd(const tps_tensor* X, const tps_tensor* W, const tps_tensor* dY, const tps_tensor* Z,
                              int32_t act, int32_t weight_layout, const tps_tensor* dX, const tps_tensor* dW,
                              const tps_tensor* dbias, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  clear_detail();
  Linear c;
  int rc;
  if ((rc = check_linear(X, W, act, weight_layout, false, &c))) return rc;
  const bool acted = act != TPS_ACT_NONE, bf16 = c.dt == TPS_BF16;
  DzParams p = {};
  if ((rc = float_rows(dY, "dY", false, c.T, c.N, &p.dy))) return rc;
  if (acted != (Z != nullptr)) return fail(TPS_ERR_ARG, "Z goes with an activation");
  if (acted && (rc = float_rows(Z, "Z", false, c.T, c.N, &p.z))) return rc;
  Rows dx = {};
  Mat dw;
  if (dX != nullptr && (rc = float_rows(dX, "dX", true, c.T, c.K, &dx))) return rc;
  if (dW != nullptr) {
    if ((rc = as_mat(dW, "dW", false, &dw)) || (rc = expect(dw, "dW", c.w.rows, c.w.cols))) return rc;
    if (dw.dtype != TPS_F32 && dw.dtype != TPS_BF16) return fail(TPS_ERR_DTYPE, "dW must be f32 or bf16");
    const bool by_rows = dw.sc == 1;
    if ((by_rows ? dw.rows : dw.cols) > 1 && (by_rows ? dw.sr < dw.cols : dw.sc < dw.rows))
      return fail(TPS_ERR_LAYOUT, "dW: rows overlap");
    if (reinterpret_cast<uintptr_t>(dw.data) % es_of(dw.dtype) != 0) return fail(TPS_ERR_LAYOUT, "dW: misaligned data");
  }
  if (dbias != nullptr) {
    if (dbias->dtype != TPS_F32 && dbias->dtype != TPS_BF16) return fail(TPS_ERR_DTYPE, "dbias must be f32 or bf16");
    if ((rc = aligned_vector(dbias, "dbias", dbias->dtype, c.N))) return rc;
  }
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (c.T == 0) {  // sums of nothing
    if (dW != nullptr && (rc = launch_fill(dw.data, dw.dtype, dw.rows, dw.cols, dw.sr, dw.sc, s))) return rc;
    return dbias != nullptr ? launch_fill(dbias->data, dbias->dtype, 1, c.N, c.N, 1, s) : TPS_OK;
  }
  if (dX != nullptr && (rc = contraction(c.dt, c.N))) return rc;
  if (dW != nullptr && (rc = contraction(c.dt, c.T))) return rc;
  // dz: dy itself where nothing multiplies it and the products can read it
  const bool as_is = !acted && p.dy.dtype == c.dt && (!bf16 || direct_of(p.dy.p, c.T, c.N, p.dy.ld, 1));
  const bool products = dX != nullptr || dW != nullptr;
  const bool x_ok = bf16 && direct_of(c.x.data, c.T, c.K, c.x.sr, c.x.sc);
  const bool w_ok = bf16 && direct_of(c.w.data, c.K, c.N, c.w_in, c.w_out);
  const int planes = bf16 ? 1 : 3, es = bf16 ? 2 : 4;
  const int64_t ld = round_up(c.N, 8);
  size_t need = 0;
  if (products && !as_is) need += align256(es * c.T * ld);
  if (dbias != nullptr) need += align256(4 * kParts * c.N);
  if (products && !bf16) need += align256(laid_bytes(c.T, c.N, planes));
  if (dW != nullptr && !x_ok) need += align256(laid_bytes(c.T, c.K, planes));
  if (dX != nullptr && !w_ok) need += align256(laid_bytes(c.K, c.N, planes));
  if ((rc = need_room(workspace, workspace_bytes, need))) return rc;
  Room room{static_cast<char*>(workspace), 0};
  p.T = c.T;
  p.N = c.N;
  p.act = act;
  if (products && !as_is) p.dz = Rows{room.take(es * c.T * ld), ld, c.dt};
  if (dbias != nullptr) p.part = reinterpret_cast<float*>(room.take(4 * kParts * c.N));
  if (p.dz.p != nullptr || p.part != nullptr) {
    const bool wide = c.N % 8 == 0 && starts_runs(p.dy, c.T) && starts_runs(p.z, c.T) && starts_runs(p.dz, c.T);
    const int64_t gx = (c.N + (wide ? 256 : 32) - 1) / (wide ? 256 : 32), groups = (c.T + kDzRows - 1) / kDzRows;
    // four waves of four blocks an SM, as far as there are groups of rows
    int64_t gy = 152 * 16 / gx;
    if (gy > groups) gy = groups;
    if (gy > kParts) gy = kParts;
    if (gy < 1) gy = 1;
    ProfScope prof("linear_dz", "bwd", 0.0,
                   double(c.T) * double(c.N) * (es_of(p.dy.dtype) + (p.z.p ? es_of(p.z.dtype) : 0) + (p.dz.p ? es : 0)), s);
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
    wide ? launch_dz<8>(p, grid, s) : launch_dz<1>(p, grid, s);
    if ((rc = launched("linear_dz"))) return rc;
    if (p.part != nullptr && (rc = launch_sum_rows(p.part, gy, c.N, dbias->data, dbias->dtype, c.T < (1ll << 24) / c.N, s))) return rc;
  }
  if (!products) return TPS_OK;
  const Rows& src = p.dz.p != nullptr ? p.dz : p.dy;
  Lay lay{c.dt, &room};
  const Operand dz = lay.operand(src.p, c.T, c.N, src.ld, 1, bf16);
  Operand w, x;
  if (dX != nullptr) w = lay.operand(c.w.data, c.K, c.N, c.w_in, c.w_out, w_ok);
  if (dW != nullptr) x = lay.operand(c.x.data, c.T, c.K, c.x.sr, c.x.sc, x_ok);
  if ((rc = lay.launch(s))) return rc;
  if (dX != nullptr) {
    GemmDesc g = linear_gemm("linear_dX", c.dt, c.T, c.K, c.N);
    set_a(&g, dz, false);
    set_b(&g, w, true);
    g.epi.d = dx.p;
    g.epi.d_dtype = dx.dtype;
    if ((rc = run_linear(g, dx.ld, 1, s))) return rc;
  }
  if (dW != nullptr) {
    // rows of dW as it is stored: those of X's columns, or of dz's
    const bool io = weight_layout == TPS_W_IN_OUT;
    GemmDesc g = linear_gemm("linear_dW", c.dt, dw.rows, dw.cols, c.T);
    set_a(&g, io ? x : dz, true);
    set_b(&g, io ? dz : x, false);
    g.epi.d = dw.data;
    g.epi.d_dtype = dw.dtype;
    if ((rc = run_linear(g, dw.sr, dw.sc, s))) return rc;
  }
  return TPS_OK;
}
