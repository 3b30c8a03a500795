// dropout.cu -- dropout whose mask is computed where it is needed, from a
// counter-based generator (rows.cuh), and never stored; with the residual
// that it is added to.  The backward pass is the same product with the mask.
//
// Bound by memory: eight elements a thread and step, which share one call of
// the generator, with the loads of the next step issued before it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "api_common.cuh"
#include "rows.cuh"
#include "rows_host.cuh"

namespace tps {

namespace {

struct DropParams {
  Rows x, res, y;    // p of res: nullptr when absent
  int64_t rows, d;   // contiguous tensors are one row
  int64_t per_row;   // units of a row
  Dropout drop;
};

// One unit of N elements from column c of a row.
template <class TX, class TR, class TY, int N>
struct DropUnit {
  Typed<TX, N> x;
  Typed<TR, N> r;
  __device__ __forceinline__ void load(const DropParams& p, int64_t row, int64_t c) {
    x.load(reinterpret_cast<const TX*>(p.x.p) + row * p.x.ld + c);
    if (p.res.p != nullptr) r.load(reinterpret_cast<const TR*>(p.res.p) + row * p.res.ld + c);
  }
  __device__ __forceinline__ void finish(const DropParams& p, uint64_t key, int64_t row, int64_t c) const {
    float v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = x.at(j);
    if (p.drop.step != 0u) drop(p.drop, key, row * p.d + c, v);
    if (p.res.p != nullptr) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] += r.at(j);
    }
    Typed<TY, N> y;
    y.set(v);
    y.store(reinterpret_cast<TY*>(p.y.p) + row * p.y.ld + c);
  }
};

// Units of eight consecutive elements, the last one of a row perhaps shorter
// (FLAT: one row), or of one element (N = 1).  Two units of a thread are in
// flight together (8192 x 14336 in bf16: 84 us; four 87).  The generator and the
// masking take some hundred instructions a unit, two thirds of the time that
// memory takes.
constexpr int kUnits = 2;
template <class TX, class TR, class TY, int N, bool FLAT>
__global__ void __launch_bounds__(256) dropout_kernel(const DropParams p) {
  const uint64_t key = p.drop.step != 0u ? p.drop.key() : 0;
  const int64_t units = FLAT ? p.per_row : p.rows * p.per_row, step = int64_t(gridDim.x) * 256;
  auto row_of = [&](int64_t i) { return FLAT ? 0 : i / p.per_row; };
  const int64_t whole = FLAT ? p.d / N : units;  // FLAT: units before the end
  int64_t i = blockIdx.x * int64_t(256) + threadIdx.x;
  for (; i < whole; i += kUnits * step) {
    DropUnit<TX, TR, TY, N> a, b;
    const int64_t ra = row_of(i), ca = (i - ra * p.per_row) * N, j = i + step;
    a.load(p, ra, ca);
    if (j < whole) {
      const int64_t rb = row_of(j), cb = (j - rb * p.per_row) * N;
      b.load(p, rb, cb);
      a.finish(p, key, ra, ca);
      b.finish(p, key, rb, cb);
    } else {
      a.finish(p, key, ra, ca);
    }
  }
  if (FLAT && N > 1 && blockIdx.x == 0 && threadIdx.x < p.d - whole * N) {  // the end of the row
    const int64_t c = whole * N + threadIdx.x;
    DropUnit<TX, TR, TY, 1> a;
    a.load(p, 0, c);
    a.finish(p, key, 0, c);
  }
}

template <class TX, class TR, class TY>
void launch(const DropParams& p, bool wide, unsigned grid, cudaStream_t s) {
  if (wide && p.rows == 1)
    dropout_kernel<TX, TR, TY, 8, true><<<grid, 256, 0, s>>>(p);
  else if (wide)
    dropout_kernel<TX, TR, TY, 8, false><<<grid, 256, 0, s>>>(p);
  else
    dropout_kernel<TX, TR, TY, 1, false><<<grid, 256, 0, s>>>(p);
}
template <class TX, class TR>
void launch_y(const DropParams& p, bool wide, unsigned grid, cudaStream_t s) {
  if (p.y.dtype == TPS_F32)
    launch<TX, TR, float>(p, wide, grid, s);
  else
    launch<TX, TR, __nv_bfloat16>(p, wide, grid, s);
}

int dropout(const tps_tensor* X, const tps_tensor* residual, const tps_dropout* o, const tps_tensor* Y,
            const char* label, void* cuda_stream) {
  clear_detail();
  DropParams p = {};
  int64_t rows, d;
  int rc;
  if (o == nullptr) return fail(TPS_ERR_ARG, "dropout missing");
  if ((rc = rows_view(X, "X", false, &p.x, &rows, &d))) return rc;
  if (p.x.dtype == TPS_E4M3) return fail(TPS_ERR_DTYPE, "X must be f32 or bf16");
  if ((rc = too_large(rows, d))) return rc;
  if ((rc = dropout_of(o, &p.drop))) return rc;
  if (residual != nullptr && (rc = float_rows(residual, "residual", false, rows, d, &p.res))) return rc;
  if ((rc = float_rows(Y, "Y", true, rows, d, &p.y))) return rc;
  if (rows == 0 || d == 0) return TPS_OK;
  auto dense = [&](const Rows& r) { return r.p == nullptr || rows == 1 || r.ld == d; };
  p.rows = rows;
  p.d = d;
  if (dense(p.x) && dense(p.res) && dense(p.y)) {
    p.d = rows * d;
    p.rows = 1;
  }
  const bool wide = (p.rows == 1 || p.d % 8 == 0) && starts_runs(p.x, p.rows) && starts_runs(p.res, p.rows) &&
                    starts_runs(p.y, p.rows);
  p.per_row = wide ? (p.d + 7) / 8 : p.d;
  const int64_t units = p.rows * p.per_row, blocks = (units + 255) / 256;
  // Few units: one a thread.  Many: kUnits a thread at a time, up to eight times what the device holds.
  const int64_t most = 152 * 8 * 8, some = blocks < 152 * 8 ? blocks : (blocks + kUnits - 1) / kUnits;
  const unsigned grid = static_cast<unsigned>(some < most ? some : most);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  ProfScope prof("dropout", label, 0.0,
                 double(rows) * double(d) * (es_of(p.x.dtype) + (p.res.p ? es_of(p.res.dtype) : 0) + es_of(p.y.dtype)), s);
  using bf16 = __nv_bfloat16;
  const int tr = p.res.p != nullptr ? p.res.dtype : p.x.dtype;
  if (p.x.dtype == TPS_F32)
    tr == TPS_F32 ? launch_y<float, float>(p, wide, grid, s) : launch_y<float, bf16>(p, wide, grid, s);
  else
    tr == TPS_F32 ? launch_y<bf16, float>(p, wide, grid, s) : launch_y<bf16, bf16>(p, wide, grid, s);
  return launched("dropout");
}

}  // namespace

int dropout_of(const tps_dropout* o, Dropout* d) {
  *d = Dropout{};
  if (o == nullptr) return TPS_OK;
  if (!(o->p >= 0.0) || !(o->p <= 1.0)) return fail(TPS_ERR_ARG, "dropout must be in [0, 1]");
  if (reinterpret_cast<uintptr_t>(o->seed_ptr) % 8 != 0) return fail(TPS_ERR_LAYOUT, "seed: misaligned data");
  d->seed = o->seed;
  d->seed_ptr = o->seed_ptr;
  d->site = o->site;
  uint32_t k0 = static_cast<uint32_t>(o->seed), k1 = static_cast<uint32_t>(o->seed >> 32);
  for (int i = 0; i < 10; ++i) {
    d->keys[2 * i] = k0;
    d->keys[2 * i + 1] = k1;
    k0 += kPhiloxW0;
    k1 += kPhiloxW1;
  }
  d->step = static_cast<uint32_t>(std::nearbyint(o->p * 65536.0));
  d->below = (d->step << 16) - 1;  // all ones for a step of 65536, which nothing exceeds
  d->scale = d->step < 65536u ? static_cast<float>(65536.0 / (65536.0 - d->step)) : 0.0f;
  return TPS_OK;
}

}  // namespace tps

using namespace tps;

extern "C" int tps_dropout_fwd(const tps_tensor* X, const tps_tensor* residual, const tps_dropout* dropout_,
                               const tps_tensor* Y, void* cuda_stream) {
  return dropout(X, residual, dropout_, Y, "fwd", cuda_stream);
}

extern "C" int tps_dropout_bwd(const tps_tensor* dY, const tps_dropout* dropout_, const tps_tensor* dX,
                               void* cuda_stream) {
  return dropout(dY, nullptr, dropout_, dX, "bwd", cuda_stream);
}
