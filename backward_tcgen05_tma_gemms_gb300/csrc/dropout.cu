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

// Units of eight consecutive elements (N = 8), the last one of a row perhaps
// shorter, or of one element (N = 1).
template <int N>
__global__ void __launch_bounds__(256) dropout_kernel(const DropParams p) {
  const uint64_t key = p.drop.key();
  const int64_t units = p.rows * p.per_row;
  for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < units; i += int64_t(gridDim.x) * 256) {
    const int64_t row = p.rows == 1 ? 0 : i / p.per_row, c = (i - row * p.per_row) * N;
    if (N == 1 || c + N <= p.d) {
      Raw<N> x, r;
      raw_load(p.x.at(row, c), p.x.dtype, x);
      if (p.res.p != nullptr) raw_load(p.res.at(row, c), p.res.dtype, r);
      float v[N];
      raw_value(x, p.x.dtype, v);
      drop(p.drop, key, row * p.d + c, v);
      if (p.res.p != nullptr) {
        float q[N];
        raw_value(r, p.res.dtype, q);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] += q[j];
      }
      run_store(p.y.at(row, c), p.y.dtype, v);
    } else {  // the end of a single row
      for (int64_t e = c; e < p.d; ++e) {
        Raw<1> x;
        float v[1];
        raw_load(p.x.at(row, e), p.x.dtype, x);
        raw_value(x, p.x.dtype, v);
        drop(p.drop, key, row * p.d + e, v);
        if (p.res.p != nullptr) {
          float q[1];
          raw_load(p.res.at(row, e), p.res.dtype, x);
          raw_value(x, p.res.dtype, q);
          v[0] += q[0];
        }
        run_store(p.y.at(row, e), p.y.dtype, v);
      }
    }
  }
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
  const unsigned grid = static_cast<unsigned>(blocks < 152 * 8 * 8 ? blocks : 152 * 8 * 8);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  ProfScope prof("dropout", label, 0.0,
                 double(rows) * double(d) * (es_of(p.x.dtype) + (p.res.p ? es_of(p.res.dtype) : 0) + es_of(p.y.dtype)), s);
  if (wide)
    dropout_kernel<8><<<grid, 256, 0, s>>>(p);
  else
    dropout_kernel<1><<<grid, 256, 0, s>>>(p);
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
  d->step = static_cast<uint32_t>(std::nearbyint(o->p * 65536.0));
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
