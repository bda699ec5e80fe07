// Host side of the C ABI's sequence operators (include/rcu.h): the handle,
// argument checks and the launches of the gated linear recurrence (linrec_*.cu),
// layer norm (layernorm_*.cu) and 8-bit activation checkpoints (act8.cu).
#include <cmath>
#include <cstdint>
#include <new>

#include "api_seq.h"

using namespace rcu;
using namespace rcu_api;
using namespace rcu_seq_api;

namespace {

int check_linrec(const char *fn, rcu_seq *h, int dtype, int layout, int T, int B, int H,
                 const float *lambda, double c) {
  const int rc = check_handle(fn, h);
  if (rc != RCU_OK) return rc;
  if (!dtype_ok(dtype)) return fail(RCU_ERR_INVALID, "%s: dtype must be RCU_F32 or RCU_BF16", fn);
  if (layout != RCU_TIME_FIRST && layout != RCU_BATCH_FIRST)
    return fail(RCU_ERR_INVALID, "%s: unknown layout %d", fn, layout);
  if (T < 0 || B < 0 || H < 1)
    return fail(RCU_ERR_INVALID, "%s: T, B must be >= 0 and H >= 1 (got %d, %d, %d)", fn, T, B, H);
  if (H > WIDEST) return fail(RCU_ERR_UNSUPPORTED, "%s: H above 2^31 - 8192", fn);
  // tiles and rows are counted in 32 bits
  if (T > (1 << 30) || (int64_t)B * ((H + 31) / 32) > (1 << 30))
    return fail(RCU_ERR_UNSUPPORTED, "%s: T or B * H / 32 above 2^30", fn);
  if (!lambda) return fail(RCU_ERR_INVALID, "%s: lambda is NULL", fn);
  // c is used in fp32: it has to be a positive number there too
  if (!((float)c > 0.f) || !std::isfinite((float)c))
    return fail(RCU_ERR_INVALID, "%s: c must be positive and finite", fn);
  return RCU_OK;
}

int check_rows(const char *fn, rcu_seq *h, int dtype, int64_t rows, int n) {
  const int rc = check_handle(fn, h);
  if (rc != RCU_OK) return rc;
  if (!dtype_ok(dtype)) return fail(RCU_ERR_INVALID, "%s: dtype must be RCU_F32 or RCU_BF16", fn);
  if (rows < 0 || n < 1)
    return fail(RCU_ERR_INVALID, "%s: rows must be >= 0 and n >= 1 (got %lld, %d)", fn,
                (long long)rows, n);
  if (n > WIDEST) return fail(RCU_ERR_UNSUPPORTED, "%s: n above 2^31 - 8192", fn);
  return RCU_OK;
}

}  // namespace

extern "C" int rcu_seq_create(rcu_seq **out) {
  if (!out) return fail(RCU_ERR_INVALID, "rcu_seq_create: out is NULL");
  *out = nullptr;
  auto *h = new (std::nothrow) rcu_seq_s();
  if (!h) return fail(RCU_ERR_INVALID, "rcu_seq_create: out of host memory");
  h->nsm = device_sm_count(&h->device);
  cudaError_t e = h->ctl.ensure(256);
  if (e == cudaSuccess) e = cudaMemset(h->ctl.p, 0, 256);
  if (e != cudaSuccess) {
    delete h;
    return fail(RCU_ERR_CUDA, "rcu_seq_create: %s", cudaGetErrorString(e));
  }
  *out = h;
  return RCU_OK;
}

extern "C" int rcu_seq_destroy(rcu_seq *h) {
  if (!h) return RCU_OK;
  cudaDeviceSynchronize();
  delete h;
  return RCU_OK;
}

extern "C" int rcu_seq_get_status(rcu_seq *h, void *stream) {
  if (!h) return fail(RCU_ERR_INVALID, "rcu_seq_get_status: NULL handle");
  cudaStream_t s = (cudaStream_t)stream;
  int v = 0;
  CU(cudaMemcpyAsync(&v, h->ctl.p, 4, cudaMemcpyDeviceToHost, s));
  CU(cudaStreamSynchronize(s));
  CU(cudaMemsetAsync(h->ctl.p, 0, 4, s));
  if (v == DEV_LENGTHS) return fail(RCU_ERR_LENGTHS, "a length was outside [0, T]");
  if (v == DEV_SLOTS) return fail(RCU_ERR_SLOTS, "a state slot was outside [-1, slots)");
  return status_from_dev(v);
}

extern "C" int rcu_seq_set_attr(rcu_seq *h, int attr, int64_t value) {
  if (!h) return fail(RCU_ERR_INVALID, "rcu_seq_set_attr: NULL handle");
  if (attr == RCU_ATTR_PROFILE) {
    h->profile = value != 0;
    return RCU_OK;
  }
  if (attr == RCU_ATTR_FORCE_PATH) {
    if (value != 0 && value != 1)
      return fail(RCU_ERR_INVALID, "rcu_seq_set_attr: force_path must be 0 or 1");
    h->force_path = (int)value;
    return RCU_OK;
  }
  return fail(RCU_ERR_INVALID, "rcu_seq_set_attr: unknown attribute %d", attr);
}

extern "C" int rcu_seq_profile_entry(rcu_seq *h, int i, const char **name, double *total_ms,
                                     int64_t *count) {
  if (!h) return fail(RCU_ERR_INVALID, "rcu_seq_profile_entry: NULL handle");
  return h->entry(i, name, total_ms, count);
}

extern "C" int rcu_seq_profile_reset(rcu_seq *h) {
  if (!h) return fail(RCU_ERR_INVALID, "rcu_seq_profile_reset: NULL handle");
  h->reset();
  return RCU_OK;
}

extern "C" int rcu_seq_last_launch_count(rcu_seq *h) {
  if (!h) return fail(RCU_ERR_INVALID, "rcu_seq_last_launch_count: NULL handle");
  return h->launches;
}

extern "C" int rcu_linrec_forward(rcu_seq *h, int dtype, int layout, int T, int B, int H,
                                  const void *x, int64_t ldx, const void *r, int64_t ldr,
                                  const void *i, int64_t ldi, const float *lambda, double c,
                                  const int32_t *lengths, const float *h0, void *y, int64_t ldy,
                                  float *h_n, float *states, void *stream) {
  const int rc = check_linrec(__func__, h, dtype, layout, T, B, H, lambda, c);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (B == 0) return RCU_OK;
  if (T == 0) {
    CU(copy_or_zero(h_n, h0, (size_t)B * H, s));
    return RCU_OK;
  }
  MAT(x, ldx, H, true);
  MAT(r, ldr, H, true);
  MAT(i, ldi, H, true);
  MAT(y, ldy, H, true);
  const LinrecFwd p{dtype, T, B, H, seq_in(layout, T, B, x, ldx), seq_in(layout, T, B, r, ldr),
                    seq_in(layout, T, B, i, ldi), lambda, (float)c, lengths, h0,
                    seq_out(layout, T, B, y, ldy), h_n, states};
  begin(h, "linrec_forward", s);
  CU(launch_linrec_fwd(p, *h, (int *)h->ctl.p, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_linrec_backward(rcu_seq *h, int dtype, int saved, int layout, int T, int B,
                                   int H, const void *x, int64_t ldx, const void *r, int64_t ldr,
                                   const void *i, int64_t ldi, const int8_t *xe, const int8_t *re,
                                   const int8_t *ie, const float *lambda, double c,
                                   const int32_t *lengths, const float *states, const void *dy,
                                   int64_t lddy, const float *dh_n, void *dx, int64_t lddx,
                                   void *dr, int64_t lddr, void *di, int64_t lddi, float *dlambda,
                                   float *dh0, void *stream) {
  const int rc = check_linrec(__func__, h, dtype, layout, T, B, H, lambda, c);
  if (rc != RCU_OK) return rc;
  if (saved != dtype && saved != RCU_I8)
    return fail(RCU_ERR_INVALID, "rcu_linrec_backward: saved must be dtype or RCU_I8");
  const bool q8 = saved == RCU_I8;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (T == 0 || B == 0) {
    CU(copy_or_zero(dlambda, nullptr, H, s));
    CU(copy_or_zero(dh0, dh_n, (size_t)B * H, s));
    return RCU_OK;
  }
  MAT(x, ldx, H, true);
  MAT(r, ldr, H, true);
  MAT(i, ldi, H, true);
  MAT(dy, lddy, H, true);
  MAT(dx, lddx, H, false);
  MAT(dr, lddr, H, false);
  MAT(di, lddi, H, false);
  if (!states) return fail(RCU_ERR_INVALID, "rcu_linrec_backward: states is NULL");
  if (q8 != (xe != nullptr) || q8 != (re != nullptr) || q8 != (ie != nullptr))
    return fail(RCU_ERR_INVALID,
                "rcu_linrec_backward: exponents are required with RCU_I8 and NULL without");
  LinrecBwd p{dtype, saved, T, B, H, seq_in(layout, T, B, x, ldx, xe),
              seq_in(layout, T, B, r, ldr, re), seq_in(layout, T, B, i, ldi, ie), 0, 0, lambda,
              (float)c, lengths, states, seq_in(layout, T, B, dy, lddy), dh_n,
              seq_out(layout, T, B, dx, lddx), seq_out(layout, T, B, dr, lddr),
              seq_out(layout, T, B, di, lddi), dlambda, dh0};
  strides(layout, T, B, 1, &p.et, &p.eb);
  begin(h, "linrec_backward", s);
  CU(launch_linrec_bwd(p, *h, (int *)h->ctl.p, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_linrec_step(rcu_seq *h, int dtype, int B, int H, const void *x, int64_t ldx,
                               const void *r, int64_t ldr, const void *i, int64_t ldi,
                               const float *lambda, double c, float *state, int slots,
                               const int32_t *slot, void *y, int64_t ldy, void *stream) {
  const int rc = check_linrec(__func__, h, dtype, RCU_TIME_FIRST, 1, B, H, lambda, c);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (B == 0) return RCU_OK;
  MAT(x, ldx, H, true);
  MAT(r, ldr, H, true);
  MAT(i, ldi, H, true);
  MAT(y, ldy, H, true);
  if (!state) return fail(RCU_ERR_INVALID, "rcu_linrec_step: state is NULL");
  if (slots < 0 || (!slot && slots < B))
    return fail(RCU_ERR_INVALID, "rcu_linrec_step: %d state rows for %d requests", slots, B);
  begin(h, "linrec_step", s);
  CU(launch_linrec_step(dtype, B, H, x, ldx, r, ldr, i, ldi, lambda, (float)c, state, slots, slot,
                        y, ldy, (int *)h->ctl.p, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_layernorm_forward(rcu_seq *h, int dtype, int64_t rows, int n, const void *x,
                                     int64_t ldx, const void *residual, int64_t ldres,
                                     const float *weight, const float *bias, double eps, void *y,
                                     int64_t ldy, void *sum, int64_t ldsum, float *mean,
                                     float *rstd, void *stream) {
  const int rc = check_rows(__func__, h, dtype, rows, n);
  if (rc != RCU_OK) return rc;
  if (!(eps >= 0) || !std::isfinite((float)eps))
    return fail(RCU_ERR_INVALID, "rcu_layernorm_forward: eps must be >= 0 and finite");
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (rows == 0) return RCU_OK;
  MAT(x, ldx, n, true);
  MAT(residual, ldres, n, false);
  MAT(y, ldy, n, true);
  MAT(sum, ldsum, n, false);
  if ((residual != nullptr) != (sum != nullptr))
    return fail(RCU_ERR_INVALID, "rcu_layernorm_forward: residual and sum go together");
  const LnFwd p{dtype, rows, n, x, residual, ldx, ldres, weight, bias, (float)eps, y, sum, ldy,
                ldsum, mean, rstd};
  begin(h, "layernorm_forward", s);
  CU(launch_ln_fwd(p, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_layernorm_backward(rcu_seq *h, int dtype, int saved, int64_t rows, int n,
                                      const void *dy, int64_t lddy, const void *u, int64_t ldu,
                                      const int8_t *ue, const float *weight, const float *mean,
                                      const float *rstd, const void *dsum, int64_t ldds, void *du,
                                      int64_t lddu, float *dweight, float *dbias, void *stream) {
  const int rc = check_rows(__func__, h, dtype, rows, n);
  if (rc != RCU_OK) return rc;
  if (saved != dtype && saved != RCU_I8)
    return fail(RCU_ERR_INVALID, "rcu_layernorm_backward: saved must be dtype or RCU_I8");
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (rows == 0) {
    CU(copy_or_zero(dweight, nullptr, n, s));
    CU(copy_or_zero(dbias, nullptr, n, s));
    return RCU_OK;
  }
  MAT(dy, lddy, n, true);
  MAT(u, ldu, n, true);
  MAT(dsum, ldds, n, false);
  MAT(du, lddu, n, true);
  if (!mean || !rstd) return fail(RCU_ERR_INVALID, "rcu_layernorm_backward: mean or rstd is NULL");
  if ((saved == RCU_I8) != (ue != nullptr))
    return fail(RCU_ERR_INVALID,
                "rcu_layernorm_backward: exponents are required with RCU_I8 and NULL without");
  const LnBwd p{dtype, saved, rows, n, dy, u, lddy, ldu, ue, weight, mean, rstd, dsum, ldds, du,
                lddu, dweight, dbias};
  begin(h, "layernorm_backward", s);
  CU(launch_ln_bwd(p, *h, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_act8_pack(rcu_seq *h, int dtype, int64_t rows, int n, const void *x,
                             int64_t ldx, int8_t *codes, int64_t ldc, int8_t *exps, void *stream) {
  const int rc = check_rows(__func__, h, dtype, rows, n);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (rows == 0) return RCU_OK;
  MAT(x, ldx, n, true);
  MAT(codes, ldc, n, true);
  if (!exps) return fail(RCU_ERR_INVALID, "rcu_act8_pack: exps is NULL");
  begin(h, "act8_pack", s);
  CU(launch_act8_pack(dtype, rows, n, x, ldx, codes, ldc, exps, h->nsm, !h->force_path, s,
                      &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_act8_unpack(rcu_seq *h, int dtype, int64_t rows, int n, const int8_t *codes,
                               int64_t ldc, const int8_t *exps, void *y, int64_t ldy,
                               void *stream) {
  const int rc = check_rows(__func__, h, dtype, rows, n);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (rows == 0) return RCU_OK;
  MAT(codes, ldc, n, true);
  MAT(y, ldy, n, true);
  if (!exps) return fail(RCU_ERR_INVALID, "rcu_act8_unpack: exps is NULL");
  begin(h, "act8_unpack", s);
  CU(launch_act8_unpack(dtype, rows, n, codes, ldc, exps, y, ldy, h->nsm, !h->force_path, s,
                        &h->launches));
  h->prof_end(s);
  return RCU_OK;
}
