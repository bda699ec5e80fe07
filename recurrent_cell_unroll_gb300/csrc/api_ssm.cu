// Host side of the selective state space operators of include/rcu.h: argument
// checks and the launches of the short causal convolution (conv.cu) and the
// selective scan (selscan_*.cu).
#include "api_seq.h"
#include "ssm.h"

using namespace rcu;
using namespace rcu_api;
using namespace rcu_seq_api;

namespace {

// What all of them check.  Threads and blocks are counted in 32 bits, over rows and
// groups of channels: a channel's states or taps stand beside one another.
int check_ssm(const char *fn, rcu_seq *h, int dtype, int layout, int T, int B, int H, int per,
              const char *per_name, int most) {
  const int rc = check_handle(fn, h);
  if (rc != RCU_OK) return rc;
  if (!dtype_ok(dtype)) return fail(RCU_ERR_INVALID, "%s: dtype must be RCU_F32 or RCU_BF16", fn);
  if (layout != RCU_TIME_FIRST && layout != RCU_BATCH_FIRST)
    return fail(RCU_ERR_INVALID, "%s: unknown layout %d", fn, layout);
  if (T < 0 || B < 0 || H < 1)
    return fail(RCU_ERR_INVALID, "%s: T, B must be >= 0 and H >= 1 (got %d, %d, %d)", fn, T, B, H);
  if (per < 1) return fail(RCU_ERR_INVALID, "%s: %s must be >= 1 (got %d)", fn, per_name, per);
  if (per > most) return fail(RCU_ERR_UNSUPPORTED, "%s: %s above %d", fn, per_name, most);
  if (T > (1 << 30)) return fail(RCU_ERR_UNSUPPORTED, "%s: T above 2^30", fn);
  if ((int64_t)B * H > ((int64_t)1 << 35) / 64 || (int64_t)T * B > ((int64_t)1 << 35) / 64)
    return fail(RCU_ERR_UNSUPPORTED, "%s: B * H or T * B above 2^29", fn);
  return RCU_OK;
}
int check_conv(const char *fn, rcu_seq *h, int dtype, int layout, int T, int B, int H, int W,
               const float *weight) {
  const int rc = check_ssm(fn, h, dtype, layout, T, B, H, W, "W", RCU_CONV_MAX_TAPS);
  if (rc != RCU_OK) return rc;
  return weight ? RCU_OK : fail(RCU_ERR_INVALID, "%s: weight is NULL", fn);
}
int check_scan(const char *fn, rcu_seq *h, int dtype, int layout, int T, int B, int H, int N,
               const float *a_log) {
  const int rc = check_ssm(fn, h, dtype, layout, T, B, H, N, "N", RCU_SELSCAN_MAX_STATES);
  if (rc != RCU_OK) return rc;
  return a_log ? RCU_OK : fail(RCU_ERR_INVALID, "%s: a_log is NULL", fn);
}

// [B, W - 1, H] of a dtype: copied, or zeros where there is no source.
cudaError_t pass_state(int dtype, int B, int H, int W, const void *from, void *to, cudaStream_t s) {
  const size_t bytes = (size_t)B * H * (W - 1) * (dtype == RCU_BF16 ? 2 : 4);
  if (!to || !bytes || to == from) return cudaSuccess;
  return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s)
              : cudaMemsetAsync(to, 0, bytes, s);
}

int check_slots(const char *fn, int B, const void *state, int slots, const int32_t *slot) {
  if (!state) return fail(RCU_ERR_INVALID, "%s: state is NULL", fn);
  if (slots < 0 || (!slot && slots < B))
    return fail(RCU_ERR_INVALID, "%s: %d state rows for %d requests", fn, slots, B);
  return RCU_OK;
}

}  // namespace

extern "C" int rcu_conv_forward(rcu_seq *h, int dtype, int layout, int T, int B, int H, int W,
                                const void *x, int64_t ldx, const float *weight, const float *bias,
                                int silu, const int32_t *lengths, const void *state, void *y,
                                int64_t ldy, void *state_n, void *stream) {
  const int rc = check_conv(__func__, h, dtype, layout, T, B, H, W, weight);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (B == 0) return RCU_OK;
  if (T == 0) {
    CU(pass_state(dtype, B, H, W, state, state_n, s));
    return RCU_OK;
  }
  MAT(x, ldx, H, true);
  MAT(y, ldy, H, true);
  const ConvFwd p{dtype, T, B, H, W, silu != 0, seq_in(layout, T, B, x, ldx), weight, bias, lengths,
                  state, seq_out(layout, T, B, y, ldy), W > 1 ? state_n : nullptr};
  begin(h, "conv_forward", s);
  CU(launch_conv_fwd(p, (int *)h->ctl.p, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_conv_backward(rcu_seq *h, int dtype, int layout, int T, int B, int H, int W,
                                 const void *x, int64_t ldx, const float *weight, const float *bias,
                                 int silu, const int32_t *lengths, const void *state, const void *dy,
                                 int64_t lddy, const void *dstate_n, void *dx, int64_t lddx,
                                 float *dweight, float *dbias, void *dstate, void *stream) {
  const int rc = check_conv(__func__, h, dtype, layout, T, B, H, W, weight);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (T == 0 || B == 0) {
    CU(copy_or_zero(dweight, nullptr, (size_t)H * W, s));
    CU(copy_or_zero(dbias, nullptr, H, s));
    CU(pass_state(dtype, B, H, W, dstate_n, dstate, s));
    return RCU_OK;
  }
  MAT(x, ldx, H, true);
  MAT(dy, lddy, H, true);
  MAT(dx, lddx, H, false);
  if (W > 1 && dstate && dstate == dstate_n)
    return fail(RCU_ERR_INVALID, "rcu_conv_backward: dstate must not be dstate_n");
  const ConvBwd p{dtype, T, B, H, W, silu != 0, seq_in(layout, T, B, x, ldx), weight, bias, lengths,
                  state, seq_in(layout, T, B, dy, lddy), W > 1 ? dstate_n : nullptr,
                  seq_out(layout, T, B, dx, lddx), dweight, dbias, W > 1 ? dstate : nullptr};
  begin(h, "conv_backward", s);
  CU(launch_conv_bwd(p, *h, (int *)h->ctl.p, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_conv_step(rcu_seq *h, int dtype, int B, int H, int W, const void *x, int64_t ldx,
                             const float *weight, const float *bias, int silu, void *state, int slots,
                             const int32_t *slot, void *y, int64_t ldy, void *stream) {
  const int rc = check_conv(__func__, h, dtype, RCU_TIME_FIRST, 1, B, H, W, weight);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (B == 0) return RCU_OK;
  MAT(x, ldx, H, true);
  MAT(y, ldy, H, true);
  const int sc = check_slots(__func__, B, state, slots, slot);
  if (sc != RCU_OK) return sc;
  const ConvStep p{dtype, B, H, W, silu != 0, x, ldx, weight, bias, state, slots, slot, y, ldy};
  begin(h, "conv_step", s);
  CU(launch_conv_step(p, (int *)h->ctl.p, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_selscan_forward(rcu_seq *h, int dtype, int layout, int T, int B, int H, int N,
                                   const void *x, int64_t ldx, const void *dt, int64_t lddt,
                                   const float *a_log, const void *b, int64_t ldb, const void *c,
                                   int64_t ldc, const float *d, const float *dt_bias, const void *z,
                                   int64_t ldz, const int32_t *lengths, const float *h0, void *y,
                                   int64_t ldy, float *h_n, float *states, void *stream) {
  const int rc = check_scan(__func__, h, dtype, layout, T, B, H, N, a_log);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (B == 0) return RCU_OK;
  if (T == 0) {
    if (h_n != h0) CU(copy_or_zero(h_n, h0, (size_t)B * H * N, s));
    return RCU_OK;
  }
  MAT(x, ldx, H, true);
  MAT(dt, lddt, H, true);
  MAT(b, ldb, N, true);
  MAT(c, ldc, N, true);
  MAT(z, ldz, H, false);
  MAT(y, ldy, H, true);
  const ScanFwd p{{dtype, T, B, H, N, seq_in(layout, T, B, x, ldx), seq_in(layout, T, B, dt, lddt),
                   seq_in(layout, T, B, b, ldb), seq_in(layout, T, B, c, ldc),
                   seq_in(layout, T, B, z, ldz), a_log, d, dt_bias, lengths},
                  h0, seq_out(layout, T, B, y, ldy), h_n, states};
  begin(h, "selscan_forward", s);
  CU(launch_scan_fwd(p, *h, (int *)h->ctl.p, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_selscan_backward(rcu_seq *h, int dtype, int layout, int T, int B, int H, int N,
                                    const void *x, int64_t ldx, const void *dt, int64_t lddt,
                                    const float *a_log, const void *b, int64_t ldb, const void *c,
                                    int64_t ldc, const float *d, const float *dt_bias, const void *z,
                                    int64_t ldz, const int32_t *lengths, const float *states,
                                    const void *dy, int64_t lddy, const float *dh_n, void *dx,
                                    int64_t lddx, void *ddt, int64_t ldddt, float *da_log, void *db,
                                    int64_t lddb, void *dc, int64_t lddc, float *dd, float *ddt_bias,
                                    void *dz, int64_t lddz, float *dh0, void *stream) {
  const int rc = check_scan(__func__, h, dtype, layout, T, B, H, N, a_log);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (T == 0 || B == 0) {
    CU(copy_or_zero(da_log, nullptr, (size_t)H * N, s));
    CU(copy_or_zero(dd, nullptr, H, s));
    CU(copy_or_zero(ddt_bias, nullptr, H, s));
    if (dh0 != dh_n) CU(copy_or_zero(dh0, dh_n, (size_t)B * H * N, s));
    return RCU_OK;
  }
  MAT(x, ldx, H, true);
  MAT(dt, lddt, H, true);
  MAT(b, ldb, N, true);
  MAT(c, ldc, N, true);
  MAT(z, ldz, H, false);
  MAT(dy, lddy, H, true);
  MAT(dx, lddx, H, false);
  MAT(ddt, ldddt, H, false);
  MAT(db, lddb, N, false);
  MAT(dc, lddc, N, false);
  MAT(dz, lddz, H, false);
  if (!states) return fail(RCU_ERR_INVALID, "rcu_selscan_backward: states is NULL");
  if (dz && !z) return fail(RCU_ERR_INVALID, "rcu_selscan_backward: dz without z");
  if (dd && !d) return fail(RCU_ERR_INVALID, "rcu_selscan_backward: dd without d");
  const ScanBwd p{{dtype, T, B, H, N, seq_in(layout, T, B, x, ldx), seq_in(layout, T, B, dt, lddt),
                   seq_in(layout, T, B, b, ldb), seq_in(layout, T, B, c, ldc),
                   seq_in(layout, T, B, z, ldz), a_log, d, dt_bias, lengths},
                  states, seq_in(layout, T, B, dy, lddy), dh_n, seq_out(layout, T, B, dx, lddx),
                  seq_out(layout, T, B, ddt, ldddt), seq_out(layout, T, B, db, lddb),
                  seq_out(layout, T, B, dc, lddc), seq_out(layout, T, B, dz, lddz), da_log, dd,
                  ddt_bias, dh0};
  begin(h, "selscan_backward", s);
  CU(launch_scan_bwd(p, *h, (int *)h->ctl.p, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_selscan_step(rcu_seq *h, int dtype, int B, int H, int N, const void *x,
                                int64_t ldx, const void *dt, int64_t lddt, const float *a_log,
                                const void *b, int64_t ldb, const void *c, int64_t ldc,
                                const float *d, const float *dt_bias, const void *z, int64_t ldz,
                                float *state, int slots, const int32_t *slot, void *y, int64_t ldy,
                                void *stream) {
  const int rc = check_scan(__func__, h, dtype, RCU_TIME_FIRST, 1, B, H, N, a_log);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (B == 0) return RCU_OK;
  MAT(x, ldx, H, true);
  MAT(dt, lddt, H, true);
  MAT(b, ldb, N, true);
  MAT(c, ldc, N, true);
  MAT(z, ldz, H, false);
  MAT(y, ldy, H, true);
  const int sc = check_slots(__func__, B, state, slots, slot);
  if (sc != RCU_OK) return sc;
  const ScanStep p{dtype, B, H, N, x, dt, b, c, z, ldx, lddt, ldb, ldc, ldz, a_log, d, dt_bias,
                   state, slots, slot, y, ldy};
  begin(h, "selscan_step", s);
  CU(launch_scan_step(p, (int *)h->ctl.p, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}
