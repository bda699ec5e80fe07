// Launchers of the selective state space operators (short causal convolution,
// selective scan) and of the AdamW step, shared by their kernel files and
// api_ssm.cu / api_adamw.cu.  Arguments have been checked: dtype is RCU_F32 or
// RCU_BF16, T, B, H >= 1, row strides >= the row width.  `vec` false forbids the
// wide accesses that aligned rows otherwise use.  *launches counts kernels.
#pragma once

#include "rcu.h"
#include "seq.h"

namespace rcu {

struct ConvFwd {
  int dtype, T, B, H, W, silu;
  SeqIn x;
  const float *weight, *bias;
  const int32_t *lengths;
  const void *state;
  SeqOut y;
  void *state_n;
};
struct ConvBwd {
  int dtype, T, B, H, W, silu;
  SeqIn x;
  const float *weight, *bias;
  const int32_t *lengths;
  const void *state;
  SeqIn dy;
  const void *dstate_n;
  SeqOut dx;
  float *dweight, *dbias;
  void *dstate;
};
struct ConvStep {
  int dtype, B, H, W, silu;
  const void *x;
  int64_t ldx;
  const float *weight, *bias;
  void *state;
  int slots;
  const int32_t *slot;
  void *y;
  int64_t ldy;
};
cudaError_t launch_conv_fwd(const ConvFwd &p, int *err, int nsm, bool vec, cudaStream_t s,
                            int *launches);
cudaError_t launch_conv_bwd(const ConvBwd &p, DevMem &ws, int *err, int nsm, bool vec,
                            cudaStream_t s, int *launches);
cudaError_t launch_conv_step(const ConvStep &p, int *err, int nsm, bool vec, cudaStream_t s,
                             int *launches);

struct ScanIn {  // what the scan's passes share
  int dtype, T, B, H, N;
  SeqIn x, dt, b, c, z;
  const float *a_log, *d, *dt_bias;
  const int32_t *lengths;
};
struct ScanFwd {
  ScanIn in;
  const float *h0;
  SeqOut y;
  float *h_n, *states;
};
struct ScanBwd {
  ScanIn in;
  const float *states;
  SeqIn dy;
  const float *dh_n;
  SeqOut dx, ddt, db, dc, dz;
  float *da_log, *dd, *ddt_bias, *dh0;
};
struct ScanStep {
  int dtype, B, H, N;
  const void *x, *dt, *b, *c, *z;
  int64_t ldx, lddt, ldb, ldc, ldz;
  const float *a_log, *d, *dt_bias;
  float *state;
  int slots;
  const int32_t *slot;
  void *y;
  int64_t ldy;
};
cudaError_t launch_scan_fwd(const ScanFwd &p, DevMem &ws, int *err, int nsm, bool vec,
                            cudaStream_t s, int *launches);
cudaError_t launch_scan_bwd(const ScanBwd &p, DevMem &ws, int *err, int nsm, bool vec,
                            cudaStream_t s, int *launches);
cudaError_t launch_scan_step(const ScanStep &p, int *err, int nsm, bool vec, cudaStream_t s,
                             int *launches);

// Sums of the rows of a [rows, cols] fp32 matrix in a fixed order; columns from
// 0 to n0 go to out0, the next n1 to out1, the rest to out2 (NULL: dropped).
struct ColumnSum {
  const float *part;
  int64_t rows, cols;
  int64_t n0, n1;
  float *out0, *out1, *out2;
};
cudaError_t launch_column_sum(const ColumnSum &p, cudaStream_t s, int *launches);

struct AdamWStep {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;
  uint32_t seed;
  const float *scale;
  const int32_t *step_dev;
  const float *lr_dev;
};
cudaError_t launch_adamw(const AdamWStep &p, int64_t count, const rcu_adamw_tensor *tensors,
                         int nsm, bool vec, cudaStream_t s, int *launches);
cudaError_t launch_state8_pack(int is_signed, int64_t n, const float *x, int8_t *codes,
                               int8_t *exps, int nsm, bool vec, cudaStream_t s, int *launches);
cudaError_t launch_state8_unpack(int is_signed, int64_t n, const int8_t *codes,
                                 const int8_t *exps, float *y, int nsm, bool vec, cudaStream_t s,
                                 int *launches);

}  // namespace rcu
