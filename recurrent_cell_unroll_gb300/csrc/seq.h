// Launchers of the sequence operators (gated linear recurrence, layer norm,
// 8-bit activation checkpoints), shared by their kernel files and api_seq.cu.
// Arguments have been checked: dtype is RCU_F32 or RCU_BF16, sizes are >= 1,
// row strides >= the row width.  `vec` false forbids the wide and asynchronous
// accesses that aligned rows otherwise use.  *launches counts kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace rcu {

// A [T, B, H] tensor: element (t, b, h) at p + t*st + b*sb + h (elements).
struct SeqIn {
  const void *p;
  int64_t st, sb;
  const int8_t *e;  // 8-bit checkpoint: exponents [rows][ceil(H/64)]; else NULL
};
struct SeqOut {
  void *p;
  int64_t st, sb;
};

struct LinrecFwd {
  int dtype, T, B, H;
  SeqIn x, r, i;  // one behind another: kernels take them by number
  const float *lambda;
  float c;
  const int32_t *lengths;
  const float *h0;
  SeqOut y;
  float *h_n, *states;
};

struct LinrecBwd {
  int dtype, saved, T, B, H;
  SeqIn x, r, i;  // one behind another: kernels take them by number
  int64_t et, eb;  // rows of the exponents: row (t, b) = t*et + b*eb
  const float *lambda;
  float c;
  const int32_t *lengths;
  const float *states;
  SeqIn dy;
  const float *dh_n;
  SeqOut dx, dr, di;  // as x, r, i
  float *dlambda, *dh0;
};

// Device memory that a call may use between its launches; it grows on demand
// and is the handle's.
struct DevMem {
  virtual cudaError_t grow(size_t bytes, void **p) = 0;
  cudaError_t get(size_t bytes, void **p) { return grow(bytes, p); }
  template <typename T>
  cudaError_t get(size_t bytes, T **p) {
    void *v = nullptr;
    const cudaError_t e = grow(bytes, &v);
    *p = static_cast<T *>(v);
    return e;
  }
};

// A launch of a kernel that sums what the one before it on the stream wrote, and
// starts with wait_for_previous(): its blocks are brought up while that one ends.
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*fn)(KArgs...), dim3 grid, int threads, cudaStream_t s,
                         Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}
// Until the kernel before this one on the stream has ended and its writes are seen.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

cudaError_t launch_linrec_fwd(const LinrecFwd &p, DevMem &ws, int *err, int nsm, bool vec,
                              cudaStream_t s, int *launches);
cudaError_t launch_linrec_bwd(const LinrecBwd &p, DevMem &ws, int *err, int nsm, bool vec,
                              cudaStream_t s, int *launches);
cudaError_t launch_linrec_step(int dtype, int B, int H, const void *x, int64_t ldx, const void *r,
                               int64_t ldr, const void *i, int64_t ldi, const float *lambda,
                               float c, float *state, int slots, const int32_t *slot, void *y,
                               int64_t ldy, int *err, int nsm, bool vec, cudaStream_t s,
                               int *launches);

struct LnFwd {
  int dtype;
  int64_t rows;
  int n;
  const void *x, *res;
  int64_t ldx, ldres;
  const float *weight, *bias;
  float eps;
  void *y, *sum;
  int64_t ldy, ldsum;
  float *mean, *rstd;
};
struct LnBwd {
  int dtype, saved;
  int64_t rows;
  int n;
  const void *dy, *u;
  int64_t lddy, ldu;
  const int8_t *ue;
  const float *weight, *mean, *rstd;
  const void *dsum;
  int64_t ldds;
  void *du;
  int64_t lddu;
  float *dweight, *dbias;
};
cudaError_t launch_ln_fwd(const LnFwd &p, int nsm, bool vec, cudaStream_t s, int *launches);
cudaError_t launch_ln_bwd(const LnBwd &p, DevMem &ws, int nsm, bool vec, cudaStream_t s,
                          int *launches);

cudaError_t launch_act8_pack(int dtype, int64_t rows, int n, const void *x, int64_t ldx,
                             int8_t *codes, int64_t ldc, int8_t *exps, int nsm, bool vec,
                             cudaStream_t s, int *launches);
cudaError_t launch_act8_unpack(int dtype, int64_t rows, int n, const int8_t *codes, int64_t ldc,
                               const int8_t *exps, void *y, int64_t ldy, int nsm, bool vec,
                               cudaStream_t s, int *launches);

}  // namespace rcu
