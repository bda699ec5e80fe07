// The handle of the sequence operators and the argument checks that its entry
// points share (api_seq.cu, api_ssm.cu, api_adamw.cu).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "rcu.h"
#include "common.cuh"
#include "seq.h"
#include "api_host.h"

using rcu::DevMem;
using rcu::SeqIn;
using rcu::SeqOut;
using rcu_api::DevBuf;
using rcu_api::EventProfiler;
using rcu_api::fail;

struct rcu_seq_s : EventProfiler, DevMem {
  int device, nsm;
  DevBuf ctl;  // device error word
  DevBuf ws;   // partial sums of the call in flight
  // An outgrown buffer lives as long as the handle: a captured graph may still
  // use it.  Growing to twice the size at least bounds what they hold together.
  std::vector<void *> outgrown;
  cudaError_t grow(size_t bytes, void **p) override {
    if (bytes > ws.n && ws.p) {
      outgrown.push_back(ws.p);
      bytes = std::max(bytes, 2 * ws.n);
      ws.p = nullptr;
      ws.n = 0;
    }
    const cudaError_t e = ws.ensure(bytes);
    if (e != cudaSuccess) cudaGetLastError();  // reported here, not by the next launch too
    *p = ws.p;
    return e;
  }
  ~rcu_seq_s() {
    for (void *p : outgrown) cudaFree(p);
  }
  int force_path = 0;
  int launches = 0;
};

namespace rcu_seq_api {

// Begin a call: no kernels counted yet, its span opened.
inline void begin(rcu_seq *h, const char *name, cudaStream_t s) {
  h->launches = 0;
  h->prof_begin(name, s);
}

// A row's columns are counted in 32 bits, and blocks of them end past its own end (by
// 4096 at most: layer norm of long rows).
constexpr int WIDEST = INT32_MAX - 8191;

inline bool dtype_ok(int dtype) { return dtype == RCU_F32 || dtype == RCU_BF16; }

// The handle, and that its device is the current one.
inline int check_handle(const char *fn, rcu_seq *h) {
  if (!h) return fail(RCU_ERR_INVALID, "%s: NULL handle", fn);
  int dev = -1;
  CU(cudaGetDevice(&dev));
  if (dev != h->device)
    return fail(RCU_ERR_INVALID, "%s: the handle belongs to device %d, the current one is %d", fn,
                h->device, dev);
  return RCU_OK;
}

// A matrix operand: present, and its rows do not overlap.
inline int check_mat(const char *fn, const char *name, const void *p, int64_t ld, int width,
              bool required) {
  if (!p) return required ? fail(RCU_ERR_INVALID, "%s: %s is NULL", fn, name) : RCU_OK;
  if (ld < width)
    return fail(RCU_ERR_INVALID, "%s: row stride of %s is %lld, below its width %d", fn, name,
                (long long)ld, width);
  return RCU_OK;
}

#define MAT(p, ld, width, required)                                        \
  do {                                                                     \
    const int rc_ = check_mat(__func__, #p, (p), (ld), (width), required); \
    if (rc_ != RCU_OK) return rc_;                                         \
  } while (0)

// Strides of a [T, B, H] tensor in elements of its rows' stride.
inline void strides(int layout, int T, int B, int64_t ld, int64_t *st, int64_t *sb) {
  *st = layout == RCU_BATCH_FIRST ? ld : (int64_t)B * ld;
  *sb = layout == RCU_BATCH_FIRST ? (int64_t)T * ld : ld;
}
inline SeqIn seq_in(int layout, int T, int B, const void *p, int64_t ld, const int8_t *e = nullptr) {
  SeqIn v{p, 0, 0, e};
  strides(layout, T, B, ld, &v.st, &v.sb);
  return v;
}
inline SeqOut seq_out(int layout, int T, int B, void *p, int64_t ld) {
  SeqOut v{p, 0, 0};
  strides(layout, T, B, ld, &v.st, &v.sb);
  return v;
}

// Copy [n] floats, or zero them where there is no source.
inline cudaError_t copy_or_zero(float *dst, const float *src, size_t n, cudaStream_t s) {
  if (!dst || !n) return cudaSuccess;
  return src ? cudaMemcpyAsync(dst, src, n * 4, cudaMemcpyDeviceToDevice, s)
             : cudaMemsetAsync(dst, 0, n * 4, s);
}

}  // namespace rcu_seq_api
