// Gated linear recurrence: forward, backward and single-token step.
#include "common.cuh"
#include "linrec_math.cuh"
#include "rcu.h"
#include "seq.h"

namespace rcu {
namespace {

using namespace linrec;
using bf16 = __nv_bfloat16;

constexpr int CHUNK = RCU_LINREC_CHUNK;
constexpr int BLOCK8 = RCU_ACT8_BLOCK;

// The length of row b, clamped to [0, T]; an outside value is reported.
__device__ __forceinline__ int row_length(const int32_t *lengths, int b, int T, int *err) {
  if (!lengths) return T;
  const int len = lengths[b];
  if (len < 0 || len > T) atomicCAS(err, (int)DEV_OK, (int)DEV_LENGTHS);
  return min(max(len, 0), T);
}

template <typename T>
__device__ __forceinline__ float value(const SeqIn &v, int t, int b, int h, int64_t erow, int nb) {
  return to_f(static_cast<const T *>(v.p)[t * v.st + b * v.sb + h]);
}
// what a code of an 8-bit checkpoint stands for
__device__ __forceinline__ float decode8(int code, int e) {
  return code == -128 ? __int_as_float(0x7fc00000)
                      : (float)code * __int_as_float((e + 127) << 23);
}
template <>
__device__ __forceinline__ float value<int8_t>(const SeqIn &v, int t, int b, int h, int64_t erow,
                                               int nb) {
  return decode8(static_cast<const int8_t *>(v.p)[t * v.st + b * v.sb + h],
                 v.e[erow * nb + h / BLOCK8]);
}

template <typename T>
__global__ void linrec_fwd_kernel(LinrecFwd p, int *err) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= (int64_t)p.B * p.H) return;
  const int b = (int)(id / p.H), h = (int)(id % p.H);
  const int len = row_length(p.lengths, b, p.T, err);
  const float k2 = decay_rate2(p.lambda[h], p.c);
  float s = p.h0 ? p.h0[id] : 0.f;
  T *y = static_cast<T *>(p.y.p);
  for (int t = 0; t < p.T; ++t) {
    if (p.states && t % CHUNK == 0) p.states[(int64_t)(t / CHUNK) * p.B * p.H + id] = s;
    float out = 0.f;
    if (t < len) {
      float em1, in;
      gate(value<T>(p.x, t, b, h, 0, 0), value<T>(p.r, t, b, h, 0, 0),
           value<T>(p.i, t, b, h, 0, 0), k2, em1, in);
      out = s = step(em1, s, in);
    }
    y[t * p.y.st + b * p.y.sb + h] = from_f<T>(out);
  }
  if (p.h_n) p.h_n[id] = s;
}

// IT: the saved inputs' type, T: the gradients'
template <typename IT, typename T>
__global__ void linrec_bwd_kernel(LinrecBwd p, float *partial, int *err) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= (int64_t)p.B * p.H) return;
  const int b = (int)(id / p.H), h = (int)(id % p.H), nb = ceil_div(p.H, BLOCK8);
  const int len = row_length(p.lengths, b, p.T, err);
  const float k2 = decay_rate2(p.lambda[h], p.c), k = k2 * (1.f / LOG2E);
  float come = p.dh_n ? p.dh_n[id] : 0.f, sum = 0.f;
  float hp[CHUNK];
  for (int c = (p.T - 1) / CHUNK; c >= 0; --c) {
    const int t0 = c * CHUNK, n = min(CHUNK, p.T - t0);
    float s = p.states[(int64_t)c * p.B * p.H + id];
    for (int j = 0; j < n && t0 + j < len; ++j) {
      const int t = t0 + j;
      const int64_t er = t * p.et + b * p.eb;
      float em1, in;
      hp[j] = s;
      gate(value<IT>(p.x, t, b, h, er, nb), value<IT>(p.r, t, b, h, er, nb),
           value<IT>(p.i, t, b, h, er, nb), k2, em1, in);
      s = step(em1, s, in);
    }
    for (int j = n - 1; j >= 0; --j) {
      const int t = t0 + j;
      const int64_t er = t * p.et + b * p.eb;
      Grad d{0.f, 0.f, 0.f, 0.f};
      if (t < len) {
        const float x = value<IT>(p.x, t, b, h, er, nb);
        const Sig v = sigmoids(value<IT>(p.r, t, b, h, er, nb), value<IT>(p.i, t, b, h, er, nb));
        const float em1 = ex2m1(k2 * v.s);
        const float e = come + value<T>(p.dy, t, b, h, 0, 0);
        d = grads(x, v, em1, k, hp[j], e);
        come = step(em1, e, 0.f);
        sum += d.dlog_s;
      }
      if (p.dx.p) static_cast<T *>(p.dx.p)[t * p.dx.st + b * p.dx.sb + h] = from_f<T>(d.dx);
      if (p.dr.p) static_cast<T *>(p.dr.p)[t * p.dr.st + b * p.dr.sb + h] = from_f<T>(d.dr);
      if (p.di.p) static_cast<T *>(p.di.p)[t * p.di.st + b * p.di.sb + h] = from_f<T>(d.di);
    }
  }
  if (p.dh0) p.dh0[id] = come;
  partial[id] = sum;
}

// dlambda[h] = -c sigmoid(lambda) * the sum of the rows' partial sums, in row order
__global__ void linrec_dlambda_kernel(const float *partial, int rows, int H, const float *lambda,
                                      float c, float *dlambda) {
  const int h = blockIdx.x * blockDim.x + threadIdx.x;
  if (h >= H) return;
  float s = 0.f;
  for (int b = 0; b < rows; ++b) s += partial[(int64_t)b * H + h];
  dlambda[h] = -c * s / (1.f + expf(-lambda[h]));
}

template <typename T>
__global__ void linrec_step_kernel(int B, int H, const T *x, int64_t ldx, const T *r, int64_t ldr,
                                   const T *i, int64_t ldi, const float *lambda, float c,
                                   float *state, int slots, const int32_t *slot, T *y,
                                   int64_t ldy, int *err) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= (int64_t)B * H) return;
  const int64_t b = id / H;
  const int h = (int)(id % H);
  int64_t row = slot ? slot[b] : b;
  if (row < -1 || row >= slots) {
    atomicCAS(err, (int)DEV_OK, (int)DEV_SLOTS);
    row = -1;
  }
  float out = 0.f;
  if (row >= 0) {
    float em1, in;
    gate(to_f(x[b * ldx + h]), to_f(r[b * ldr + h]), to_f(i[b * ldi + h]),
         decay_rate2(lambda[h], c), em1, in);
    out = state[row * H + h] = step(em1, state[row * H + h], in);
  }
  y[b * ldy + h] = from_f<T>(out);
}

}  // namespace

size_t linrec_fwd_workspace(const LinrecFwd &, int) { return 0; }

cudaError_t launch_linrec_fwd(const LinrecFwd &p, void *, int *err, int, bool, cudaStream_t s,
                              int *launches) {
  const unsigned grid = (unsigned)(((int64_t)p.B * p.H + 127) / 128);
  if (p.dtype == RCU_BF16)
    linrec_fwd_kernel<bf16><<<grid, 128, 0, s>>>(p, err);
  else
    linrec_fwd_kernel<float><<<grid, 128, 0, s>>>(p, err);
  ++*launches;
  return cudaGetLastError();
}

size_t linrec_bwd_workspace(const LinrecBwd &p, int) { return (size_t)p.B * p.H * 4; }

cudaError_t launch_linrec_bwd(const LinrecBwd &p, void *ws, int *err, int, bool, cudaStream_t s,
                              int *launches) {
  const unsigned grid = (unsigned)(((int64_t)p.B * p.H + 127) / 128);
  float *partial = static_cast<float *>(ws);
  const bool q8 = p.saved == RCU_I8;
  if (p.dtype == RCU_BF16) {
    if (q8) linrec_bwd_kernel<int8_t, bf16><<<grid, 128, 0, s>>>(p, partial, err);
    else linrec_bwd_kernel<bf16, bf16><<<grid, 128, 0, s>>>(p, partial, err);
  } else {
    if (q8) linrec_bwd_kernel<int8_t, float><<<grid, 128, 0, s>>>(p, partial, err);
    else linrec_bwd_kernel<float, float><<<grid, 128, 0, s>>>(p, partial, err);
  }
  ++*launches;
  if (p.dlambda) {
    linrec_dlambda_kernel<<<ceil_div(p.H, 128), 128, 0, s>>>(partial, p.B, p.H, p.lambda, p.c,
                                                             p.dlambda);
    ++*launches;
  }
  return cudaGetLastError();
}

cudaError_t launch_linrec_step(int dtype, int B, int H, const void *x, int64_t ldx, const void *r,
                               int64_t ldr, const void *i, int64_t ldi, const float *lambda,
                               float c, float *state, int slots, const int32_t *slot, void *y,
                               int64_t ldy, int *err, bool, cudaStream_t s, int *launches) {
  const unsigned grid = (unsigned)(((int64_t)B * H + 127) / 128);
  if (dtype == RCU_BF16)
    linrec_step_kernel<bf16><<<grid, 128, 0, s>>>(B, H, (const bf16 *)x, ldx, (const bf16 *)r, ldr,
                                                  (const bf16 *)i, ldi, lambda, c, state, slots,
                                                  slot, (bf16 *)y, ldy, err);
  else
    linrec_step_kernel<float><<<grid, 128, 0, s>>>(B, H, (const float *)x, ldx, (const float *)r,
                                                   ldr, (const float *)i, ldi, lambda, c, state,
                                                   slots, slot, (float *)y, ldy, err);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace rcu
