// Gated linear recurrence, one step of many requests: states in a table of
// slots, updated in place.  24 bytes (fp32) or 16 (bf16) an element: at serving
// sizes the launch is what it costs.
#include "linrec_tile.cuh"

namespace rcu {
namespace {

using namespace linrec;

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
    const float k2 = decay_rate2(lambda[h], c);
    const F2 vx[1] = {f2(to_f(x[b * ldx + h]))};
    const F2 vr[1] = {f2(limit_r(to_f(r[b * ldr + h]), limits(k2)))};
    const F2 vi[1] = {f2(to_f(i[b * ldi + h]))};
    F2 em1, nb, ns, ng;
    gates_n<false, 1>(vx, vr, vi, f2(k2), &em1, &nb, &ns, &ng);
    out = state[row * H + h] = step(lo(em1), state[row * H + h], -lo(nb));
  }
  y[b * ldy + h] = from_f<T>(out);
}

}  // namespace

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
