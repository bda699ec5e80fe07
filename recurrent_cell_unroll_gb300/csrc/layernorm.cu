// Layer norm: forward (with the residual addition before it) and backward
// (with the reduction of the weight's and bias's gradients).
#include "common.cuh"
#include "linrec_math.cuh"
#include "rcu.h"
#include "seq.h"

namespace rcu {
namespace {

using bf16 = __nv_bfloat16;
using linrec::from_f;
using linrec::to_f;

constexpr int NT = 256;

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[NT / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) v += part[w];
  return v;
}

template <typename T>
__global__ void ln_fwd_kernel(LnFwd p) {
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T *>(p.x) + row * p.ldx;
  const T *res = p.res ? static_cast<const T *>(p.res) + row * p.ldres : nullptr;
  T *sum = p.sum ? static_cast<T *>(p.sum) + row * p.ldsum : nullptr;
  T *y = static_cast<T *>(p.y) + row * p.ldy;
  auto u = [&](int c) {
    return res ? to_f(from_f<T>(to_f(x[c]) + to_f(res[c]))) : to_f(x[c]);
  };
  float s = 0.f;
  for (int c = threadIdx.x; c < p.n; c += NT) {
    const float v = u(c);
    if (sum) sum[c] = from_f<T>(v);
    s += v;
  }
  const float mean = block_sum(s) / p.n;
  s = 0.f;
  for (int c = threadIdx.x; c < p.n; c += NT) {
    const float d = u(c) - mean;
    s += d * d;
  }
  const float rstd = 1.f / sqrtf(block_sum(s) / p.n + p.eps);
  for (int c = threadIdx.x; c < p.n; c += NT)
    y[c] = from_f<T>((u(c) - mean) * rstd * (p.weight ? p.weight[c] : 1.f) +
                     (p.bias ? p.bias[c] : 0.f));
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

template <typename IT>
__device__ __forceinline__ float saved(const LnBwd &p, int64_t row, int c) {
  return to_f(static_cast<const IT *>(p.u)[row * p.ldu + c]);
}
template <>
__device__ __forceinline__ float saved<int8_t>(const LnBwd &p, int64_t row, int c) {
  const int code = static_cast<const int8_t *>(p.u)[row * p.ldu + c];
  const int e = p.ue[row * ceil_div(p.n, RCU_ACT8_BLOCK) + c / RCU_ACT8_BLOCK];
  return code == -128 ? __int_as_float(0x7fc00000) : (float)code * __int_as_float((e + 127) << 23);
}

template <typename IT, typename T>
__global__ void ln_bwd_kernel(LnBwd p) {
  const int64_t row = blockIdx.x;
  const T *dy = static_cast<const T *>(p.dy) + row * p.lddy;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < p.n; c += NT) {
    const float q = to_f(dy[c]) * (p.weight ? p.weight[c] : 1.f);
    s1 += q;
    s2 += q * (saved<IT>(p, row, c) - mean) * rstd;
  }
  s1 = block_sum(s1) / p.n;
  s2 = block_sum(s2) / p.n;
  for (int c = threadIdx.x; c < p.n; c += NT) {
    const float q = to_f(dy[c]) * (p.weight ? p.weight[c] : 1.f);
    const float xh = (saved<IT>(p, row, c) - mean) * rstd;
    float d = rstd * (q - s1 - xh * s2);
    if (p.dsum) d += to_f(static_cast<const T *>(p.dsum)[row * p.ldds + c]);
    static_cast<T *>(p.du)[row * p.lddu + c] = from_f<T>(d);
  }
}

template <typename IT, typename T>
__global__ void ln_bwd_columns_kernel(LnBwd p) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.n) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = 0; row < p.rows; ++row) {
    const float g = to_f(static_cast<const T *>(p.dy)[row * p.lddy + c]);
    dw += g * (saved<IT>(p, row, c) - p.mean[row]) * p.rstd[row];
    db += g;
  }
  if (p.dweight) p.dweight[c] = dw;
  if (p.dbias) p.dbias[c] = db;
}

template <typename IT, typename T>
void bwd(const LnBwd &p, cudaStream_t s, int *launches) {
  ln_bwd_kernel<IT, T><<<(unsigned)p.rows, NT, 0, s>>>(p);
  ++*launches;
  if (p.dweight || p.dbias) {
    ln_bwd_columns_kernel<IT, T><<<ceil_div(p.n, 32), 32, 0, s>>>(p);
    ++*launches;
  }
}

}  // namespace

cudaError_t launch_ln_fwd(const LnFwd &p, int, bool, cudaStream_t s, int *launches) {
  if (p.dtype == RCU_BF16)
    ln_fwd_kernel<bf16><<<(unsigned)p.rows, NT, 0, s>>>(p);
  else
    ln_fwd_kernel<float><<<(unsigned)p.rows, NT, 0, s>>>(p);
  ++*launches;
  return cudaGetLastError();
}

size_t ln_bwd_workspace(const LnBwd &, int) { return 0; }

cudaError_t launch_ln_bwd(const LnBwd &p, void *, int, bool, cudaStream_t s, int *launches) {
  const bool q8 = p.saved == RCU_I8;
  if (p.dtype == RCU_BF16) {
    if (q8) bwd<int8_t, bf16>(p, s, launches);
    else bwd<bf16, bf16>(p, s, launches);
  } else {
    if (q8) bwd<int8_t, float>(p, s, launches);
    else bwd<float, float>(p, s, launches);
  }
  return cudaGetLastError();
}

}  // namespace rcu
