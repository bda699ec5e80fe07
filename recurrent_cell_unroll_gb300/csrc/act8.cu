// 8-bit activation checkpoints: pack and unpack (include/rcu.h has the format).
#include "common.cuh"
#include "linrec_math.cuh"
#include "rcu.h"
#include "seq.h"

namespace rcu {
namespace {

using bf16 = __nv_bfloat16;
using linrec::from_f;
using linrec::to_f;

constexpr int BLOCK8 = RCU_ACT8_BLOCK;
constexpr int NT = 256;

// The smallest e in [-126, 121] with top <= 127 * 2^e (top >= 0, finite).
// top = m * 2^k with m in [1, 2): 127 * 2^e reaches it for e = k - 6 exactly
// when m * 64 <= 127, that is when the fraction is at most 63/64.  At e = 122
// a code of 64 would already stand for infinity, so e stops at 121 and the
// codes of a larger top at 127.
__device__ __forceinline__ int exponent8(float top) {
  const int bits = __float_as_int(top);
  const int e = (bits >> 23) - 127 - 6 + ((bits & 0x7fffff) > 0x7e0000);
  return min(max(e, -126), 121);
}
__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }

// The code of v at the scale inv = 2^-e.
__device__ __forceinline__ int code8(float v, float inv) {
  return isfinite(v) ? min(max(__float2int_rn(v * inv), -127), 127) : -128;
}

template <typename T>
__global__ void act8_pack_kernel(int64_t rows, int n, const T *x, int64_t ldx, int8_t *codes,
                                 int64_t ldc, int8_t *exps) {
  const int nb = ceil_div(n, BLOCK8), lane = threadIdx.x % 32;
  const int64_t id = (int64_t)blockIdx.x * (NT / 32) + threadIdx.x / 32;  // a warp per block
  if (id >= rows * nb) return;
  const int64_t row = id / nb;
  const int c0 = (int)(id % nb) * BLOCK8;
  float v[2], top = 0.f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = c0 + 32 * j + lane;
    v[j] = c < n ? to_f(x[row * ldx + c]) : 0.f;
    if (isfinite(v[j])) top = fmaxf(top, fabsf(v[j]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int e = exponent8(top);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = c0 + 32 * j + lane;
    if (c < n)
      codes[row * ldc + c] = (int8_t)code8(v[j], power2(-e));
  }
  if (lane == 0) exps[id] = (int8_t)e;
}

template <typename T>
__global__ void act8_unpack_kernel(int64_t rows, int n, const int8_t *codes, int64_t ldc,
                                   const int8_t *exps, T *y, int64_t ldy) {
  const int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (id >= rows * n) return;
  const int64_t row = id / n;
  const int c = (int)(id % n);
  const int code = codes[row * ldc + c];
  const float v = code == -128 ? __int_as_float(0x7fc00000)
                               : code * power2(exps[row * ceil_div(n, BLOCK8) + c / BLOCK8]);
  y[row * ldy + c] = from_f<T>(v);
}

}  // namespace

cudaError_t launch_act8_pack(int dtype, int64_t rows, int n, const void *x, int64_t ldx,
                             int8_t *codes, int64_t ldc, int8_t *exps, int, bool, cudaStream_t s,
                             int *launches) {
  const unsigned grid = (unsigned)((rows * ceil_div(n, BLOCK8) + NT / 32 - 1) / (NT / 32));
  if (dtype == RCU_BF16)
    act8_pack_kernel<bf16><<<grid, NT, 0, s>>>(rows, n, (const bf16 *)x, ldx, codes, ldc, exps);
  else
    act8_pack_kernel<float><<<grid, NT, 0, s>>>(rows, n, (const float *)x, ldx, codes, ldc, exps);
  ++*launches;
  return cudaGetLastError();
}

cudaError_t launch_act8_unpack(int dtype, int64_t rows, int n, const int8_t *codes, int64_t ldc,
                               const int8_t *exps, void *y, int64_t ldy, int, bool, cudaStream_t s,
                               int *launches) {
  const unsigned grid = (unsigned)((rows * n + NT - 1) / NT);
  if (dtype == RCU_BF16)
    act8_unpack_kernel<bf16><<<grid, NT, 0, s>>>(rows, n, codes, ldc, exps, (bf16 *)y, ldy);
  else
    act8_unpack_kernel<float><<<grid, NT, 0, s>>>(rows, n, codes, ldc, exps, (float *)y, ldy);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace rcu
