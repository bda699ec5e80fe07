// 8-bit activation checkpoints: pack and unpack.
//
// Bound by memory.  A block of 64 values belongs to as many lanes as hold it in
// 16-byte words (8 of bf16, 16 of fp32): its largest magnitude is a maximum over
// those lanes, and the codes go out 8 or 4 bytes a lane.  Rows that are not
// 16-byte aligned, or end inside a block, go value by value, a warp a block.
#include <algorithm>

#include "act8.cuh"
#include "common.cuh"
#include "linrec_math.cuh"
#include "seq.h"

namespace rcu {
namespace {

using bf16 = __nv_bfloat16;
using linrec::from_f;
using linrec::to_f;

constexpr int BLOCK8 = RCU_ACT8_BLOCK;
constexpr int NT = 256;

template <typename T>
struct Wide {  // a 16-byte word of values, and the codes of it
  static constexpr int VEC = 16 / (int)sizeof(T), LANES = BLOCK8 / VEC;
};
__device__ __forceinline__ void store_codes(int8_t *p, const uint32_t (&w)[1]) {
  *reinterpret_cast<uint32_t *>(p) = w[0];
}
__device__ __forceinline__ void store_codes(int8_t *p, const uint32_t (&w)[2]) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void load_codes(const int8_t *p, uint32_t (&w)[1]) {
  w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
}
__device__ __forceinline__ void load_codes(const int8_t *p, uint32_t (&w)[2]) {
  const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
  w[0] = v.x, w[1] = v.y;
}

// Rows of whole words; the last block of a row may be short (whole words too).
template <typename T>
__global__ void __launch_bounds__(NT)
    act8_pack_wide_kernel(int64_t rows, int n, const T *__restrict__ x, int64_t ldx,
                          int8_t *__restrict__ codes, int64_t ldc, int8_t *__restrict__ exps) {
  constexpr int VEC = Wide<T>::VEC, LANES = Wide<T>::LANES;
  const int nb = ceil_div(n, BLOCK8);
  const int64_t total = rows * nb * LANES;  // words, with those a short block lacks
  for (int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x; id - threadIdx.x % 32 < total;
       id += (int64_t)gridDim.x * NT) {
    const int64_t blk = id / LANES, row = blk / nb;
    const int c = (int)(blk % nb) * BLOCK8 + (int)(id % LANES) * VEC;
    const bool on = id < total && c < n;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (on) raw = __ldg(reinterpret_cast<const uint4 *>(x + row * ldx + c));
    const T *v = reinterpret_cast<const T *>(&raw);
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float a = fabsf(to_f(v[j]));
      if (a < __int_as_float(0x7f800000)) top = fmaxf(top, a);
    }
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = act8_exponent(top);
    const float inv = power2(-e);
    if (!on) continue;
    uint32_t w[VEC / 4];
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
      w[q] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[q] |= (uint32_t)(act8_code(to_f(v[4 * q + j]), inv) & 0xff) << (8 * j);
    }
    store_codes(codes + row * ldc + c, w);
    if (id % LANES == 0) exps[blk] = (int8_t)e;
  }
}

template <typename T>
__global__ void __launch_bounds__(NT)
    act8_unpack_wide_kernel(int64_t rows, int n, const int8_t *__restrict__ codes, int64_t ldc,
                            const int8_t *__restrict__ exps, T *__restrict__ y, int64_t ldy) {
  constexpr int VEC = Wide<T>::VEC;
  const int nw = n / VEC, nb = ceil_div(n, BLOCK8);
  const int64_t total = rows * nw;
  for (int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x; id < total;
       id += (int64_t)gridDim.x * NT) {
    const int64_t row = id / nw;
    const int c = (int)(id % nw) * VEC;
    uint32_t w[VEC / 4];
    load_codes(codes + row * ldc + c, w);
    const int e = __ldg(exps + row * nb + c / BLOCK8);
    uint4 raw;
    T *v = reinterpret_cast<T *>(&raw);
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      v[j] = from_f<T>(act8_value((int8_t)(w[j / 4] >> (8 * (j % 4))), e));
    *reinterpret_cast<uint4 *>(y + row * ldy + c) = raw;
  }
}

template <typename T>
__global__ void __launch_bounds__(NT)
    act8_pack_kernel(int64_t rows, int n, const T *__restrict__ x, int64_t ldx,
                     int8_t *__restrict__ codes, int64_t ldc, int8_t *__restrict__ exps) {
  const int nb = ceil_div(n, BLOCK8), lane = threadIdx.x % 32;
  for (int64_t id = (int64_t)blockIdx.x * (NT / 32) + threadIdx.x / 32; id < rows * nb;
       id += (int64_t)gridDim.x * (NT / 32)) {  // a warp per block
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
    const int e = act8_exponent(top);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = c0 + 32 * j + lane;
      if (c < n) codes[row * ldc + c] = (int8_t)act8_code(v[j], power2(-e));
    }
    if (lane == 0) exps[id] = (int8_t)e;
  }
}

template <typename T>
__global__ void __launch_bounds__(NT)
    act8_unpack_kernel(int64_t rows, int n, const int8_t *__restrict__ codes, int64_t ldc,
                       const int8_t *__restrict__ exps, T *__restrict__ y, int64_t ldy) {
  const int nb = ceil_div(n, BLOCK8), lane = threadIdx.x % 32;
  for (int64_t id = (int64_t)blockIdx.x * (NT / 32) + threadIdx.x / 32; id < rows * nb;
       id += (int64_t)gridDim.x * (NT / 32)) {
    const int64_t row = id / nb;
    const int c0 = (int)(id % nb) * BLOCK8, e = exps[id];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = c0 + 32 * j + lane;
      if (c < n) y[row * ldy + c] = from_f<T>(act8_value(codes[row * ldc + c], e));
    }
  }
}

// Blocks for `threads` threads, at most 16 on an SM: each then takes more.
int grid_for(int64_t threads, int nsm) {
  return (int)std::min<int64_t>((threads + NT - 1) / NT, 16 * nsm);
}

bool aligned(const void *p, int64_t ld, int size, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * size % bytes == 0;
}

template <typename T>
void pack(int64_t rows, int n, const T *x, int64_t ldx, int8_t *codes, int64_t ldc, int8_t *exps,
          int nsm, bool vec, cudaStream_t s) {
  constexpr int VEC = Wide<T>::VEC;
  const int nb = ceil_div(n, BLOCK8);
  if (vec && n % VEC == 0 && aligned(x, ldx, sizeof(T), 16) && aligned(codes, ldc, 1, VEC))
    act8_pack_wide_kernel<T><<<grid_for(rows * nb * Wide<T>::LANES, nsm), NT, 0, s>>>(
        rows, n, x, ldx, codes, ldc, exps);
  else
    act8_pack_kernel<T><<<grid_for(rows * nb * 32, nsm), NT, 0, s>>>(rows, n, x, ldx, codes, ldc,
                                                                      exps);
}
template <typename T>
void unpack(int64_t rows, int n, const int8_t *codes, int64_t ldc, const int8_t *exps, T *y,
            int64_t ldy, int nsm, bool vec, cudaStream_t s) {
  constexpr int VEC = Wide<T>::VEC;
  if (vec && n % VEC == 0 && aligned(y, ldy, sizeof(T), 16) && aligned(codes, ldc, 1, VEC))
    act8_unpack_wide_kernel<T><<<grid_for(rows * (n / VEC), nsm), NT, 0, s>>>(rows, n, codes, ldc,
                                                                             exps, y, ldy);
  else
    act8_unpack_kernel<T><<<grid_for(rows * ceil_div(n, BLOCK8) * 32, nsm), NT, 0, s>>>(
        rows, n, codes, ldc, exps, y, ldy);
}

}  // namespace

cudaError_t launch_act8_pack(int dtype, int64_t rows, int n, const void *x, int64_t ldx,
                             int8_t *codes, int64_t ldc, int8_t *exps, int nsm, bool vec,
                             cudaStream_t s, int *launches) {
  if (dtype == RCU_BF16)
    pack<bf16>(rows, n, static_cast<const bf16 *>(x), ldx, codes, ldc, exps, nsm, vec, s);
  else
    pack<float>(rows, n, static_cast<const float *>(x), ldx, codes, ldc, exps, nsm, vec, s);
  ++*launches;
  return cudaGetLastError();
}

cudaError_t launch_act8_unpack(int dtype, int64_t rows, int n, const int8_t *codes, int64_t ldc,
                               const int8_t *exps, void *y, int64_t ldy, int nsm, bool vec,
                               cudaStream_t s, int *launches) {
  if (dtype == RCU_BF16)
    unpack<bf16>(rows, n, codes, ldc, exps, static_cast<bf16 *>(y), ldy, nsm, vec, s);
  else
    unpack<float>(rows, n, codes, ldc, exps, static_cast<float *>(y), ldy, nsm, vec, s);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace rcu
