// Pieces of the layer norm kernels (layernorm_fwd.cu, layernorm_bwd.cu).
#pragma once

#include <algorithm>

#include "act8.cuh"
#include "common.cuh"
#include "linrec_math.cuh"
#include "per_device.h"
#include "rcu.h"
#include "seq.h"

namespace rcu {
namespace ln {

using bf16 = __nv_bfloat16;
using linrec::from_f;
using linrec::to_f;

// ---- VEC consecutive values as they lie in memory

template <int BYTES>
struct Raw;
template <>
struct Raw<16> { typedef uint4 type; };
template <>
struct Raw<8> { typedef uint2 type; };
template <>
struct Raw<4> { typedef uint32_t type; };
template <>
struct Raw<2> { typedef unsigned short type; };
template <>
struct Raw<1> { typedef unsigned char type; };

template <typename T, int VEC>
struct Vals {
  typename Raw<VEC * (int)sizeof(T)>::type raw;
  __device__ __forceinline__ void load(const T *p) {
    raw = __ldg(reinterpret_cast<const decltype(raw) *>(p));
  }
  __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<decltype(raw) *>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = decltype(raw){}; }
  __device__ __forceinline__ void block(const int8_t *) {}
  __device__ __forceinline__ float operator[](int j) const {
    return to_f(reinterpret_cast<const T *>(&raw)[j]);
  }
  __device__ __forceinline__ void set(int j, float v) {
    reinterpret_cast<T *>(&raw)[j] = from_f<T>(v);
  }
  __device__ __forceinline__ void decode(float (&f)[VEC]) const {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = (*this)[j];
  }
};
// 8-bit codes with their block's exponent (VEC divides the block)
template <int VEC>
struct Vals<int8_t, VEC> {
  typename Raw<VEC>::type raw;
  int8_t e;
  __device__ __forceinline__ void load(const int8_t *p) {
    raw = __ldg(reinterpret_cast<const decltype(raw) *>(p));
  }
  __device__ __forceinline__ void zero() { raw = decltype(raw){}, e = 0; }
  __device__ __forceinline__ void block(const int8_t *p) { e = __ldg(p); }
  __device__ __forceinline__ void decode(float (&f)[VEC]) const {
    const float scale = power2(e);
    if (VEC == 1) {
      f[0] = act8_value((int8_t)*reinterpret_cast<const unsigned char *>(&raw), e);
      return;
    }
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&raw);
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[4 * q + j] = act8_whole(w[q], j) * scale;
      if (act8_any_nan(w[q])) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f[4 * q + j] = act8_value((int8_t)(w[q] >> (8 * j)), e);
      }
    }
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sums of a and b over a row's W warps, the same in all of them.  Warp w of
// the row writes its part; `buf` alternates, so one barrier a sum is enough, and
// it is the row's own (a block's rows do not wait for one another).
template <int W>
__device__ __forceinline__ void row_sum(float &a, float &b, float2 (*part)[32], int &buf) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (W > 1) {
    const int warp = threadIdx.x / 32;
    if (threadIdx.x % 32 == 0) part[buf][warp] = make_float2(a, b);
    asm volatile("barrier.sync %0, %1;" ::"r"(warp / W + 1), "r"(32 * W) : "memory");
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 v = part[buf][warp / W * W + w];
      a += v.x;
      b += v.y;
    }
    buf ^= 1;
  }
}

// the sum over a block of LONG_NT threads
constexpr int LONG_NT = 512;
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[LONG_NT / 32];
  v = warp_sum(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < LONG_NT / 32; ++w) v += part[w];
  return v;
}

// ---- host side

constexpr int VEC_F32 = 4, VEC_BF16 = 8;  // values of a 16-byte word

// Whether rows of this operand start on multiples of `bytes` (NULL: no matter).
inline bool aligned(const void *p, int64_t ld, int size, int bytes) {
  return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * size % bytes == 0);
}

// Blocks of a kernel that fit on the GPU at once.
template <typename... KArgs>
int resident_blocks(void (*fn)(KArgs...), int threads, size_t smem, int nsm) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return std::max(1, n) * nsm;
}

}  // namespace ln
}  // namespace rcu
