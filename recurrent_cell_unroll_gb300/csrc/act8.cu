// 8-bit activation checkpoints: pack and unpack.
//
// Bound by memory.  A block of 64 values belongs to as many lanes as hold it in
// 16-byte words (8 of bf16, 16 of fp32): its largest magnitude is a maximum over
// those lanes, and the codes go out 8 or 4 bytes a lane.  Rows that are not
// 16-byte aligned, or not of whole words, go value by value, a warp a block.
// Measured: bf16 32768x2048 30 us to pack, 31 to unpack (5.9 TB/s together); the
// ALU pipe, with the conversions, is three quarters busy.
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

// Division of a word's index by a row's words.  Where rows lie one behind another
// and hold whole blocks (FLAT) the matrix is one long row and none is needed; else
// it is a multiplication by 2^32 / d, rounded up, which is exact as long as the
// index times d stays below 2^32 (larger products take the division itself).
struct Divide {
  uint32_t d, inv;
  bool quick;
  __device__ __forceinline__ int64_t operator()(int64_t i) const {
    return quick ? (int64_t)__umulhi((uint32_t)i, inv) : i / d;
  }
};
inline Divide divide(int64_t total, int d) {
  Divide v;
  v.d = (uint32_t)d;
  v.inv = (uint32_t)(((1ull << 32) + d - 1) / d);
  v.quick = d > 1 && (double)(total + 64) * d < 4294967296.0;
  return v;
}

constexpr int UNROLL = 4;  // words of a thread in flight

// The largest magnitude of a word's values as fp32 bits: as whole numbers the
// bits order like the magnitudes, with infinity and NaN above all.
__device__ __forceinline__ uint32_t top_bits(const uint4 &v, const float *) {
  const uint32_t m = 0x7fffffffu;
  return max(max(v.x & m, v.y & m), max(v.z & m, v.w & m));
}
__device__ __forceinline__ uint32_t top_bits(const uint4 &v, const bf16 *) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(a << 16, a & 0xffff0000u);
}
// Codes of finite values that all fit at the scale inv: adding 1.5 * 2^23 rounds
// to a whole number, to the nearest even, whose low byte is the code.
__device__ __forceinline__ uint32_t quick_code(float v, float inv) {
  return __float_as_uint(fmaf(v, inv, 12582912.f));
}
__device__ __forceinline__ uint32_t join4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
__device__ __forceinline__ void quick_codes(const uint4 &v, float inv, uint32_t (&w)[1],
                                            const float *) {
  w[0] = join4(quick_code(__uint_as_float(v.x), inv), quick_code(__uint_as_float(v.y), inv),
               quick_code(__uint_as_float(v.z), inv), quick_code(__uint_as_float(v.w), inv));
}
__device__ __forceinline__ void quick_codes(const uint4 &v, float inv, uint32_t (&w)[2],
                                            const bf16 *) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    q[2 * j] = quick_code(__uint_as_float(u[j] << 16), inv);
    q[2 * j + 1] = quick_code(__uint_as_float(u[j] & 0xffff0000u), inv);
  }
  w[0] = join4(q[0], q[1], q[2], q[3]);
  w[1] = join4(q[4], q[5], q[6], q[7]);
}

// Rows of whole words; the last block of a row may be short (whole words too).
template <typename T, bool FLAT>
__global__ void __launch_bounds__(NT)
    act8_pack_wide_kernel(Divide by_row, int64_t rows, int n, const T *__restrict__ x, int64_t ldx,
                          int8_t *__restrict__ codes, int64_t ldc, int8_t *__restrict__ exps) {
  constexpr int VEC = Wide<T>::VEC, LANES = Wide<T>::LANES;
  const int nb = ceil_div(n, BLOCK8);
  const int64_t total = rows * nb * LANES;  // words, with those a short block lacks
  // a warp's lanes stay in step: the maxima below are over lanes of one warp
  for (int64_t first = ((int64_t)blockIdx.x * UNROLL) * NT + threadIdx.x;
       first - threadIdx.x % 32 < total; first += (int64_t)gridDim.x * UNROLL * NT) {
    uint4 raw[UNROLL];
    int64_t row[UNROLL];
    int c[UNROLL];
#pragma unroll
    for (int q = 0; q < UNROLL; ++q) {
      const int64_t id = first + q * NT, blk = id / LANES;
      row[q] = FLAT ? 0 : by_row(blk);
      c[q] = (int)(blk - row[q] * nb) * BLOCK8 + (int)(id % LANES) * VEC;
      raw[q] = make_uint4(0, 0, 0, 0);
      if (id < total && (FLAT || c[q] < n))
        raw[q] = __ldg(reinterpret_cast<const uint4 *>(FLAT ? x + id * VEC : x + row[q] * ldx + c[q]));
    }
#pragma unroll
    for (int q = 0; q < UNROLL; ++q) {
      const int64_t id = first + q * NT;
      uint32_t top = top_bits(raw[q], static_cast<const T *>(nullptr));
#pragma unroll
      for (int o = LANES / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      // not finite, or above the largest scale: value by value (a block's lanes together)
      const bool plain = top <= __float_as_uint(127.f * power2(121));
      if (__any_sync(0xffffffffu, !plain)) {
        float most = 0.f;
        const T *v = reinterpret_cast<const T *>(&raw[q]);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (isfinite(to_f(v[j]))) most = fmaxf(most, fabsf(to_f(v[j])));
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1)
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        top = __float_as_uint(most);
      }
      const int e = act8_exponent(__uint_as_float(top));
      if (id >= total || (!FLAT && c[q] >= n)) continue;
      uint32_t w[VEC / 4];
      if (plain) {
        quick_codes(raw[q], power2(-e), w, static_cast<const T *>(nullptr));
      } else {
        const T *v = reinterpret_cast<const T *>(&raw[q]);
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
          w[k] = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[k] |= (uint32_t)(act8_code(to_f(v[4 * k + j]), power2(-e)) & 0xff) << (8 * j);
        }
      }
      store_codes(FLAT ? codes + id * VEC : codes + row[q] * ldc + c[q], w);
      if (id % LANES == 0) exps[id / LANES] = (int8_t)e;
    }
  }
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(NT)
    act8_unpack_wide_kernel(Divide by_row, int64_t rows, int n, const int8_t *__restrict__ codes,
                            int64_t ldc, const int8_t *__restrict__ exps, T *__restrict__ y,
                            int64_t ldy) {
  constexpr int VEC = Wide<T>::VEC, LANES = Wide<T>::LANES;
  const int nw = n / VEC, nb = ceil_div(n, BLOCK8);
  const int64_t total = rows * nw;
  for (int64_t first = ((int64_t)blockIdx.x * UNROLL) * NT + threadIdx.x; first < total;
       first += (int64_t)gridDim.x * UNROLL * NT) {
    uint32_t w[UNROLL][VEC / 4];
    int64_t to[UNROLL];
    int e[UNROLL];
#pragma unroll
    for (int q = 0; q < UNROLL; ++q) {
      const int64_t id = first + q * NT;
      if (id >= total) break;
      const int64_t row = FLAT ? 0 : by_row(id);
      const int c = (int)(id - row * nw) * VEC;
      to[q] = FLAT ? id * VEC : row * ldy + c;
      load_codes(codes + (FLAT ? id * VEC : row * ldc + c), w[q]);
      e[q] = __ldg(exps + (FLAT ? id / LANES : row * nb + c / BLOCK8));
    }
#pragma unroll
    for (int q = 0; q < UNROLL; ++q) {
      if (first + q * NT >= total) break;
      uint4 raw;
      T *v = reinterpret_cast<T *>(&raw);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        v[j] = from_f<T>(act8_value((int8_t)(w[q][j / 4] >> (8 * (j % 4))), e[q]));
      *reinterpret_cast<uint4 *>(y + to[q]) = raw;
    }
  }
}

// Value by value: a warp has UNROLL blocks at once, two values of each a lane.
template <typename T>
__global__ void __launch_bounds__(NT)
    act8_pack_kernel(Divide by_row, int64_t rows, int n, const T *__restrict__ x, int64_t ldx,
                     int8_t *__restrict__ codes, int64_t ldc, int8_t *__restrict__ exps) {
  const int nb = ceil_div(n, BLOCK8), lane = threadIdx.x % 32;
  const int64_t total = rows * nb;
  for (int64_t id = ((int64_t)blockIdx.x * (NT / 32) + threadIdx.x / 32) * UNROLL; id < total;
       id += (int64_t)gridDim.x * (NT / 32) * UNROLL) {
    float v[UNROLL][2];
    int64_t row[UNROLL];
    int c0[UNROLL];
#pragma unroll
    for (int q = 0; q < UNROLL; ++q) {
      row[q] = by_row(id + q);
      c0[q] = id + q < total ? (int)(id + q - row[q] * nb) * BLOCK8 : n;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = c0[q] + 32 * j + lane;
        v[q][j] = c < n ? to_f(x[row[q] * ldx + c]) : 0.f;
      }
    }
#pragma unroll
    for (int q = 0; q < UNROLL; ++q) {
      uint32_t top = 0;  // fp32 bits order like the magnitudes
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (isfinite(v[q][j])) top = max(top, __float_as_uint(v[q][j]) & 0x7fffffffu);
      const int e = act8_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, top)));
      const float inv = power2(-e);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = c0[q] + 32 * j + lane;
        if (c < n) codes[row[q] * ldc + c] = (int8_t)act8_code(v[q][j], inv);
      }
      if (lane == 0 && c0[q] < n) exps[id + q] = (int8_t)e;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(NT)
    act8_unpack_kernel(Divide by_row, int64_t rows, int n, const int8_t *__restrict__ codes,
                       int64_t ldc, const int8_t *__restrict__ exps, T *__restrict__ y,
                       int64_t ldy) {
  const int nb = ceil_div(n, BLOCK8), lane = threadIdx.x % 32;
  const int64_t total = rows * nb;
  for (int64_t id = ((int64_t)blockIdx.x * (NT / 32) + threadIdx.x / 32) * UNROLL; id < total;
       id += (int64_t)gridDim.x * (NT / 32) * UNROLL) {
    int code[UNROLL][2], e[UNROLL], c0[UNROLL];
    int64_t row[UNROLL];
#pragma unroll
    for (int q = 0; q < UNROLL; ++q) {
      row[q] = by_row(id + q);
      c0[q] = id + q < total ? (int)(id + q - row[q] * nb) * BLOCK8 : n;
      e[q] = c0[q] < n ? exps[id + q] : 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = c0[q] + 32 * j + lane;
        code[q][j] = c < n ? codes[row[q] * ldc + c] : 0;
      }
    }
#pragma unroll
    for (int q = 0; q < UNROLL; ++q)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = c0[q] + 32 * j + lane;
        if (c < n) y[row[q] * ldy + c] = from_f<T>(act8_value(code[q][j], e[q]));
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
  const int64_t words = rows * nb * Wide<T>::LANES;
  const int grid = grid_for((words + UNROLL - 1) / UNROLL, nsm);
  if (!vec || n % VEC || !aligned(x, ldx, sizeof(T), 16) || !aligned(codes, ldc, 1, VEC))
    act8_pack_kernel<T><<<grid_for((rows * nb + UNROLL - 1) / UNROLL * 32, nsm), NT, 0, s>>>(
        divide(rows * nb, nb), rows, n, x, ldx, codes, ldc, exps);
  else if (n % BLOCK8 == 0 && ldx == n && ldc == n)
    act8_pack_wide_kernel<T, true><<<grid, NT, 0, s>>>(Divide{}, rows, n, x, ldx, codes, ldc, exps);
  else
    act8_pack_wide_kernel<T, false><<<grid, NT, 0, s>>>(divide(rows * nb, nb), rows, n, x, ldx,
                                                        codes, ldc, exps);
}
template <typename T>
void unpack(int64_t rows, int n, const int8_t *codes, int64_t ldc, const int8_t *exps, T *y,
            int64_t ldy, int nsm, bool vec, cudaStream_t s) {
  constexpr int VEC = Wide<T>::VEC;
  const int nb = ceil_div(n, BLOCK8);
  const int64_t words = rows * (n / VEC);
  const int grid = grid_for((words + UNROLL - 1) / UNROLL, nsm);
  if (!vec || n % VEC || !aligned(y, ldy, sizeof(T), 16) || !aligned(codes, ldc, 1, VEC))
    act8_unpack_kernel<T><<<grid_for((rows * nb + UNROLL - 1) / UNROLL * 32, nsm), NT, 0, s>>>(
        divide(rows * nb, nb), rows, n, codes, ldc, exps, y, ldy);
  else if (n % BLOCK8 == 0 && ldy == n && ldc == n)
    act8_unpack_wide_kernel<T, true><<<grid, NT, 0, s>>>(Divide{}, rows, n, codes, ldc, exps, y,
                                                         ldy);
  else
    act8_unpack_wide_kernel<T, false><<<grid, NT, 0, s>>>(divide(words, n / VEC), rows, n, codes,
                                                          ldc, exps, y, ldy);
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
