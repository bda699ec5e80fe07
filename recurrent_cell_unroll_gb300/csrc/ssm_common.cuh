// Device helpers that the selective state space kernels share.
#pragma once

#include "common.cuh"
#include "linrec_math.cuh"
#include "ssm.h"

namespace rcu {
namespace ssm {

using linrec::F2;
using linrec::LOG2E;
using linrec::add2;
using linrec::ex2;
using linrec::f2;
using linrec::fma2;
using linrec::from_f;
using linrec::hi;
using linrec::lo;
using linrec::mul2;
using linrec::rcp;
using linrec::to_f;
typedef __nv_bfloat16 bf16;

template <typename T, int N>
struct alignas(N * sizeof(T)) Word {
  T v[N];
};

// sigmoid(v) = 1 / (1 + e^-v): exact at infinite v
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-LOG2E * v)); }

// The steps of row b that take part; a length out of range is clamped and reported.
__device__ __forceinline__ int row_length(const int32_t *lengths, int b, int T, int *err) {
  if (!lengths) return T;
  const int n = lengths[b];
  if (n < 0 || n > T) {
    atomicCAS(err, (int)DEV_OK, (int)DEV_LENGTHS);
    return min(max(n, 0), T);
  }
  return n;
}

// Whether rows from p on, `stride` elements apart, can be read as words of n.
inline bool aligned(const void *p, int64_t stride, int size, int n) {
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)(size * n) == 0 && stride % n == 0;
}
inline bool aligned(const SeqIn &v, int size, int n) {
  return aligned(v.p, v.st, size, n) && v.sb % n == 0;
}
inline bool aligned(const SeqOut &v, int size, int n) {
  return aligned(v.p, v.st, size, n) && v.sb % n == 0;
}

}  // namespace ssm
}  // namespace rcu
