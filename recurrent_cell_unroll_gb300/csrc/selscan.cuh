// Selective scan: what its forward and backward passes share.
//
//   delta = softplus(dt + dt_bias), A2 = -exp(a_log) log2(e)
//   h_t[n] = 2^(delta A2[n]) h_{t-1}[n] + (delta x_t) b_t[n]
//
// The work is N exponentials and some 4 N products a step and channel against 8
// bytes moved in bf16, so the arithmetic units bound it, not the memory.  A thread
// keeps 8 states of a channel in registers, and LANES = N / 8 threads that stand
// side by side in a warp make up the channel; what does not depend on the state
// (softplus, gates) is computed once for a tile of TILE steps and put into shared
// memory, as are the tile's rows of b and c, which all channels read.  States are
// computed as packed pairs.
//
// Long sequences of few channels are split over time into segments: a first
// kernel finds each segment's last states from states of 0 and its sum of delta
// (a segment's decay is 2^(A2 sum)), a second one chains them, and the main
// kernel starts every segment with the states that enter it.
#pragma once

#include <initializer_list>
#include <type_traits>

#include "per_device.h"
#include "ssm_common.cuh"

namespace rcu {
namespace selscan {

using namespace ssm;

constexpr int S = 8;                       // states of a thread
constexpr int TILE = RCU_SELSCAN_CHUNK;    // steps of a tile

// ln(1 + e) for 0 <= e <= 1 with its relative precision.
__device__ __forceinline__ float log1p_small(float e) { return log1pf(e); }
// softplus(v) = max(v, 0) + ln(1 + e^-|v|)
__device__ __forceinline__ float softplus(float v) {
  float top;  // not fmaxf, which drops a NaN
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(top) : "f"(v));
  return top + log1p_small(ex2(-LOG2E * fabsf(v)));
}

// -exp(a_log) log2(e), finite, so that a step of delta 0 leaves any state alone.
__device__ __forceinline__ float rate2(float a_log) {
  const float r = -LOG2E * expf(a_log);
  return r < -3e38f ? -3e38f : r;
}

// A tile's tensor [TILE][CC] of a block's channels, read a tile ahead into
// registers: EV words of VE values a thread (VE = 1: rows that are not aligned).
template <typename T, int NT, int CC, int VE>
struct Ahead {
  static constexpr int EV = TILE * CC / (NT * VE);
  static constexpr int PER_ROW = CC / VE;
  Word<T, VE> w[EV];
  __device__ __forceinline__ static int row(int k) { return (k * NT + (int)threadIdx.x) / PER_ROW; }
  __device__ __forceinline__ static int col(int k) { return (k * NT + (int)threadIdx.x) % PER_ROW * VE; }
  // rows t0 .. t0 + TILE that are before `end`, channels before `width`
  __device__ __forceinline__ void read(const T *p, int64_t st, int t0, int end, int h0, int width) {
#pragma unroll
    for (int k = 0; k < EV; ++k) {
      const int t = t0 + row(k), h = h0 + col(k);
      if (t < end && h < width) w[k] = *reinterpret_cast<const Word<T, VE> *>(p + t * st + h);
    }
  }
};

// The same of b or c [TILE][N], single values.
template <typename T, int NT, int NP>
struct AheadRows {
  static constexpr int EV = (TILE * NP + NT - 1) / NT;
  T v[EV];
  __device__ __forceinline__ void read(const T *p, int64_t st, int t0, int end, int N) {
#pragma unroll
    for (int k = 0; k < EV; ++k) {
      const int at = k * NT + threadIdx.x, t = at / NP, n = at % NP;
      if (t < TILE && t0 + t < end && n < N) v[k] = p[(t0 + t) * st + n];
    }
  }
  __device__ __forceinline__ void put(float (*out)[NP], int t0, int end, int N) const {
#pragma unroll
    for (int k = 0; k < EV; ++k) {
      const int at = k * NT + threadIdx.x, t = at / NP, n = at % NP;
      if (t < TILE) out[t][n] = t0 + t < end && n < N ? to_f(v[k]) : 0.f;
    }
  }
};

// 8 states of [.., N] fp32 at p, `n` of them there.
__device__ __forceinline__ void load_states(const float *p, int n, bool wide, float (&v)[S]) {
  if (wide && n == S) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
#pragma unroll
  for (int k = 0; k < S; ++k) v[k] = k < n ? p[k] : 0.f;
}
__device__ __forceinline__ void store_states(float *p, int n, bool wide, const float (&v)[S]) {
  if (wide && n == S) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
#pragma unroll
  for (int k = 0; k < S; ++k)
    if (k < n) p[k] = v[k];
}

// Two neighbouring values of shared memory as a pair.
__device__ __forceinline__ void load_pairs(const float *p, F2 (&v)[S / 2]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p);
  const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
__device__ __forceinline__ F2 ex2_2(F2 v) { return f2(ex2(lo(v)), ex2(hi(v))); }

// v[t] of LANES steps summed over the channel's LANES lanes; lane l gets step l's.
template <int LANES>
__device__ __forceinline__ float sum_over_lanes(float (&v)[LANES], int lane) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o /= 2)
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float keep = lane & o ? v[j + o] : v[j], give = lane & o ? v[j] : v[j + o];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  return v[0];
}

// How a sequence is split: segments of `len` steps (whole tiles).
struct Segments {
  int n, len;
};

// Segments so that `blocks` blocks a segment make `want` in all, of 4 tiles at
// least.  A split costs the first kernel, some 0.6 of the main one's work.
inline Segments segments_of(int T, int64_t blocks, int64_t want) {
  const int tiles = ceil_div(T, TILE);
  int n = 1;
  if (blocks * 2 <= want) n = (int)std::min<int64_t>(want / blocks, std::max(tiles / 4, 1));
  const int len = ceil_div(tiles, n) * TILE;
  return {ceil_div(T, len), len};
}

// Where a segment's kernel meets the others: end [n][B][H][N] (last states, then
// the states that enter), sums [n][B][H] of delta.
struct Meeting {
  Segments seg;
  float *end, *sums;
};

// The local pass and the chaining of segments (selscan_fwd.cu); backwards they
// chain gradients of the states, with `dy` and c in the place of delta x and b.
cudaError_t launch_local(const ScanIn &p, bool backwards, const SeqIn &dy, const float *first,
                         const Meeting &m, int *err, bool vec, cudaStream_t s, int *launches);

inline int lanes_of(int N) { return N <= 8 ? 1 : N <= 16 ? 2 : N <= 32 ? 4 : 8; }

template <typename F>
cudaError_t by_lanes(int N, F f) {
  switch (lanes_of(N)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    default: return f(std::integral_constant<int, 8>());
  }
}

}  // namespace selscan
}  // namespace rcu
