// Selective scan: what its forward and backward passes share.
//
//   delta = softplus(dt + dt_bias), A2 = -exp(a_log) log2(e)
//   h_t[n] = 2^(delta A2[n]) h_{t-1}[n] + (delta x_t) b_t[n]
//
// The work is N exponentials and some 4 N products a step and channel against 8
// bytes moved in bf16, so the arithmetic units bound it, not the memory: the special
// function unit (32 exponentials a cycle and SM) and the issue of instructions.  So
// states are worked on as packed pairs, of two neighbouring channels: the pair's
// steps and inputs then lie beside one another, and what all channels share (b, c) is
// laid out twice.  What does not depend on the state (softplus, gates) is computed
// once for a tile of steps, in shared memory.
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

constexpr int CHUNK = RCU_SELSCAN_CHUNK;  // steps between kept states

__device__ __forceinline__ float max0(float v) {  // not fmaxf, which drops a NaN
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
  return r;
}
// softplus(v) = max(v, 0) + ln(1 + e), e = e^-|v|, with the relative precision of
// its small values: ln(1 + e) = s p(s^2), s = e / (2 + e), p a polynomial fitted to
// 2 artanh(s) / s over 0 <= s <= 1/3 with the least relative error (4e-9; 2e-7 as
// rounded).
__device__ __forceinline__ F2 softplus(F2 v) {
  const F2 e = f2(ex2(-LOG2E * fabsf(lo(v))), ex2(-LOG2E * fabsf(hi(v))));
  const F2 d = add2(e, f2(2.f)), s = mul2(e, f2(rcp(lo(d)), rcp(hi(d)))), q = mul2(s, s);
  F2 p = f2(0.2817833423614502f);
  p = fma2(p, q, f2(0.27960601449012756f));
  p = fma2(p, q, f2(0.40024909377098083f));
  p = fma2(p, q, f2(0.6666631698608398f));
  p = fma2(p, q, f2(2.f));
  return fma2(s, p, f2(max0(lo(v)), max0(hi(v))));
}
__device__ __forceinline__ float softplus(float v) { return lo(softplus(f2(v, v))); }
__device__ __forceinline__ F2 silu(F2 v) {
  return mul2(v, f2(sigmoid(lo(v)), sigmoid(hi(v))));
}

// -exp(a_log) log2(e), finite, so that a step of delta 0 leaves any state alone.
__device__ __forceinline__ float rate2(float a_log) {
  const float r = -LOG2E * expf(a_log);
  return r < -3e38f ? -3e38f : r;
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void *to, const void *from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "n"(BYTES) : "memory");
}

// A tile [TILE][CC] of a tensor's rows t0 .. and channels h0 .. (a multiple of 4) on its
// way to shared memory, all of it asynchronous: 16 bytes at a time where rows are aligned,
// 4 where they are not (T=512 B=16 H=1001 N=16: fp32 123 us, bf16 118; as plain values 451, 287).
// bf16 rows that start in the middle of a word are copied with the value before them, and
// lie one value further on (`shift`); that value is the tensor's or in front of its first,
// in the same 4 bytes.  What is past the row's end or the last channel keeps what was
// there, or is 0.  Made once for a block.
template <typename T, int NT, int TILE, int CC, bool ALIGNED>
struct Fetch {
  static constexpr bool SHIFTS = !ALIGNED && sizeof(T) == 2;
  static constexpr int RS = CC + (SHIFTS ? 4 : 0);                      // values of a row in shared memory
  static constexpr int V = (ALIGNED ? 16 : 4) / sizeof(T), ROW = CC / V;  // pieces of a row
  static constexpr int PASS = NT / ROW > 0 ? NT / ROW : 1;              // rows of a pass
  static constexpr int ACROSS = ROW > NT ? ROW / NT : 1;                // passes of a row
  static_assert(PASS * ROW == NT * ACROSS, "whole rows");
  const T *from;   // at the thread's row and channel of step 0
  int64_t st;
  int row, col, left;  // left: channels from the thread's on
  __device__ __forceinline__ Fetch(const T *p, int64_t st_, int h0, int width) : st(st_) {
    row = threadIdx.x / ROW, col = threadIdx.x % ROW * V;
    if (ROW > NT) row = 0, col = threadIdx.x * V;
    from = p + row * st + h0 + col;
    left = width - h0 - col;
  }
  // values that row `r` of the tile at t0 lies further on
  __device__ __forceinline__ int shift(int t0, int r) const {
    if constexpr (!SHIFTS) return 0;
    return (int)(reinterpret_cast<uintptr_t>(from + (t0 + r - row) * st) / 2 & 1);
  }
  __device__ __forceinline__ void start(T (*to)[RS], int t0, int end) const {
    const T *p = from + t0 * st;
    const int rows = end - t0 - row;  // of the thread's, that exist
#pragma unroll
    for (int k = 0; k < (TILE + PASS - 1) / PASS; ++k, p += PASS * st) {
      if (k * PASS >= rows || (TILE % PASS && k * PASS + row >= TILE)) break;
#pragma unroll
      for (int q = 0; q < ACROSS; ++q) {
        T *s = &to[k * PASS + row][col + q * NT * V];
        const T *g = p + q * NT * V;
        if constexpr (SHIFTS) {
          const int off = reinterpret_cast<uintptr_t>(g) / 2 & 1;
          word(s, g - off, left + off - q * NT * V);
          if (off && col + q * NT * V == CC - V) word(s + 2, g + 1, left - 1 - q * NT * V);
        } else {
          if (q * NT * V >= left) break;
          if constexpr (ALIGNED)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(s)),
                         "l"(g) : "memory");
          else
            copy_async<4>(s, g);
        }
      }
    }
  }
  // 4 bytes, of which the first `n` values are read
  static __device__ __forceinline__ void word(T *s, const T *g, int n) {
    if (n <= 0) return;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(s)),
                 "l"(g), "r"(n > 1 ? 4 : 2) : "memory");
  }
};
__device__ __forceinline__ void fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A tile's rows of b or c [TILE][N], read a tile ahead into registers, four neighbouring
// values at a time (`words`: as words), in fp32 in shared memory.
template <typename T, int NT, int TILE, int NP>
struct Weights {
  static constexpr int ROW = NP / 4, PASS = NT / ROW, EV = (TILE + PASS - 1) / PASS;
  static_assert(NT % ROW == 0, "whole rows");
  const T *from;
  int64_t st;
  int row, rows, left;  // rows: of the tile in v, from the thread's on, that exist
  bool words;
  Word<T, 4> v[EV];
  __device__ __forceinline__ Weights(const T *p, int64_t st_, int N, bool words_)
      : st(st_), rows(0), words(words_) {
    row = threadIdx.x / ROW;
    from = p + row * st + threadIdx.x % ROW * 4;
    left = N - (int)threadIdx.x % ROW * 4;
  }
  __device__ __forceinline__ void read(int t0, int end) {
    const T *p = from + t0 * st;
    rows = left > 0 ? end - t0 - row : 0;
#pragma unroll
    for (int k = 0; k < EV; ++k, p += PASS * st) {
      if (k * PASS >= rows) break;
      if (words) {
        v[k] = *reinterpret_cast<const Word<T, 4> *>(p);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < left) v[k].v[j] = p[j];
      }
    }
  }
  // NaN where one of them is not finite, else 0.
  __device__ __forceinline__ float put(float (*out)[NP]) const {
    float probe = 0.f;
#pragma unroll
    for (int k = 0; k < EV; ++k) {
      if (TILE % PASS && k * PASS + row >= TILE) break;
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = k * PASS < rows && j < left ? to_f(v[k].v[j]) : 0.f;
        probe = fmaf(w[j], 0.f, probe);
      }
      *reinterpret_cast<float4 *>(&out[k * PASS + row][threadIdx.x % ROW * 4]) =
          make_float4(w[0], w[1], w[2], w[3]);
    }
    return probe;
  }
};

// Two pairs: four neighbouring values of T.
struct Four {
  F2 a, b;
};
__device__ __forceinline__ Four four(const float *p) {
  const float4 v = *reinterpret_cast<const float4 *>(p);
  return {f2(v.x, v.y), f2(v.z, v.w)};
}
__device__ __forceinline__ Four four(const bf16 *p) {
  const Word<bf16, 4> v = *reinterpret_cast<const Word<bf16, 4> *>(p);
  return {f2(to_f(v.v[0]), to_f(v.v[1])), f2(to_f(v.v[2]), to_f(v.v[3]))};
}
// Of a row in shared memory, its first value at `row + shift` (Fetch).
template <bool SHIFTS, typename T>
__device__ __forceinline__ Four four(const T *row, int col, int shift) {
  if constexpr (SHIFTS) {
    const uint2 w = *reinterpret_cast<const uint2 *>(row + col);
    const uint32_t next = *reinterpret_cast<const uint32_t *>(row + col + 4);
    const uint32_t a = __funnelshift_r(w.x, w.y, 16 * shift), b = __funnelshift_r(w.y, next, 16 * shift);
    return {f2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u)),
            f2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u))};
  } else {
    return four(row + col);
  }
}
__device__ __forceinline__ void put_four(float *p, const Four &v) {
  *reinterpret_cast<float4 *>(p) = make_float4(lo(v.a), hi(v.a), lo(v.b), hi(v.b));
}
__device__ __forceinline__ void put_four(bf16 *p, const Four &v) {
  Word<bf16, 4> w;
  w.v[0] = from_f<bf16>(lo(v.a)), w.v[1] = from_f<bf16>(hi(v.a));
  w.v[2] = from_f<bf16>(lo(v.b)), w.v[3] = from_f<bf16>(hi(v.b));
  *reinterpret_cast<Word<bf16, 4> *>(p) = w;
}
// Four channels' constants [H], 0 where there are none.
__device__ __forceinline__ Four constants(const float *p, int h, int width) {
  float v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = p && h + k < width ? p[h + k] : 0.f;
  return {f2(v[0], v[1]), f2(v[2], v[3])};
}

// S states of [.., N] fp32 at p, `n` of them there.
template <int S>
__device__ __forceinline__ void load_states(const float *p, int n, bool wide, float (&v)[S]) {
  if (wide && n == S) {
#pragma unroll
    for (int k = 0; k < S; k += 4) {
      const float4 a = *reinterpret_cast<const float4 *>(p + k);
      v[k] = a.x, v[k + 1] = a.y, v[k + 2] = a.z, v[k + 3] = a.w;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < S; ++k) v[k] = k < n ? p[k] : 0.f;
}
template <int S>
__device__ __forceinline__ void store_states(float *p, int n, bool wide, const float (&v)[S]) {
  if (wide && n == S) {
#pragma unroll
    for (int k = 0; k < S; k += 4)
      *reinterpret_cast<float4 *>(p + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < S; ++k)
    if (k < n) p[k] = v[k];
}

// N neighbouring pairs of shared memory.
template <int N>
__device__ __forceinline__ void load_pairs(const float *p, F2 (&v)[N]) {
  if (N == 1) v[0] = *reinterpret_cast<const F2 *>(p);
#pragma unroll
  for (int k = 0; k + 1 < N; k += 2) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p + 2 * k);
    v[k] = a.x, v[k + 1] = a.y;
  }
}
__device__ __forceinline__ void load_row(const float *p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ F2 ex2_2(F2 v) { return f2(ex2(lo(v)), ex2(hi(v))); }

// How a sequence is split: segments of `len` steps (whole chunks).
struct Segments {
  int n, len;
};

// Segments of a sequence whose kernel takes `blocks` blocks a segment: some `per_sm`
// blocks an SM, of two chunks or more.  A split costs the first kernel, 0.6 of the
// main one's work on all segments but one, and two launches, so there is one only
// where an SM would have two blocks or fewer, of eight chunks or more.
//
// Measured, bf16, us, one segment -> split by this rule:
//   forward, H=1024 T=512: B=4 N=8 114 -> 36, N=16 80 -> 37, N=64 92 -> 95; B=8 N=16 80 -> 52;
//     B=16 N=4 122 -> 74, N=8 115 -> 74, N=16 82 -> 87, N=32 99 -> 140, N=64 179 -> 292;
//     T=2048 B=4 N=16 300 -> 91; H=2048 T=2048 B=8 N=8 440 -> 243, N=16 310 -> 288
//   where the rule has none and two segments are forced: T=300 B=32 N=16 70, 97; T=512 B=24 111, 126
//   backward, H=1024 T=512: B=4 N=8 233 -> 66, N=16 168 -> 86, N=64 264 -> 297; B=8 N=16 182 -> 152;
//     B=16 N=4 287 -> 224, N=8 285 -> 227, N=16 238 -> 277, N=32 and 64 no split (436, 969);
//     T=2048 B=4 N=16 712 -> 284; H=2048 T=2048 B=8 N=8 1093 -> 819, N=16 898 -> 1014
// So it is right for the few warps a block of N <= 8 up to its limit, and at N=16 up to some
// 130 blocks (forward, of long sequences, to 256); from there on, and with the more warps a
// block of more states, a split loses: the rule counts blocks, not warps.
inline Segments segments_of(int T, int64_t blocks, int nsm, int per_sm) {
  const int chunks = ceil_div(T, CHUNK);
  int n = 1;
  if (blocks <= 2 * nsm && chunks >= 8)
    n = (int)std::max<int64_t>(std::min<int64_t>((int64_t)per_sm * nsm / blocks, chunks / 2), 1);
  const int len = ceil_div(chunks, n) * CHUNK;
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

}  // namespace selscan
}  // namespace rcu
