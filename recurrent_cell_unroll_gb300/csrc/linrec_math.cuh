// Elementwise mathematics of the gated linear recurrence, shared by its
// forward, backward and single-step kernels.
//
// Per element, with K = c softplus(lambda) of its channel:
//   s = sigmoid(r), g = sigmoid(i), a = exp(-K s), w = 1 - a^2, beta = sqrt(w)
//   h_t = a h_{t-1} + beta g x
// a lies near 1 (a state remembers for 1 / (1 - a) steps), so what is kept is
// em1 = a - 1, computed as expm1 without cancellation:
//   a h + b  =  h + (em1 h + b)        the decay keeps its relative precision
//   w = 1 - a^2 = -em1 (2 + em1)       and so does the input's scale
// An a rounded to fp32 has a step of 6e-8; times 2000 steps of memory that was
// measured as an error of 7e-6 in dh0, against 1e-6 in this form.  (The products of
// several steps' decays are plain fp32: what is lost there shows where a state
// remembers for millions of steps.)
//
// The forward in bf16 moves 8 bytes an element, which leaves an SM about 0.34
// cycles for it, or 43 issue slots: every operation counts.  So arithmetic runs
// as packed pairs, and expm1 is a polynomial on the FMA units.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace rcu {
namespace linrec {

constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float root(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rsq(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// the minimum, which keeps a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two fp32 values in one 64-bit register pair: on sm_100 and later one packed
// instruction adds, multiplies or fuses both, which halves what the arithmetic
// takes of the issue slots (the forward's other limit beside the memory).
typedef unsigned long long F2;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float v) { return f2(v, v); }
__device__ __forceinline__ float lo(F2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi(F2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// c softplus(lambda) log2(e): -log2(a) per unit of s.  Held at 1e20, where a is
// 2^-60 at the lowest sigmoid already.
__device__ __forceinline__ float decay_rate2(float lambda, float c) {
  const float sp = lambda > 0.f ? lambda + log1pf(expf(-lambda)) : log1pf(expf(lambda));
  return min_nan(c * sp * LOG2E, 1e20f);
}

// 2^t - 1 for -126 <= t <= 0, relative error 2e-7.  t = n + f, n whole, |f| <= 1/2:
// 2^n (2^f - 1) + (2^n - 1), with (2^f - 1) / f a polynomial of degree 5
// fitted to the least relative error (1.1e-8 before rounding); n = 0 leaves
// the polynomial alone, so that small t keep their precision.
__device__ __forceinline__ F2 ex2m1(F2 t) {
  const F2 m = add2(t, f2(12582912.f));  // 1.5 * 2^23: rounds t to a whole number in the low bits
  const F2 f = fma2(add2(m, f2(-12582912.f)), f2(-1.f), t);
  F2 p = f2(1.5403512e-4f);
  p = fma2(p, f, f2(1.3390735e-3f));
  p = fma2(p, f, f2(9.6182376e-3f));
  p = fma2(p, f, f2(5.5503573e-2f));
  p = fma2(p, f, f2(2.4022649e-1f));
  p = fma2(p, f, f2(6.9314718e-1f));
  const F2 s = f2(__int_as_float((__float_as_int(lo(m)) << 23) + 0x3f800000),  // 2^n
                  __int_as_float((__float_as_int(hi(m)) << 23) + 0x3f800000));
  return fma2(s, mul2(p, f), add2(s, f2(-1.f)));
}

// The same for -1/2 <= t <= 0, where n is 0 for the half of them and the
// polynomial alone reaches: a third of the operations.  Decay rates up to
// SMALL_RATE keep t there whatever the gates do (a state remembers for two
// steps or more at an open gate, as trained recurrences over long sequences
// do); a warp whose channels all have such rates takes this form.
constexpr float SMALL_RATE = 0.5f;
template <int N>
__device__ __forceinline__ void ex2m1_small(const F2 (&t)[N], F2 *v) {
  const F2 c[4] = {f2(9.5412815e-3f), f2(5.54904081e-2f), f2(2.40225643e-1f), f2(6.93147182e-1f)};
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = f2(1.15445221e-3f);
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = fma2(v[n], t[n], c[k]);
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = mul2(v[n], t[n]);
}
__device__ __forceinline__ bool small_rate(float k2) { return k2 <= SMALL_RATE; }
__device__ __forceinline__ bool small_rate(F2 k2) {
  return lo(k2) <= SMALL_RATE && hi(k2) <= SMALL_RATE;
}

// bf16: the two sigmoids share one reciprocal, of the product of their denominators:
// logits stop at -42, where e^42 = 2^60.6 keeps that product a normal number and
// a sigmoid is 6e-19, and a NaN in one gate reaches the other.  fp32, and the single
// step, have a reciprocal for each, where e^inf = inf makes an infinite logit exact:
// there it costs nothing (bf16 T=512 B=256 H=1024 forward 181 us with it, 174 without;
// fp32 T=253 B=134 H=989 113 and 115).  r above r_ceiling of its channel's rate, where a is 2^-90, is
// taken as that: what the state would still pass on is below any rounding, and
// ex2m1 keeps its range (SMALL_RATE needs no ceiling).  A NaN stays one.  bf16
// logits are limited as packed pairs, two at a time; a ceiling rounded to bf16 moves
// by at most 1/4, the exponent by a factor of e^(1/4): to 2^-116 at worst.
constexpr float LOGIT_FLOOR = -42.f;
__device__ __forceinline__ float r_ceiling(float k2) {
  const float s = 90.f / k2;  // sigmoid(r) at the limit
  return s < 1.f ? fmaxf(logf(s / (1.f - s)), LOGIT_FLOOR) : __int_as_float(0x7f800000);
}
__device__ __forceinline__ uint32_t floor_logit(uint32_t v) {  // bf16 -42 = 0xc228
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0xc228c228u));
  return r;
}
struct Limits {
  float top;       // fp32: of the lane's channel
  uint32_t top2;   // bf16: of its two channels
};
__device__ __forceinline__ float limit_r(float v, const Limits &l) { return min_nan(v, l.top); }
__device__ __forceinline__ uint32_t limit_r(uint32_t v, const Limits &l) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(floor_logit(v)), "r"(l.top2));
  return r;
}
__device__ __forceinline__ F2 exponent_of(F2 logit) { return mul2(logit, f2(-LOG2E)); }
__device__ __forceinline__ Limits limits(float k2) { return {r_ceiling(k2), 0u}; }
__device__ __forceinline__ Limits limits(F2 k2) {
  const float a = r_ceiling(lo(k2)), b = r_ceiling(hi(k2));
  return {0.f, (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u)};
}

// w = 1 - a^2 = em1 (-2 - em1) from em1 = a - 1, and its roots.  A decay rate
// of 0 makes w 0: where 1 / sqrt(w) is wanted a tiny addend keeps that finite,
// and every use multiplies it by something that is 0 then.
__device__ __forceinline__ F2 one_minus_a2(F2 em1, F2 tiny) {
  return fma2(em1, fma2(em1, f2(-1.f), f2(-2.f)), tiny);
}
__device__ __forceinline__ float one_minus_a2(float em1, float tiny) {
  return fmaf(em1, -2.f - em1, tiny);
}
__device__ __forceinline__ F2 inv_beta(F2 w) { return f2(rsq(lo(w)), rsq(hi(w))); }
__device__ __forceinline__ float inv_beta(float w) { return rsq(w); }

// Of N pairs of elements: em1 = a - 1, nb = -beta g x, and the sigmoids negated
// (ns makes the decay's exponent k2 ns; the other signs cancel in products).  The
// gates come as exponents, tr = -r log2(e) and ti likewise, of limited logits.  SMALL:
// of rates up to SMALL_RATE; SHARED: with one reciprocal for both sigmoids.
// Written stage by stage over the N pairs: each stage's operations are
// independent, and a warp has few others to hide the latency of a chain of
// twenty dependent ones behind.
template <bool SMALL, bool SHARED, int N>
__device__ __forceinline__ void gates_n(const F2 (&x)[N], const F2 (&tr)[N], const F2 (&ti)[N],
                                        F2 k2, F2 *em1, F2 *nb, F2 *ns, F2 *ng) {
  F2 pr[N], pi[N], t[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    pr[n] = f2(ex2(lo(tr[n])), ex2(hi(tr[n])));
    pi[n] = f2(ex2(lo(ti[n])), ex2(hi(ti[n])));
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    pr[n] = add2(pr[n], f2(1.f));
    pi[n] = add2(pi[n], f2(1.f));
    if (SHARED) t[n] = mul2(pr[n], pi[n]);
  }
  if (SHARED) {
#pragma unroll
    for (int n = 0; n < N; ++n) t[n] = f2(rcp(-lo(t[n])), rcp(-hi(t[n])));
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    ns[n] = SHARED ? mul2(t[n], pi[n]) : f2(rcp(-lo(pr[n])), rcp(-hi(pr[n])));
    ng[n] = SHARED ? mul2(t[n], pr[n]) : f2(rcp(-lo(pi[n])), rcp(-hi(pi[n])));
    t[n] = mul2(k2, ns[n]);
  }
  if (SMALL) {
    ex2m1_small<N>(t, em1);
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) em1[n] = ex2m1(t[n]);
  }
#pragma unroll
  for (int n = 0; n < N; ++n) t[n] = mul2(em1[n], fma2(em1[n], f2(-1.f), f2(-2.f)));
#pragma unroll
  for (int n = 0; n < N; ++n) t[n] = f2(root(lo(t[n])), root(hi(t[n])));
#pragma unroll
  for (int n = 0; n < N; ++n) nb[n] = mul2(t[n], mul2(ng[n], x[n]));
}

// One step, a h + b, on the negated state and input: -h moves like h.
__device__ __forceinline__ F2 step(F2 em1, F2 h, F2 b) { return add2(h, fma2(em1, h, b)); }
__device__ __forceinline__ float step(float em1, float h, float b) { return h + fmaf(em1, h, b); }

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

}  // namespace linrec
}  // namespace rcu
