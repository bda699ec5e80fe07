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
// measured as an error of 7e-6 in dh0, against 1e-6 in this form.
//
// The forward in bf16 moves 8 bytes an element, which leaves an SM about 0.34
// cycles for it: a direct evaluation's six special-function operations (16 a
// cycle) alone would take 0.38.  So the two sigmoids share one reciprocal and
// expm1 is a polynomial on the FMA units; two exponentials, a reciprocal and a
// reciprocal root remain.
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
__device__ __forceinline__ float rsq(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// minimum / maximum that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// -c softplus(lambda) log2(e): the exponent of a per unit of s, base 2.
__device__ __forceinline__ float decay_rate2(float lambda, float c) {
  const float sp = lambda > 0.f ? lambda + log1pf(expf(-lambda)) : log1pf(expf(lambda));
  return -c * sp * LOG2E;
}

// 2^t - 1 for t <= 0, relative error 2e-7.  t = n + f, n whole, |f| <= 1/2:
// 2^n (2^f - 1) + (2^n - 1), with (2^f - 1) / f a polynomial of degree 5
// fitted to the least relative error (1.1e-8 before rounding); n = 0 leaves
// the polynomial alone, so that small t keep their precision.
__device__ __forceinline__ float ex2m1(float t) {
  t = max_nan(t, -126.f);
  const float m = t + 12582912.f;  // 1.5 * 2^23: rounds t to a whole number in the low bits
  const float f = t - (m - 12582912.f);
  float p = 1.5403512e-4f;
  p = fmaf(p, f, 1.3390735e-3f);
  p = fmaf(p, f, 9.6182376e-3f);
  p = fmaf(p, f, 5.5503573e-2f);
  p = fmaf(p, f, 2.4022649e-1f);
  p = fmaf(p, f, 6.9314718e-1f);
  const float s = __int_as_float((__float_as_int(m) << 23) + 0x3f800000);  // 2^n
  return fmaf(s, p * f, s - 1.f);
}

// The two sigmoids: er = e^-r, ei = e^-i, s = 1 / (1 + er), g = 1 / (1 + ei).
// The exponents stop at 62, where the product of the denominators is still a
// normal number: a sigmoid below 2^-62 is held there.  A NaN stays one.
struct Sig {
  float er, ei, s, g;
};
__device__ __forceinline__ Sig sigmoids(float r, float i) {
  Sig v;
  v.er = ex2(min_nan(r * -LOG2E, 62.f));
  v.ei = ex2(min_nan(i * -LOG2E, 62.f));
  const float pr = 1.f + v.er, pi = 1.f + v.ei;
  const float inv = rcp(pr * pi);
  v.s = inv * pi;
  v.g = inv * pr;
  return v;
}

// w = 1 - a^2 from em1 = a - 1, and 1 / sqrt(w).  w = 0 (a decay rate of 0)
// gives a large finite root: every use multiplies it by something that is 0.
__device__ __forceinline__ float one_minus_a2(float em1) { return -em1 * (2.f + em1); }
__device__ __forceinline__ float inv_beta(float w) { return rsq(max_nan(w, 1e-37f)); }

// em1 and b = beta g x of one element.
__device__ __forceinline__ void gate(float x, float r, float i, float k2, float &em1, float &b) {
  const Sig v = sigmoids(r, i);
  em1 = ex2m1(k2 * v.s);
  const float w = one_minus_a2(em1);
  b = w * inv_beta(w) * (v.g * x);
}

// One step: a h + b.
__device__ __forceinline__ float step(float em1, float h, float b) { return h + fmaf(em1, h, b); }

// Local gradients of one element given e = dL/dh_t and the state before it.
struct Grad {
  float dx, dr, di, dlog_s;  // dlog_s: dL/da a s, summed over elements into dlambda
};
__device__ __forceinline__ Grad grads(float x, const Sig &v, float em1, float k, float hp,
                                      float e) {
  const float w = one_minus_a2(em1), rb = inv_beta(w), beta = w * rb;
  const float gx = v.g * x, a = 1.f + em1;
  Grad d;
  d.dx = e * (beta * v.g);
  d.di = e * (beta * gx) * (v.ei * v.g);
  // s / beta stays finite as s goes to 0 (like sqrt(s)), so s comes in before 1 / beta's product
  d.dlog_s = e * (fmaf(em1, hp, hp) * v.s - a * a * gx * (v.s * rb));
  d.dr = k * d.dlog_s * (v.er * v.s);
  return d;
}

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
