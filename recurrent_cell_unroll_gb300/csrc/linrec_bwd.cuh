// What the backward kernels of the gated linear recurrence share: decoding their
// saved inputs, the gates of a few steps and one step's gradients.
#pragma once

#include "act8.cuh"
#include "linrec_tile.cuh"

namespace rcu {
namespace linrec {

// 8-bit codes: c + 128 in the low bits of 2^23 is exact in fp32.  A code of -128
// (not a number) comes out as -128 here; any_nan tells whether a lane has one, and
// its results are made NaN afterwards.
__device__ __forceinline__ float code_bits(uint32_t biased, int j) {  // 2^23 + byte j
  return __uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7540 + j));
}
template <int CPT>
__device__ __forceinline__ uint32_t nan_flags(uint32_t raw) {  // a byte of raw ^ 0x80.. is 0
  const uint32_t one = CPT == 1 ? 0x01u : 0x0101u, t = raw ^ (one << 7);
  return (t - one) & ~t & (one << 7);
}
// One step's values: x, and the gates' exponents (-logit log2(e), of logits within
// their limits).  8-bit codes are scaled by `scale`, the gates' by its product
// with -log2(e): their limits are on the exponents.  Blocks up to FREE_EXP have logits
// within them (127 / 4 < 42) and go without: gates with SMALL take that for granted
// (bf16 T=512 B=256 H=1024 from 8 bits 428 us, 434 with limits).
constexpr int FREE_EXP = -2;
constexpr float EXP_TOP = -LOGIT_FLOOR * LOG2E;
template <typename IT, typename V>
struct Decode;
template <>
struct Decode<bf16, F2> {
  __device__ __forceinline__ static F2 x(uint32_t v, float) { return bf16_pair(v); }
  __device__ __forceinline__ static F2 r(uint32_t v, float, const Limits &l) {
    return exponent_of(bf16_pair(limit_r(v, l)));
  }
  __device__ __forceinline__ static F2 i(uint32_t v, float) {
    return exponent_of(bf16_pair(floor_logit(v)));
  }
  __device__ __forceinline__ static F2 bounded(uint32_t v, float s) { return i(v, s); }
};
template <>
struct Decode<int8_t, F2> {
  __device__ __forceinline__ static F2 x(uint32_t v, float scale) {
    v ^= 0x8080u;
    return mul2(add2(f2(code_bits(v, 0), code_bits(v, 1)), f2(-8388736.f)), f2(scale));
  }
  __device__ __forceinline__ static F2 r(uint32_t v, float scale, const Limits &l) {
    const F2 t = i(v, scale);  // not limited as bf16: the channels' limits, widened
    const float a = __uint_as_float(l.top2 << 16), b = __uint_as_float(l.top2 & 0xffff0000u);
    return f2(fmaxf(lo(t), a * -LOG2E), fmaxf(hi(t), b * -LOG2E));
  }
  __device__ __forceinline__ static F2 i(uint32_t v, float scale) {
    const F2 t = x(v, scale);
    return f2(fminf(lo(t), EXP_TOP), fminf(hi(t), EXP_TOP));
  }
  __device__ __forceinline__ static F2 bounded(uint32_t v, float s) { return x(v, s); }
};
template <>
struct Decode<float, float> {
  __device__ __forceinline__ static float x(uint32_t v, float) { return __uint_as_float(v); }
  __device__ __forceinline__ static float r(uint32_t v, float, const Limits &l) {
    return limit_r(__uint_as_float(v), l) * -LOG2E;
  }
  __device__ __forceinline__ static float i(uint32_t v, float) {
    return __uint_as_float(v) * -LOG2E;
  }
  __device__ __forceinline__ static float bounded(uint32_t v, float s) { return i(v, s); }
};
template <>
struct Decode<int8_t, float> {
  __device__ __forceinline__ static float x(uint32_t v, float scale) {
    return (code_bits(v ^ 0x80u, 0) - 8388736.f) * scale;
  }
  __device__ __forceinline__ static float r(uint32_t v, float scale, const Limits &l) {
    return fmaxf(x(v, scale), l.top * -LOG2E);
  }
  __device__ __forceinline__ static float i(uint32_t v, float scale) { return x(v, scale); }
  __device__ __forceinline__ static float bounded(uint32_t v, float s) { return x(v, s); }
};

// Of each of N steps, BATCH pairs at a time: em1 = a - 1, nb = -beta g x, ns = -sigmoid(r), ng = -sigmoid(i).
template <typename IT, bool SMALL, int BATCH, int N>
__device__ __forceinline__ void gates(const uint32_t (&raw)[3][N], const float (&scale)[3][N], F2 k2,
                                      const Limits &lim, F2 (&em1)[N], F2 (&nb)[N], F2 (&ns)[N],
                                      F2 (&ng)[N]) {
  typedef Decode<IT, F2> D;
  static_assert(N % BATCH == 0, "the steps are whole batches");
#pragma unroll
  for (int s = 0; s < N; s += BATCH) {
    F2 x[BATCH], r[BATCH], i[BATCH];
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      const int q = s + n;
      x[n] = D::x(raw[0][q], scale[0][q]);
      r[n] = SMALL ? D::bounded(raw[1][q], scale[1][q]) : D::r(raw[1][q], scale[1][q], lim);
      i[n] = SMALL ? D::bounded(raw[2][q], scale[2][q]) : D::i(raw[2][q], scale[2][q]);
    }
    gates_n<SMALL, true, BATCH>(x, r, i, k2, em1 + s, nb + s, ns + s, ng + s);
  }
}
// fp32 has one channel a lane: there the arithmetic pairs two steps
template <typename IT, bool SMALL, int BATCH, int N>
__device__ __forceinline__ void gates(const uint32_t (&raw)[3][N], const float (&scale)[3][N],
                                      float k2, const Limits &lim, float (&em1)[N], float (&nb)[N],
                                      float (&ns)[N], float (&ng)[N]) {
  typedef Decode<IT, float> D;
  static_assert(N % (2 * BATCH) == 0, "the steps are whole batches");
#pragma unroll
  for (int s = 0; s < N; s += 2 * BATCH) {
    F2 x[BATCH], r[BATCH], i[BATCH], m[BATCH], b[BATCH], vs[BATCH], vg[BATCH];
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      const int q = s + 2 * n;
      x[n] = f2(D::x(raw[0][q], scale[0][q]), D::x(raw[0][q + 1], scale[0][q + 1]));
      r[n] = SMALL ? f2(D::bounded(raw[1][q], scale[1][q]), D::bounded(raw[1][q + 1], scale[1][q + 1]))
                   : f2(D::r(raw[1][q], scale[1][q], lim), D::r(raw[1][q + 1], scale[1][q + 1], lim));
      i[n] = SMALL ? f2(D::bounded(raw[2][q], scale[2][q]), D::bounded(raw[2][q + 1], scale[2][q + 1]))
                   : f2(D::i(raw[2][q], scale[2][q]), D::i(raw[2][q + 1], scale[2][q + 1]));
    }
    gates_n<SMALL, false, BATCH>(x, r, i, f2(k2), m, b, vs, vg);
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      const int q = s + 2 * n;
      em1[q] = lo(m[n]), nb[q] = lo(b[n]), ns[q] = lo(vs[n]), ng[q] = lo(vg[n]);
      em1[q + 1] = hi(m[n]), nb[q + 1] = hi(b[n]), ns[q + 1] = hi(vs[n]), ng[q + 1] = hi(vg[n]);
    }
  }
}

// NaN where a step's code says so: in what x, r or i enter.
__device__ __forceinline__ bool not_a_number(uint32_t raw, int j) {
  return (raw >> (8 * j) & 0xffu) == 0x80u;
}
template <int CPT>
__device__ __forceinline__ void spoil(uint32_t x, uint32_t r, uint32_t i, float &em1, float &nb,
                                      float &ns, float &ng) {
  const float nan = __int_as_float(0x7fc00000);
  if (not_a_number(x, 0)) nb = nan;
  if (not_a_number(r, 0)) em1 = nb = ns = nan;
  if (not_a_number(i, 0)) nb = ng = nan;
}
template <int CPT>
__device__ __forceinline__ void spoil(uint32_t x, uint32_t r, uint32_t i, F2 &em1, F2 &nb, F2 &ns,
                                      F2 &ng) {
  float m[2] = {lo(em1), hi(em1)}, b[2] = {lo(nb), hi(nb)}, s[2] = {lo(ns), hi(ns)},
        g[2] = {lo(ng), hi(ng)};
#pragma unroll
  for (int j = 0; j < 2; ++j)
    spoil<1>(x >> (8 * j), r >> (8 * j), i >> (8 * j), m[j], b[j], s[j], g[j]);
  em1 = f2(m[0], m[1]), nb = f2(b[0], b[1]), ns = f2(s[0], s[1]), ng = f2(g[0], g[1]);
}

// Local gradients of one step from ne = -dL/dh_t and the state before it, which
// moves on by one step:
//   dx = e beta g,  di = e b (1 - g),  dlog_s = dL/dlog(a) s = e s (a h - a^2 b / w),
//   dr = -K dlog_s (1 - s)
template <typename V>
__device__ __forceinline__ void grads(V em1, V nb, V ns, V ng, V nk, V ne, V &h, V &dx, V &dr, V &di,
                                      V &dlog_s) {
  V one, minus, tiny;
  set(one, 1.f);
  set(minus, -1.f);
  set(tiny, 1e-37f);
  const V w = one_minus_a2(em1, tiny), rb = inv_beta(w), arb = mul_v(add_v(em1, one), rb);
  const V ah = fma_v(em1, h, h);
  dx = mul_v(ne, mul_v(mul_v(w, rb), ng));
  di = mul_v(mul_v(ne, nb), add_v(ng, one));
  dlog_s = mul_v(mul_v(ne, ns), fma_v(mul_v(arb, arb), nb, ah));
  dr = mul_v(mul_v(nk, dlog_s), add_v(ns, one));
  h = fma_v(nb, minus, ah);
}

// The same for every code of N steps that is not a number (hardly ever one).
template <int CPT, int N, typename V>
__device__ __forceinline__ void spoil_codes(const uint32_t (&raw)[3][N], V (&em1)[N], V (&nb)[N],
                                            V (&ns)[N], V (&ng)[N]) {
  uint32_t bad = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int s = 0; s < N; ++s) bad |= nan_flags<CPT>(raw[k][s]);
  if (bad) {
#pragma unroll
    for (int s = 0; s < N; ++s)
      spoil<CPT>(raw[0][s], raw[1][s], raw[2][s], em1[s], nb[s], ns[s], ng[s]);
  }
}

// dlambda from partial sums: partial [rows][H] (linrec_bwd.cu)
cudaError_t launch_dlambda(const float *partial, int64_t rows, const LinrecBwd &p, cudaStream_t s);
// The kernel for short sequences of many rows (linrec_bwd_short.cu), and whether it is
// the faster one; resident_blocks: of the tiled kernel, vec: as of launch_linrec_bwd.
bool short_bwd_pays(const LinrecBwd &p, int resident_blocks, bool vec);
cudaError_t launch_short_bwd(const LinrecBwd &p, DevMem &ws, int *err, cudaStream_t s,
                             int *launches);

}  // namespace linrec
}  // namespace rcu
