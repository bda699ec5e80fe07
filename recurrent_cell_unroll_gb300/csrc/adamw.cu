// AdamW over many tensors in few launches, states in 32 bits or in 8.
//
// Bound by memory with fp32 states: a parameter in fp32 moves 28 bytes for a dozen
// operations.  With 8-bit ones it moves some 16, and the codes take fifty operations
// more, which bound it as much: so what is rare (values that are not finite, codes
// that stand for them, the ends of a tensor) leaves a warp's usual path.
//
// Measured: fp32 states, 161M parameters, 652 us (6870 GB/s); 8-bit ones with bf16
// gradients, 51M parameters, 178 us (717 MB, at 93 instructions a parameter), and
// each state read out in 42 us.
//
// The tensors' table comes as the kernel's parameter, so a captured launch keeps it
// and nothing is copied or kept on the device; a block finds the tensor of its
// piece by halving.
//
// 8-bit states (include/rcu.h has the format): 8 threads that stand side by side
// hold a block of 64 values, 8 of them each, and find its largest magnitude by
// three exchanges.  Adding the offset o to f = |value| 2^-e makes a float whose
// upper bits are the code: its exponent and three bits, counted from o's.
#include <cmath>

#include "ssm_common.cuh"

namespace rcu {
namespace {

using namespace ssm;

constexpr int NT = 256, V = 8;
constexpr int TURN = NT * V;  // values of a block at a time: 32 blocks of 64
// A block takes as many turns as leave eight blocks an SM, 8 at most: finding its tensor
// costs as much as a turn's arithmetic on 3 values a thread (8-bit states, 51M
// parameters, 218 us with one turn, 178 with four and with eight).
constexpr int MOST_TURNS = 8;

struct Tensor {
  void *p;
  const void *g;
  void *m, *v;
  int8_t *me, *ve;
  void *copy;
  int64_t n;
  uint32_t key;    // its place in the list
  int32_t flags;   // bit 0: p bf16, 1: g bf16, 2: 8-bit states, 3: words
  int64_t first;   // pieces before it
};
constexpr int P16 = 1, G16 = 2, STATES8 = 4, WORDS = 8;
// A launch's parameters are at most 32764 bytes.
constexpr int MOST = 360, FEW = 40;

struct Constants {
  float beta1, one_beta1, beta2, one_beta2, eps;
  float kept, size, root;  // 1 - lr wd, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  uint32_t random;         // mix(seed + 0x9e3779b9 t)
};
struct Given {
  AdamWStep s;
  Constants c;
  int piece;  // values of a block
};

// a published 32-bit mixing function (include/rcu.h)
__host__ __device__ inline uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  x *= 0x846ca68bu;
  return x ^ x >> 16;
}
__host__ __device__ inline void of_step(const AdamWStep &s, double lr, int64_t t, Constants &c) {
  c.kept = (float)(1.0 - lr * s.weight_decay);
  c.size = (float)(lr / (1.0 - pow(s.beta1, (double)t)));
  c.root = (float)(1.0 / sqrt(1.0 - pow(s.beta2, (double)t)));
  c.random = mix(s.seed + 0x9e3779b9u * (uint32_t)t);
}

__device__ __forceinline__ float power(int e) { return __int_as_float((e + 127) << 23); }

// The two 8-bit formats.
template <bool SIGNED>
struct State8 {
  static constexpr int OCTAVES = SIGNED ? 14 : 30;
  static constexpr int BASE = (127 - OCTAVES) << 3;
  static constexpr int LAST = SIGNED ? 127 : 254;
  __device__ __forceinline__ static float offset() { return power(-OCTAVES); }
  __device__ __forceinline__ static int exponent(float top) {  // top >= 0, finite
    return min(max((__float_as_int(top) >> 23) - 127, -126), 126);
  }
  // `bits`: what is added behind the cut, below 2^20
  __device__ __forceinline__ static int code(float v, float scale, uint32_t bits) {
    if (!isfinite(v)) return SIGNED ? -128 : 127;
    const float f = __fadd_rn(__fmul_rn(fabsf(v), scale), offset());
    int n = min((int)((__float_as_uint(f) + bits) >> 20) - BASE, LAST);
    if (SIGNED) return v < 0.f ? -n : n;
    return v > 0.f ? max(n, 1) - 128 : -128;
  }
  __device__ __forceinline__ static float value(int q, float scale) {
    if (q == (SIGNED ? -128 : 127)) return __int_as_float(0x7fc00000);
    const int n = SIGNED ? abs(q) : q + 128;
    const float v = __fadd_rn(__int_as_float((n + BASE) << 20), -offset());
    return __fmul_rn(SIGNED && q < 0 ? -v : v, scale);
  }
};
constexpr uint32_t NEAREST = 1u << 19;

// The largest finite magnitude of a block of 64: of 8 values in each of 8 threads.
__device__ __forceinline__ float block_top(const float (&v)[V]) {
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) top = fmaxf(top, isfinite(v[k]) ? fabsf(v[k]) : 0.f);
#pragma unroll
  for (int o = 1; o < 8; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top;
}

// V values at p + i, `n` of them there (n >= V: all, by words where they are aligned).
template <typename T>
__device__ __forceinline__ void load(const T *p, int64_t n, bool words, float (&v)[V]) {
  if (words && n >= V) {
    constexpr int W = 16 / sizeof(T) < V ? 16 / sizeof(T) : V;
#pragma unroll
    for (int k = 0; k < V; k += W) {
      const Word<T, W> w = *reinterpret_cast<const Word<T, W> *>(p + k);
#pragma unroll
      for (int j = 0; j < W; ++j) v[k + j] = to_f(w.v[j]);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = k < n ? to_f(p[k]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store(T *p, int64_t n, bool words, const float (&v)[V]) {
  if (words && n >= V) {
    constexpr int W = 16 / sizeof(T) < V ? 16 / sizeof(T) : V;
#pragma unroll
    for (int k = 0; k < V; k += W) {
      Word<T, W> w;
#pragma unroll
      for (int j = 0; j < W; ++j) w.v[j] = from_f<T>(v[k + j]);
      *reinterpret_cast<Word<T, W> *>(p + k) = w;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (k < n) p[k] = from_f<T>(v[k]);
}
__device__ __forceinline__ void load8(const int8_t *p, int64_t n, bool words, int (&q)[V]) {
  if (words && n >= V) {
    const Word<int8_t, V> w = *reinterpret_cast<const Word<int8_t, V> *>(p);
#pragma unroll
    for (int k = 0; k < V; ++k) q[k] = w.v[k];
    return;
  }
#pragma unroll
  for (int k = 0; k < V; ++k) q[k] = k < n ? p[k] : 0;
}
__device__ __forceinline__ void store8(int8_t *p, int64_t n, bool words, const int (&q)[V]) {
  if (words && n >= V) {
    Word<int8_t, V> w;
#pragma unroll
    for (int k = 0; k < V; ++k) w.v[k] = (int8_t)q[k];
    *reinterpret_cast<Word<int8_t, V> *>(p) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (k < n) p[k] = (int8_t)q[k];
}

// A state's 8 values of a block with exponent e, and back.
template <bool SIGNED>
__device__ __forceinline__ void decode(const int8_t *codes, int e, int64_t n, bool words, float (&v)[V]) {
  int q[V];
  load8(codes, n, words, q);
  const float scale = power(e);
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = k < n ? State8<SIGNED>::value(q[k], scale) : 0.f;
}
template <bool SIGNED>
__device__ __forceinline__ void encode(const float (&v)[V], const uint32_t (&bits)[V], int8_t *codes,
                                       int8_t *exps, int64_t n, bool words) {
  const int e = State8<SIGNED>::exponent(block_top(v));
  const float scale = power(-e);
  int q[V];
#pragma unroll
  for (int k = 0; k < V; ++k) q[k] = State8<SIGNED>::code(v[k], scale, bits[k]);
  store8(codes, n, words, q);
  if (threadIdx.x % 8 == 0 && n > 0) *exps = (int8_t)e;
}

// The same of whole words of a warp whose codes and values are all finite; false where
// they are not (and then nothing is done).
template <bool SIGNED>
__device__ __forceinline__ bool decode_words(const uint2 &w, int e, float (&v)[V]) {
  // a byte of 0 where a code stands for what is not finite
  auto none = [](uint32_t t) { return ((t - 0x01010101u) & ~t & 0x80808080u) == 0; };
  const uint32_t nan = SIGNED ? 0x80808080u : 0x7f7f7f7fu;
  if (!__all_sync(0xffffffffu, none(w.x ^ nan) && none(w.y ^ nan))) return false;
  const float scale = power(e);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const uint32_t word = k < 4 ? w.x : w.y;
    if (SIGNED) {
      const int q = (int)(word << (24 - k % 4 * 8)) >> 24;
      const float f = __fadd_rn(__int_as_float((abs(q) << 20) + (State8<true>::BASE << 20)), -State8<true>::offset());
      v[k] = __fmul_rn(f, __int_as_float(__float_as_int(scale) | (q & 0x80000000)));
    } else {
      const int q = (word ^ 0x80808080u) >> (k % 4 * 8) & 255;
      v[k] = __fmul_rn(__fadd_rn(__int_as_float((q << 20) + (State8<false>::BASE << 20)), -State8<false>::offset()),
                       scale);
    }
  }
  return true;
}
// `random`: a word an element, of which this state takes its half
template <bool SIGNED>
__device__ __forceinline__ bool encode_words(const float (&v)[V], const uint32_t (&random)[V], int8_t *codes,
                                             int8_t *exps) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < V; ++k) top = max(top, __float_as_uint(v[k]) & (SIGNED ? 0x7fffffffu : 0xffffffffu));
#pragma unroll
  for (int o = 1; o < 8; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  // finite, and small enough that no code passes the last one
  if (!__all_sync(0xffffffffu, top < 0x7f000000u)) return false;
  const int e = max((int)(top >> 23) - 127, -126);
  const float scale = power(-e);
  constexpr uint32_t BASE = (uint32_t)State8<SIGNED>::BASE << 20;
  uint32_t q[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const float f = __fadd_rn(__fmul_rn(fabsf(v[k]), scale), State8<SIGNED>::offset());
    const uint32_t bits = (SIGNED ? random[k] << 4 : random[k] >> 12) & 0xffff0u;
    const uint32_t n = (__float_as_uint(f) + bits + (8u - BASE)) >> 20;
    if (SIGNED) {
      const uint32_t s = (int)__float_as_uint(v[k]) >> 31;
      q[k] = (n ^ s) - s;
    } else {
      q[k] = max(n, min(__float_as_uint(v[k]), 1u));
    }
  }
  uint2 w;
  w.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  w.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
  if (!SIGNED) w.x ^= 0x80808080u, w.y ^= 0x80808080u;
  *reinterpret_cast<uint2 *>(codes) = w;
  if (threadIdx.x % 8 == 0) *exps = (int8_t)e;
  return true;
}

__device__ __forceinline__ float root(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

template <int COUNT>
struct Table {
  int count;
  Tensor t[COUNT];
};

template <int COUNT>
__global__ void __launch_bounds__(NT, 4) adamw_kernel(const __grid_constant__ Table<COUNT> table,
                                                   const __grid_constant__ Given given) {
  __shared__ Constants shared;
  if (given.s.step_dev || given.s.lr_dev) {
    if (threadIdx.x == 0) {
      shared = given.c;
      const int64_t t = given.s.step_dev ? *given.s.step_dev : given.s.step;
      of_step(given.s, given.s.lr_dev ? *given.s.lr_dev : given.s.lr, t, shared);
    }
    __syncthreads();
  }
  const Constants &c = given.s.step_dev || given.s.lr_dev ? shared : given.c;
  int lo = 0, hi = table.count;  // the last tensor that starts at this piece or before
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (table.t[mid].first <= blockIdx.x) lo = mid;
    else hi = mid;
  }
  const Tensor &t = table.t[lo];
  const bool words = t.flags & WORDS, held8 = t.flags & STATES8;
  const float scale = given.s.scale ? *given.s.scale : 1.f;
  const uint32_t key = mix(c.random + t.key);
  const int64_t start = (blockIdx.x - t.first) * given.piece;
#pragma unroll 1
  for (int64_t at = start; at < min(start + given.piece, t.n); at += TURN) {
    const int64_t i = at + threadIdx.x * V;
    const int64_t n = max((int64_t)0, t.n - i);  // all of a block's threads stay for the exchanges
    float p[V], g[V], m[V], v[V];
    if (t.flags & P16) load(static_cast<const bf16 *>(t.p) + i, n, words, p);
    else load(static_cast<const float *>(t.p) + i, n, words, p);
    if (t.flags & G16) load(static_cast<const bf16 *>(t.g) + i, n, words, g);
    else load(static_cast<const float *>(t.g) + i, n, words, g);
    int8_t *me = t.me + i / 64, *ve = t.ve + i / 64, *mc = static_cast<int8_t *>(t.m) + i;
    int8_t *vc = static_cast<int8_t *>(t.v) + i;
    const bool whole = held8 && words && __all_sync(0xffffffffu, n >= V);  // of the warp
    if (held8) {
      const int em = n > 0 ? *me : 0, ev = n > 0 ? *ve : 0;
      if (whole) {
        const uint2 wm = *reinterpret_cast<const uint2 *>(mc), wv = *reinterpret_cast<const uint2 *>(vc);
        if (!decode_words<true>(wm, em, m)) decode<true>(mc, em, n, true, m);
        if (!decode_words<false>(wv, ev, v)) decode<false>(vc, ev, n, true, v);
      } else {
        decode<true>(mc, em, n, words, m);
        decode<false>(vc, ev, n, words, v);
      }
    } else {
      load(static_cast<const float *>(t.m) + i, n, words, m);
      load(static_cast<const float *>(t.v) + i, n, words, v);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (given.s.scale) g[k] = __fmul_rn(g[k], scale);
      // each product rounded by itself: a code's rounding is then the same everywhere
      m[k] = __fadd_rn(__fmul_rn(m[k], c.beta1), __fmul_rn(g[k], c.one_beta1));
      v[k] = __fadd_rn(__fmul_rn(v[k], c.beta2), __fmul_rn(__fmul_rn(g[k], c.one_beta2), g[k]));
      // the root keeps small v (an eps of 0 divides by it), the quotient is good to 2 units
      p[k] = fmaf(-c.size, m[k] * rcp(fmaf(root(v[k]), c.root, c.eps)), p[k] * c.kept);
    }
    if (t.flags & P16) store(static_cast<bf16 *>(t.p) + i, n, words, p);
    else store(static_cast<float *>(t.p) + i, n, words, p);
    if (t.copy) store(static_cast<bf16 *>(t.copy) + i, n, words, p);
    if (held8) {
      uint32_t random[V];
#pragma unroll
      for (int k = 0; k < V; ++k) random[k] = mix(((uint32_t)i + k) ^ key);
      const bool m_done = whole && encode_words<true>(m, random, mc, me);
      const bool v_done = whole && encode_words<false>(v, random, vc, ve);
      uint32_t bits[V];
      if (!m_done) {
#pragma unroll
        for (int k = 0; k < V; ++k) bits[k] = (random[k] & 0xffffu) << 4 | 8;
        encode<true>(m, bits, mc, me, n, words);
      }
      if (!v_done) {
#pragma unroll
        for (int k = 0; k < V; ++k) bits[k] = (random[k] >> 16) << 4 | 8;
        encode<false>(v, bits, vc, ve, n, words);
      }
    } else {
      store(static_cast<float *>(t.m) + i, n, words, m);
      store(static_cast<float *>(t.v) + i, n, words, v);
    }
  }
}

template <bool SIGNED>
__global__ void __launch_bounds__(NT) pack_kernel(int64_t all, const float *x, int8_t *codes, int8_t *exps,
                                                  bool words) {
  const int64_t i = ((int64_t)blockIdx.x * NT + threadIdx.x) * V, n = max((int64_t)0, all - i);
  float v[V];
  load(x + i, n, words, v);
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (!SIGNED && v[k] < 0.f) v[k] = 0.f;
  uint32_t bits[V];
#pragma unroll
  for (int k = 0; k < V; ++k) bits[k] = NEAREST;
  encode<SIGNED>(v, bits, codes + i, exps + i / 64, n, words);
}

template <bool SIGNED>
__global__ void __launch_bounds__(NT) unpack_kernel(int64_t all, const int8_t *codes, const int8_t *exps,
                                                    float *y, bool words) {
  const int64_t i = ((int64_t)blockIdx.x * NT + threadIdx.x) * V, n = all - i;
  if (n <= 0) return;
  float v[V];
  const int e = exps[i / 64];
  // (the last block's threads decide by themselves)
  if (!(words && (int64_t)(blockIdx.x + 1) * NT * V <= all &&
        decode_words<SIGNED>(*reinterpret_cast<const uint2 *>(codes + i), e, v)))
    decode<SIGNED>(codes + i, e, n, words, v);
  store(y + i, n, words, v);
}

bool whole(const void *p, int size) {  // V values are whole words of 16 bytes, or of 8
  return reinterpret_cast<uintptr_t>(p) % std::min(16, V * size) == 0;
}

template <int COUNT>
cudaError_t launch(const Tensor *t, int count, int64_t pieces, const Given &given, cudaStream_t s,
                   int *launches) {
  Table<COUNT> table;
  table.count = count;
  std::copy(t, t + count, table.t);
  ++*launches;
  adamw_kernel<COUNT><<<(unsigned)pieces, NT, 0, s>>>(table, given);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamWStep &p, int64_t count, const rcu_adamw_tensor *tensors,
                         int nsm, bool vec, cudaStream_t s, int *launches) {
  int64_t turns = 0;
  for (int64_t k = 0; k < count; ++k) turns += (tensors[k].n + TURN - 1) / TURN;
  Given given{p, {}, 0};
  given.piece = TURN * (int)std::min<int64_t>(std::max<int64_t>(turns / (8 * nsm), 1), MOST_TURNS);
  Constants &c = given.c;
  c.beta1 = (float)p.beta1, c.one_beta1 = (float)(1.0 - p.beta1);
  c.beta2 = (float)p.beta2, c.one_beta2 = (float)(1.0 - p.beta2);
  c.eps = (float)p.eps;
  of_step(p, p.lr, p.step_dev ? 1 : p.step, c);
  Tensor t[MOST];
  int held = 0;
  int64_t pieces = 0;
  auto flush = [&]() {
    if (!held) return cudaSuccess;
    const cudaError_t e = held <= FEW ? launch<FEW>(t, held, pieces, given, s, launches)
                                      : launch<MOST>(t, held, pieces, given, s, launches);
    held = 0;
    pieces = 0;
    return e;
  };
  for (int64_t k = 0; k < count; ++k) {
    const rcu_adamw_tensor &a = tensors[k];
    if (a.n == 0) continue;
    const int64_t need = (a.n + given.piece - 1) / given.piece;
    if (held == MOST || pieces + need > INT32_MAX) {
      const cudaError_t e = flush();
      if (e != cudaSuccess) return e;
    }
    const int ps = a.p_type == RCU_BF16 ? 2 : 4, gs = a.g_type == RCU_BF16 ? 2 : 4, ss = a.m_exp ? 1 : 4;
    const bool words = vec && whole(a.p, ps) && whole(a.g, gs) && whole(a.m, ss) && whole(a.v, ss) &&
                       (!a.copy || whole(a.copy, 2));
    t[held++] = {a.p, a.g, a.m, a.v, a.m_exp, a.v_exp, a.copy, a.n, (uint32_t)k,
                 (ps == 2 ? P16 : 0) | (gs == 2 ? G16 : 0) | (a.m_exp ? STATES8 : 0) | (words ? WORDS : 0),
                 pieces};
    pieces += need;
  }
  return flush();
}

cudaError_t launch_state8_pack(int is_signed, int64_t n, const float *x, int8_t *codes, int8_t *exps,
                               int nsm, bool vec, cudaStream_t s, int *launches) {
  (void)nsm;
  ++*launches;
  const unsigned blocks = (unsigned)((n + TURN - 1) / TURN);
  const bool words = vec && whole(x, 4) && whole(codes, 1);
  if (is_signed) pack_kernel<true><<<blocks, NT, 0, s>>>(n, x, codes, exps, words);
  else pack_kernel<false><<<blocks, NT, 0, s>>>(n, x, codes, exps, words);
  return cudaGetLastError();
}

cudaError_t launch_state8_unpack(int is_signed, int64_t n, const int8_t *codes, const int8_t *exps,
                                 float *y, int nsm, bool vec, cudaStream_t s, int *launches) {
  (void)nsm;
  ++*launches;
  const unsigned blocks = (unsigned)((n + TURN - 1) / TURN);
  const bool words = vec && whole(y, 4) && whole(codes, 1);
  if (is_signed) unpack_kernel<true><<<blocks, NT, 0, s>>>(n, codes, exps, y, words);
  else unpack_kernel<false><<<blocks, NT, 0, s>>>(n, codes, exps, y, words);
  return cudaGetLastError();
}

}  // namespace rcu
