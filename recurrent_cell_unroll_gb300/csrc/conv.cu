// Short causal convolution along time with an optional SiLU: forward, backward
// and one step of many requests.
//
//   v_t = bias + sum_k w[k] x_{t-W+1+k},  y = v or v sigmoid(v)
//   dv = dy y'(v),  dx_t = sum_k w[k] dv_{t+W-1-k},  dw[k] = sum_t dv_t x_{t-W+1+k}
//
// Bound by memory: 2 (forward) and 3 (backward) values moved for some 2 W + 6
// and 6 W + 10 operations.  A thread keeps VEC channels and walks a stretch of
// steps with the last W inputs (and, backwards, W gradients) in registers, so
// that an input is read once but for the W - 1 that a stretch shares with the
// one before it.  Reads run 12 steps ahead by asynchronous copies into a ring of the
// thread's own in shared memory (in registers they cost half of the threads: backward
// bf16 T=8192 B=4 H=2048 173 us, 107 so), and channels are worked on as packed pairs.
//
// Measured, W=4: forward bf16 T=512 B=256 H=1024 117 us (4590 GB/s, 68 % of the copy's
// rate), backward bf16 T=8192 B=4 H=2048 107 us (3770 GB/s, 56 %), fp32 mixed lengths
// T=500 B=64 H=512 44 us (46 %).  Neither the memory nor the issue of instructions is
// full (2.1 a cycle; 17 a value forward, 33 backward): 12 warps an SM with 160 registers
// do not hide what they wait for (four blocks in the place of three spill: 137 and 140 us).
#include <type_traits>

#include "per_device.h"
#include "ssm_common.cuh"

namespace rcu {
namespace {

using namespace ssm;

constexpr int NT = 128;
constexpr int AHEAD = 4, BATCHES = 4;  // steps that are read together, and how often in the ring
constexpr int SHORTEST = 16;  // steps of a stretch, at least
constexpr int LONG = 128;     // steps of a stretch that is cut again

// Threads are numbered over groups of VEC channels, then rows (or runs of `per`
// rows), then stretches of `len` steps.
struct Split {
  int groups, runs, per, stretches, len;
  __host__ __device__ int64_t threads() const { return (int64_t)groups * runs * stretches; }
};

// As many stretches as fill the GPU (`room` threads), of SHORTEST steps or more; rows are
// joined where there are more than that.  Long stretches are cut in `waves`, so that the
// last blocks are short ones: the W - 1 inputs that they read again are in the
// second-level cache.  (Forward in four: bf16 T=512 B=256 H=1024, 256 blocks where 456
// fit, 123 -> 118 us; the backward, whose blocks end with their sums, in one: bf16
// T=8192 B=4 H=2048 107 us, 133 in four.)
Split split_of(int T, int B, int H, int vec, int64_t room, int waves) {
  Split s;
  s.groups = ceil_div(H, vec);
  const int64_t items = (int64_t)s.groups * B;
  s.per = (int)std::min<int64_t>(std::max<int64_t>(items / room, 1), B);
  s.runs = ceil_div(B, s.per);
  const int64_t want = std::max<int64_t>(room / ((int64_t)s.groups * s.runs), 1);
  s.len = (int)std::max<int64_t>(ceil_div(T, (int)std::min<int64_t>(want, T)), SHORTEST);
  if (s.len >= LONG) s.len = ceil_div(s.len, waves);
  s.stretches = ceil_div(T, s.len);
  return s;
}

// VEC neighbouring values as pairs (of a single one: with a 0).
template <int VEC>
constexpr int pairs() { return (VEC + 1) / 2; }
template <typename T, int VEC>
__device__ __forceinline__ void widen(const Word<T, VEC> &w, F2 (&v)[pairs<VEC>()]) {
#pragma unroll
  for (int j = 0; j < pairs<VEC>(); ++j)
    v[j] = f2(to_f(w.v[2 * j]), VEC > 1 ? to_f(w.v[VEC > 1 ? 2 * j + 1 : 0]) : 0.f);
}
// LOOSE: value by value, `n` of them there.
template <typename T, int VEC, bool LOOSE = false>
__device__ __forceinline__ Word<T, VEC> word(const T *p, int n = VEC) {
  Word<T, VEC> w;
  if constexpr (LOOSE) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) w.v[j] = p[j < n ? j : 0];
  } else {
    w = *reinterpret_cast<const Word<T, VEC> *>(p);
  }
  return w;
}
template <typename T, int VEC, bool LOOSE = false>
__device__ __forceinline__ void store(T *p, const F2 (&v)[pairs<VEC>()], int n = VEC) {
  Word<T, VEC> w;
#pragma unroll
  for (int j = 0; j < VEC; ++j) w.v[j] = from_f<T>(j % 2 ? hi(v[j / 2]) : lo(v[j / 2]));
  if constexpr (LOOSE) {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < n) p[j] = w.v[j];
  } else {
    *reinterpret_cast<Word<T, VEC> *>(p) = w;
  }
}
__device__ __forceinline__ F2 sigmoid2(F2 v) { return f2(sigmoid(lo(v)), sigmoid(hi(v))); }

// Taps in registers: W, or, for W = 0, room for all the numbers of taps that a
// call may have; the call's w_n are the last ones.
template <int W>
constexpr int taps() { return W ? W : RCU_CONV_MAX_TAPS; }

template <int W, int VEC>
__device__ __forceinline__ void load_taps(const float *weight, const float *bias, int h, int w_n,
                                          F2 (&w)[taps<W>()][pairs<VEC>()], F2 (&add)[pairs<VEC>()],
                                          int n = VEC) {
  constexpr int MW = taps<W>();
#pragma unroll
  for (int j = 0; j < pairs<VEC>(); ++j) {
    const int64_t a = h + 2 * j, b = VEC > 1 && 2 * j + 1 < n ? a + 1 : a;
    add[j] = bias ? f2(bias[a], bias[b]) : f2(0.f);
#pragma unroll
    for (int k = 0; k < MW; ++k)
      w[k][j] = k >= MW - w_n ? f2(weight[a * w_n + k - (MW - w_n)], weight[b * w_n + k - (MW - w_n)])
                              : f2(0.f);
  }
}

// x_t of a row, out of the state for t < 0.
template <typename T, int VEC, bool LOOSE>
struct Row {
  const T *x, *state;  // at channel h; state rows are `wide` apart
  int64_t st;
  int w_n, wide, left;  // left: channels from h on
  __device__ __forceinline__ void at(const T *p, F2 (&v)[pairs<VEC>()]) const {
    widen<T, VEC>(word<T, VEC, LOOSE>(p, left), v);
  }
  __device__ __forceinline__ void at(int t, F2 (&v)[pairs<VEC>()]) const {
    if (t >= 0) {
      at(x + t * st, v);
    } else if (state) {
      at(state + (int64_t)(t + w_n - 1) * wide, v);
    } else {
#pragma unroll
      for (int j = 0; j < pairs<VEC>(); ++j) v[j] = f2(0.f);
    }
  }
  // the w_n - 1 inputs before step t, behind one another at the end of v
  template <int MW>
  __device__ __forceinline__ void before(int t, F2 (&v)[MW][pairs<VEC>()]) const {
#pragma unroll
    for (int k = 1; k < MW; ++k) {
#pragma unroll
      for (int j = 0; j < pairs<VEC>(); ++j) v[k - 1][j] = f2(0.f);
      if (k > MW - w_n) at(t - (MW - k), v[k - 1]);
    }
  }
};
template <typename T, int VEC, bool LOOSE>
__device__ __forceinline__ Row<T, VEC, LOOSE> row_of(const SeqIn &x, const void *state, int b, int h,
                                              int w_n, int H) {
  return {static_cast<const T *>(x.p) + b * x.sb + h,
          state ? static_cast<const T *>(state) + (int64_t)b * (w_n - 1) * H + h : nullptr, x.st,
          w_n, H, H - h};
}
// A thread's steps of a row from t0 to end, AHEAD at a time and BATCHES - 1 such
// batches ahead: words of 4 bytes or more by asynchronous copies, single bf16 values by
// plain reads one batch ahead (as pairs out of the one or two words that they lie in,
// backward T=512 B=64 H=1001 167 us, 150 so).
template <typename T, int VEC, bool LOOSE>
struct Steps {
  static constexpr bool ASYNC = sizeof(T) * VEC >= 4;
  static_assert(!LOOSE || sizeof(T) == 4, "values of 4 bytes");
  static constexpr int BYTES = ASYNC ? BATCHES * AHEAD * NT * sizeof(Word<T, VEC>) : 0;  // of a block
  const T *p;
  int64_t st;
  Word<T, VEC> *ring;
  int end, left, batch;
  Word<T, VEC> next[ASYNC ? 1 : AHEAD];
  __device__ __forceinline__ Steps(const Row<T, VEC, LOOSE> &row, void *room, int end_)
      : p(row.x), st(row.st), ring(static_cast<Word<T, VEC> *>(room) + threadIdx.x), end(end_), left(row.left), batch(0) {}
  template <int N>
  static __device__ __forceinline__ void copy(void *to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from), "n"(N) : "memory");
  }
  __device__ __forceinline__ void fetch(int t, int k) {
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      if (t + q >= end) break;
      const T *from = p + (t + q) * st;
      Word<T, VEC> *to = ring + (k * AHEAD + q) * NT;
      if constexpr (LOOSE) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (j < left) copy<4>(&to->v[j], from + j);
      } else if constexpr (ASYNC) {
        copy<sizeof(Word<T, VEC>)>(to, from);
      } else {
        next[q] = word<T, VEC>(from);
      }
    }
  }
  // the batch at t, once it has arrived
  __device__ __forceinline__ void take(int t, Word<T, VEC> (&w)[AHEAD]) {
    if constexpr (ASYNC) {
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) w[q] = ring[(batch * AHEAD + q) * NT];
      batch = batch == BATCHES - 1 ? 0 : batch + 1;
    } else {
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) w[q] = next[q];
      fetch(t + AHEAD, 0);
    }
  }
};
// The first batches of all of a thread's rows; then, before a batch is taken, the one
// BATCHES - 1 behind it (a group of copies each), and the wait for the batch itself.
template <typename... Rows>
__device__ __forceinline__ void begin(int t0, Rows &...rows) {
  constexpr bool ASYNC = (Rows::ASYNC && ...);
#pragma unroll
  for (int k = 0; k < (ASYNC ? BATCHES - 1 : 1); ++k) {
    (rows.fetch(t0 + k * AHEAD, k), ...);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
}
template <typename... Rows>
__device__ __forceinline__ void ahead(int t, Rows &...rows) {
  if constexpr ((Rows::ASYNC && ...)) {
    (rows.fetch(t + (BATCHES - 1) * AHEAD, rows.batch == 0 ? BATCHES - 1 : rows.batch - 1), ...);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(BATCHES - 1) : "memory");
  }
}

template <int N, int P>
__device__ __forceinline__ void shift(F2 (&v)[N][P]) {
#pragma unroll
  for (int k = 0; k + 1 < N; ++k)
#pragma unroll
    for (int j = 0; j < P; ++j) v[k][j] = v[k + 1][j];
}
// v = bias + taps times window
template <int W, int VEC>
__device__ __forceinline__ void filter(const F2 (&w)[taps<W>()][pairs<VEC>()], int w_n, const F2 (&bias)[pairs<VEC>()],
                                       const F2 (&win)[taps<W>()][pairs<VEC>()], F2 (&v)[pairs<VEC>()]) {
#pragma unroll
  for (int j = 0; j < pairs<VEC>(); ++j) v[j] = bias[j];
#pragma unroll
  for (int k = 0; k < taps<W>(); ++k)
    if (W || k >= taps<W>() - w_n) {
#pragma unroll
      for (int j = 0; j < pairs<VEC>(); ++j) v[j] = fma2(w[k][j], win[k][j], v[j]);
    }
}

template <typename T, int W, int VEC, bool LOOSE>
__global__ void __launch_bounds__(NT) conv_fwd_kernel(const ConvFwd a, const Split sp, int *err) {
  constexpr int MW = taps<W>(), P = pairs<VEC>();
  const int w_n = W ? W : a.W;
  const int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (id >= sp.threads()) return;
  const int h = (int)(id % sp.groups) * VEC, run = (int)(id / sp.groups % sp.runs);
  const int seg = (int)(id / sp.groups / sp.runs);
  extern __shared__ float4 ring[];
  F2 w[MW][P], bias[P];
  load_taps<W, VEC>(a.weight, a.bias, h, w_n, w, bias, a.H - h);
  const int t0 = seg * sp.len, t1 = min(t0 + sp.len, a.T);
  const int last_b = min((run + 1) * sp.per, a.B);
  for (int b = run * sp.per; b < last_b; ++b) {
    const int n = row_length(a.lengths, b, a.T, err), end = min(t1, n);
    const Row<T, VEC, LOOSE> row = row_of<T, VEC, LOOSE>(a.x, a.state, b, h, w_n, a.H);
    T *y = static_cast<T *>(a.y.p) + b * a.y.sb + h;
    Steps<T, VEC, LOOSE> in(row, ring, end);
    begin(t0, in);
    F2 win[MW][P];  // the inputs of a step, the newest last
    if (t0 < end) row.before(t0, win);
    if (seg == 0 && a.state_n) {  // after the window: state_n may be the state itself
      F2 last[MW][P];
      row.before(n, last);
      T *out = static_cast<T *>(a.state_n) + (int64_t)b * (w_n - 1) * a.H + h;
#pragma unroll
      for (int k = 1; k < MW; ++k)
        if (k > MW - w_n) store<T, VEC, LOOSE>(out + (int64_t)(k - 1 - (MW - w_n)) * a.H, last[k - 1], a.H - h);
    }
    int t = t0;
    for (; t < end; t += AHEAD) {
      Word<T, VEC> now[AHEAD];
      ahead(t, in);
      in.take(t, now);
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        if (t + q >= end) break;
        F2 v[P];
        widen<T, VEC>(now[q], win[MW - 1]);
        filter<W, VEC>(w, w_n, bias, win, v);
        if (a.silu) {
#pragma unroll
          for (int j = 0; j < P; ++j) v[j] = mul2(v[j], sigmoid2(v[j]));
        }
        store<T, VEC, LOOSE>(y + (t + q) * a.y.st, v, a.H - h);
        shift(win);
      }
    }
    F2 zero[P];
#pragma unroll
    for (int j = 0; j < P; ++j) zero[j] = f2(0.f);
    for (t = max(t0, end); t < t1; ++t) store<T, VEC, LOOSE>(y + t * a.y.st, zero, a.H - h);
  }
}

// A stretch [t0, t1) of dx needs dv up to W - 1 steps past it; the weights' sums
// take the stretch's own dv.  The first stretch also gives the state's gradient:
// dx at the steps from -(W - 1) on.
template <typename T, int W, int VEC, bool LOOSE>
__global__ void __launch_bounds__(NT) conv_bwd_kernel(const ConvBwd a, const Split sp, float *part,
                                                      int *err) {
  constexpr int MW = taps<W>(), P = pairs<VEC>();
  const int w_n = W ? W : a.W;
  const int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (id >= sp.threads()) return;
  const int h = (int)(id % sp.groups) * VEC, run = (int)(id / sp.groups % sp.runs);
  const int seg = (int)(id / sp.groups / sp.runs);
  extern __shared__ float4 ring[];
  F2 w[MW][P], bias[P], dw[MW][P], db[P], zero[P];
  load_taps<W, VEC>(a.weight, a.bias, h, w_n, w, bias, a.H - h);
#pragma unroll
  for (int j = 0; j < P; ++j) {
    zero[j] = db[j] = f2(0.f);
#pragma unroll
    for (int k = 0; k < MW; ++k) dw[k][j] = f2(0.f);
  }
  const int t0 = seg * sp.len, t1 = min(t0 + sp.len, a.T);
  const int last_b = min((run + 1) * sp.per, a.B);
  for (int b = run * sp.per; b < last_b; ++b) {
    const int n = row_length(a.lengths, b, a.T, err), end = min(t1, n);
    const Row<T, VEC, LOOSE> row = row_of<T, VEC, LOOSE>(a.x, a.state, b, h, w_n, a.H);
    const Row<T, VEC, LOOSE> row_dy = row_of<T, VEC, LOOSE>(a.dy, nullptr, b, h, w_n, a.H);
    T *dx = a.dx.p ? static_cast<T *>(a.dx.p) + b * a.dx.sb + h : nullptr;
    const T *dlast = a.dstate_n ? static_cast<const T *>(a.dstate_n) + (int64_t)b * (w_n - 1) * a.H + h
                                : nullptr;
    T *dstate = a.dstate ? static_cast<T *>(a.dstate) + (int64_t)b * (w_n - 1) * a.H + h : nullptr;
    // steps whose dv is wanted: the stretch and the MW - 1 after it; the ones past
    // the row's end have none, and only bring out what is still on its way
    const int stop = t0 < end || seg == 0 ? end + MW - 1 : t0, live = min(stop, n);
    F2 win[MW][P], grad[MW][P];  // x and dv, the newest last
#pragma unroll
    for (int k = 0; k < MW; ++k)
#pragma unroll
      for (int j = 0; j < P; ++j) grad[k][j] = f2(0.f);
    Steps<T, VEC, LOOSE> in_x(row, ring, live);
    Steps<T, VEC, LOOSE> in_y(row_dy, reinterpret_cast<char *>(ring) + Steps<T, VEC, LOOSE>::BYTES, live);
    begin(t0, in_x, in_y);
    if (t0 < live) row.before(t0, win);
    // Step t with its words; INNER: all that it touches is the row's and the stretch's.
    auto step = [&](auto inner, int t, const Word<T, VEC> &wx, const Word<T, VEC> &wy) {
      constexpr bool INNER = decltype(inner)::value;
      if (INNER || t < n) {
        F2 v[P];
        widen<T, VEC>(wx, win[MW - 1]);
        widen<T, VEC>(wy, grad[MW - 1]);
        if (a.silu) {
          filter<W, VEC>(w, w_n, bias, win, v);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const F2 s = sigmoid2(v[j]);
            const F2 slope = mul2(s, fma2(v[j], fma2(s, f2(-1.f), f2(1.f)), f2(1.f)));
            grad[MW - 1][j] = mul2(grad[MW - 1][j], slope);
          }
        }
        if (INNER || t < t1) {
#pragma unroll
          for (int j = 0; j < P; ++j) db[j] = add2(db[j], grad[MW - 1][j]);
#pragma unroll
          for (int k = 0; k < MW; ++k)
            if (W || k >= MW - w_n) {
#pragma unroll
              for (int j = 0; j < P; ++j) dw[k][j] = fma2(grad[MW - 1][j], win[k][j], dw[k][j]);
            }
        }
      } else {
#pragma unroll
        for (int j = 0; j < P; ++j) grad[MW - 1][j] = f2(0.f);
      }
      // dx of the step MW - 1 back, which tap k met as many steps later as it is from the
      // last one
      const int at = t - (MW - 1);
      if (INNER || (at >= (seg == 0 ? 1 - w_n : t0) && at < end)) {
        F2 v[P];
        if (!INNER && dlast && at >= n - (w_n - 1))
          row.at(dlast + (int64_t)(at - n + w_n - 1) * a.H, v);
        else
#pragma unroll
          for (int j = 0; j < P; ++j) v[j] = f2(0.f);
#pragma unroll
        for (int k = 0; k < MW; ++k) {
          if (W || k >= MW - w_n) {
#pragma unroll
            for (int j = 0; j < P; ++j) v[j] = fma2(w[k][j], grad[MW - 1 - k][j], v[j]);
          }
        }
        if (INNER || at >= 0) {
          if (dx) store<T, VEC, LOOSE>(dx + at * a.dx.st, v, a.H - h);
        } else if (dstate) {
          store<T, VEC, LOOSE>(dstate + (int64_t)(at + w_n - 1) * a.H, v, a.H - h);
        }
      }
      shift(win);
      shift(grad);
    };
    const int from = t0 + MW - 1;  // the step from which on dx comes out for the stretch
    for (int t = t0; t < stop; t += AHEAD) {
      Word<T, VEC> now_x[AHEAD], now_y[AHEAD];
      ahead(t, in_x, in_y);
      in_x.take(t, now_x);
      in_y.take(t, now_y);
      if (t >= from && t + AHEAD <= end) {
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) step(std::true_type(), t + q, now_x[q], now_y[q]);
      } else {
#pragma unroll
        for (int q = 0; q < AHEAD; ++q)
          if (t + q < stop) step(std::false_type(), t + q, now_x[q], now_y[q]);
      }
    }
    if (dx)
      for (int t = max(t0, end); t < t1; ++t) store<T, VEC, LOOSE>(dx + t * a.dx.st, zero, a.H - h);
  }
  if (!part) return;
  // [stretch, run][h, tap | bias]
  float *out = part + ((int64_t)seg * sp.runs + run) * a.H * (w_n + 1);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    if (LOOSE && h + j >= a.H) break;
#pragma unroll
    for (int k = 0; k < MW; ++k)
      if (k >= MW - w_n)
        out[(int64_t)(h + j) * w_n + k - (MW - w_n)] = j % 2 ? hi(dw[k][j / 2]) : lo(dw[k][j / 2]);
    out[(int64_t)a.H * w_n + h + j] = j % 2 ? hi(db[j / 2]) : lo(db[j / 2]);
  }
}

// WORDS: a thread's taps, VEC * W neighbours, as words of 16 bytes.
template <typename T, int W, int VEC, bool WORDS>
__global__ void __launch_bounds__(NT) conv_step_kernel(const ConvStep a, int *err) {
  constexpr int MW = taps<W>(), P = pairs<VEC>();
  const int w_n = W ? W : a.W, groups = a.H / VEC;
  const int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (id >= (int64_t)groups * a.B) return;
  const int h = (int)(id % groups) * VEC;
  const int64_t b = id / groups;
  int64_t slot = a.slot ? a.slot[b] : b;
  if (slot < -1 || slot >= a.slots) {
    atomicCAS(err, (int)DEV_OK, (int)DEV_SLOTS);
    slot = -1;
  }
  T *y = static_cast<T *>(a.y) + b * a.ldy + h;
  F2 v[P];
#pragma unroll
  for (int j = 0; j < P; ++j) v[j] = f2(0.f);
  if (slot >= 0) {
    T *state = static_cast<T *>(a.state) + slot * (w_n - 1) * a.H + h;
    Word<T, VEC> in[MW];  // the window, its last w_n
#pragma unroll
    for (int k = 0; k < MW; ++k)
      if (k >= MW - w_n)
        in[k] = k < MW - 1 ? word<T, VEC>(state + (int64_t)(k - (MW - w_n)) * a.H)
                           : word<T, VEC>(static_cast<const T *>(a.x) + b * a.ldx + h);
    F2 w[MW][P], bias[P], win[MW][P];
    if constexpr (WORDS) {
      float f[VEC * MW];
#pragma unroll
      for (int k = 0; k < VEC * MW; k += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(a.weight + (int64_t)h * W + k);
        f[k] = q.x, f[k + 1] = q.y, f[k + 2] = q.z, f[k + 3] = q.w;
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        bias[j] = a.bias ? f2(a.bias[h + 2 * j], a.bias[h + 2 * j + 1]) : f2(0.f);
#pragma unroll
        for (int k = 0; k < MW; ++k) w[k][j] = f2(f[2 * j * MW + k], f[(2 * j + 1) * MW + k]);
      }
    } else {
      load_taps<W, VEC>(a.weight, a.bias, h, w_n, w, bias);
    }
#pragma unroll
    for (int k = 0; k < MW; ++k)
      if (k >= MW - w_n) {
        if (k > MW - w_n) *reinterpret_cast<Word<T, VEC> *>(state + (int64_t)(k - 1 - (MW - w_n)) * a.H) = in[k];
        widen<T, VEC>(in[k], win[k]);
      }
    filter<W, VEC>(w, w_n, bias, win, v);
    if (a.silu) {
#pragma unroll
      for (int j = 0; j < P; ++j) v[j] = mul2(v[j], sigmoid2(v[j]));
    }
  }
  store<T, VEC>(y, v);
}

// Runs f with the kernel's number of taps: those of the usual widths known to the
// compiler, the others (of threads with one channel or two) not.
constexpr bool usual(int W) { return W >= 2 && W <= 4; }
template <int VEC, typename F>
cudaError_t by_taps(int W, F f) {
  if constexpr (VEC <= 2)
    if (!usual(W)) return f(std::integral_constant<int, 0>());
  switch (W) {
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    default: return cudaErrorInvalidValue;
  }
}

// A kernel's launch: its shared memory allowed, and the threads that fit on the GPU.
struct Room {
  cudaError_t set;
  int64_t threads;
};
template <typename K>
Room room_of(K fn, int bytes, int nsm) {
  Room r{cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes), 0};
  int per = 1;
  cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(&per, fn, NT, bytes, 0);
  r.threads = (int64_t)std::max(per, 1) * nsm * NT;
  return r;
}
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*fn)(KArgs...), const Split &sp, int bytes, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((sp.threads() + NT - 1) / NT));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <typename T, int VEC, bool LOOSE>
cudaError_t fwd(const ConvFwd &p, int *err, int nsm, cudaStream_t s) {
  return by_taps<VEC>(p.W, [&](auto w) {
    auto fn = conv_fwd_kernel<T, decltype(w)::value, VEC, LOOSE>;
    constexpr int bytes = Steps<T, VEC, LOOSE>::BYTES;
    static PerDevice<Room> rooms;
    const Room room = rooms.here([&] { return room_of(fn, bytes, nsm); });
    if (room.set != cudaSuccess) return room.set;
    const Split sp = split_of(p.T, p.B, p.H, VEC, room.threads, 4);
    return launch(fn, sp, bytes, s, p, sp, err);
  });
}
template <typename T, int VEC, bool LOOSE>
cudaError_t bwd(const ConvBwd &p, DevMem &ws, int *err, int nsm, cudaStream_t s, int *launches) {
  return by_taps<VEC>(p.W, [&](auto w) {
    auto fn = conv_bwd_kernel<T, decltype(w)::value, VEC, LOOSE>;
    constexpr int bytes = 2 * Steps<T, VEC, LOOSE>::BYTES;
    static PerDevice<Room> rooms;
    const Room room = rooms.here([&] { return room_of(fn, bytes, nsm); });
    if (room.set != cudaSuccess) return room.set;
    const Split sp = split_of(p.T, p.B, p.H, VEC, room.threads, 1);
    const int64_t rows = (int64_t)sp.runs * sp.stretches, cols = (int64_t)p.H * (p.W + 1);
    float *part = nullptr;
    if (p.dweight || p.dbias) {
      const cudaError_t e = ws.get(rows * cols * 4, &part);
      if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch(fn, sp, bytes, s, p, sp, part, err);
    if (e != cudaSuccess || !part) return e;
    const ColumnSum sum{part, rows, cols, (int64_t)p.H * p.W, p.H, p.dweight, p.dbias, nullptr};
    return launch_column_sum(sum, s, launches);
  });
}

bool fits(const SeqIn &x, const void *state, const void *state_n, int H, int size, int vec) {
  return H % vec == 0 && aligned(x, size, vec) && (!state || aligned(state, H, size, vec)) &&
         (!state_n || aligned(state_n, H, size, vec));
}

// The channels of a thread: as many as words of 16 (backwards 8 of bf16) bytes hold; where
// rows are not aligned to those, or the taps so many that the registers do not hold them,
// two, of bf16 as words of 4 bytes, of fp32 each by itself (LOOSE); of bf16 rows aligned to
// less, one.  W=4 T=512 B=64, forward and backward us: fp32 H=1001 55 and 113 (as single
// values 61 and 151), bf16 H=1002 47 and 75 (64 and 151); H=1024, W=5 in place of 4: 70 and
// 179 in place of 37 and 72 (as single values 119 and 329).
template <int VEC, bool LOOSE = false>
struct Kind {
  static constexpr int vec = VEC;
  static constexpr bool loose = LOOSE;
};
template <typename T, int WIDE, typename Fits, typename Run>
cudaError_t by_kind(int W, bool vec, Fits fit, Run run) {
  if (usual(W) && vec && fit(WIDE)) return run(Kind<WIDE>());
  if constexpr (sizeof(T) == 4) return run(Kind<2, true>());
  else return vec && fit(2) ? run(Kind<2>()) : run(Kind<1>());
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvFwd &p, int *err, int nsm, bool vec, cudaStream_t s,
                            int *launches) {
  ++*launches;
  const int size = p.dtype == RCU_BF16 ? 2 : 4;
  auto fit = [&](int n) { return fits(p.x, p.state, p.state_n, p.H, size, n) && aligned(p.y, size, n); };
  if (p.dtype == RCU_BF16)
    return by_kind<bf16, 8>(p.W, vec, fit, [&](auto k) { return fwd<bf16, k.vec, k.loose>(p, err, nsm, s); });
  return by_kind<float, 4>(p.W, vec, fit, [&](auto k) { return fwd<float, k.vec, k.loose>(p, err, nsm, s); });
}

cudaError_t launch_conv_bwd(const ConvBwd &p, DevMem &ws, int *err, int nsm, bool vec,
                            cudaStream_t s, int *launches) {
  ++*launches;
  const int size = p.dtype == RCU_BF16 ? 2 : 4;
  auto fit = [&](int n) {
    return fits(p.x, p.state, p.dstate_n, p.H, size, n) && fits(p.dy, p.dstate, nullptr, p.H, size, n) &&
           (!p.dx.p || aligned(p.dx, size, n));
  };
  if (p.dtype == RCU_BF16)
    return by_kind<bf16, 4>(p.W, vec, fit,
                            [&](auto k) { return bwd<bf16, k.vec, k.loose>(p, ws, err, nsm, s, launches); });
  return by_kind<float, 4>(p.W, vec, fit,
                           [&](auto k) { return bwd<float, k.vec, k.loose>(p, ws, err, nsm, s, launches); });
}

template <typename T, int VEC, bool WORDS>
static cudaError_t step(const ConvStep &p, int *err, cudaStream_t s) {
  return by_taps<VEC>(p.W, [&](auto w) {
    const int64_t threads = (int64_t)(p.H / VEC) * p.B;
    conv_step_kernel<T, decltype(w)::value, VEC, WORDS>
        <<<(unsigned)((threads + NT - 1) / NT), NT, 0, s>>>(p, err);
    return cudaGetLastError();
  });
}
template <typename T>
static cudaError_t step_of(const ConvStep &p, int *err, bool vec, cudaStream_t s) {
  const bool wide = vec && usual(p.W) && p.H % 4 == 0 && aligned(p.x, p.ldx, sizeof(T), 4) &&
                    aligned(p.y, p.ldy, sizeof(T), 4) && aligned(p.state, p.H, sizeof(T), 4);
  if (!wide) return step<T, 1, false>(p, err, s);
  return aligned(p.weight, 4, 4, 4) ? step<T, 4, true>(p, err, s) : step<T, 4, false>(p, err, s);
}

cudaError_t launch_conv_step(const ConvStep &p, int *err, int nsm, bool vec, cudaStream_t s,
                             int *launches) {
  ++*launches;
  (void)nsm;
  return p.dtype == RCU_BF16 ? step_of<bf16>(p, err, vec, s) : step_of<float>(p, err, vec, s);
}

}  // namespace rcu
