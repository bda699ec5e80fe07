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
// one before it.
#include <type_traits>

#include "per_device.h"
#include "ssm_common.cuh"

namespace rcu {
namespace {

using namespace ssm;

constexpr int NT = 128;
constexpr int AHEAD = 8;      // steps whose reads are in flight together
constexpr int SHORTEST = 16;  // steps of a stretch, at least

// Threads are numbered over groups of VEC channels, then rows (or runs of `per`
// rows), then stretches of `len` steps.
struct Split {
  int groups, runs, per, stretches, len;
  __host__ __device__ int64_t threads() const { return (int64_t)groups * runs * stretches; }
};

// As many stretches as fill the GPU (`room` threads), rows joined where there
// are more than that; a stretch of at least SHORTEST steps.
Split split_of(int T, int B, int H, int vec, int64_t room) {
  Split s;
  s.groups = ceil_div(H, vec);
  const int64_t items = (int64_t)s.groups * B;
  s.per = (int)std::min<int64_t>(std::max<int64_t>(items / room, 1), B);
  s.runs = ceil_div(B, s.per);
  const int64_t want = std::max<int64_t>(room / ((int64_t)s.groups * s.runs), 1);
  s.len = (int)std::max<int64_t>(ceil_div(T, (int)std::min<int64_t>(want, T)), SHORTEST);
  s.stretches = ceil_div(T, s.len);
  return s;
}

template <typename T, int VEC>
__device__ __forceinline__ void load(const T *p, float (&v)[VEC]) {
  const Word<T, VEC> w = *reinterpret_cast<const Word<T, VEC> *>(p);
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = to_f(w.v[j]);
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T *p, const float (&v)[VEC]) {
  Word<T, VEC> w;
#pragma unroll
  for (int j = 0; j < VEC; ++j) w.v[j] = from_f<T>(v[j]);
  *reinterpret_cast<Word<T, VEC> *>(p) = w;
}

// Taps in registers: W, or, for W = 0, room for all the numbers of taps that a
// call may have; the call's w_n are the last ones.
template <int W>
constexpr int taps() { return W ? W : RCU_CONV_MAX_TAPS; }

template <int W, int VEC>
__device__ __forceinline__ void load_taps(const float *weight, const float *bias, int h, int w_n,
                                          float (&w)[taps<W>()][VEC], float (&add)[VEC]) {
  constexpr int MW = taps<W>();
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    add[j] = bias ? bias[h + j] : 0.f;
#pragma unroll
    for (int k = 0; k < MW; ++k)
      w[k][j] = k >= MW - w_n ? weight[(int64_t)(h + j) * w_n + k - (MW - w_n)] : 0.f;
  }
}

// x_t of a row, out of the state for t < 0.
template <typename T, int VEC>
struct Row {
  const T *x, *state;  // at channel h; state rows are `wide` apart
  int64_t st;
  int w_n, wide;
  __device__ __forceinline__ void at(int t, float (&v)[VEC]) const {
    if (t >= 0) {
      load<T, VEC>(x + t * st, v);
    } else if (state) {
      load<T, VEC>(state + (int64_t)(t + w_n - 1) * wide, v);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = 0.f;
    }
  }
  // the w_n - 1 inputs before step t, behind one another at the end of v
  template <int MW>
  __device__ __forceinline__ void before(int t, float (&v)[MW][VEC]) const {
#pragma unroll
    for (int k = 1; k < MW; ++k) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[k - 1][j] = 0.f;
      if (k > MW - w_n) at(t - (MW - k), v[k - 1]);
    }
  }
};
template <typename T, int VEC>
__device__ __forceinline__ Row<T, VEC> row_of(const SeqIn &x, const void *state, int b, int h,
                                              int w_n, int H) {
  return {static_cast<const T *>(x.p) + b * x.sb + h,
          state ? static_cast<const T *>(state) + (int64_t)b * (w_n - 1) * H + h : nullptr, x.st,
          w_n, H};
}

template <typename T, int W, int VEC>
__global__ void __launch_bounds__(NT) conv_fwd_kernel(const ConvFwd a, const Split sp, int *err) {
  constexpr int MW = taps<W>();
  const int w_n = W ? W : a.W;
  const int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (id >= sp.threads()) return;
  const int h = (int)(id % sp.groups) * VEC, run = (int)(id / sp.groups % sp.runs);
  const int seg = (int)(id / sp.groups / sp.runs);
  float w[MW][VEC], bias[VEC];
  load_taps<W, VEC>(a.weight, a.bias, h, w_n, w, bias);
  const int t0 = seg * sp.len, t1 = min(t0 + sp.len, a.T);
  const int last_b = min((run + 1) * sp.per, a.B);
  for (int b = run * sp.per; b < last_b; ++b) {
    const int n = row_length(a.lengths, b, a.T, err), end = min(t1, n);
    const Row<T, VEC> row = row_of<T, VEC>(a.x, a.state, b, h, w_n, a.H);
    T *y = static_cast<T *>(a.y.p) + b * a.y.sb + h;
    float win[MW][VEC];  // the inputs of a step, the newest last
    if (t0 < end) row.before(t0, win);
    if (seg == 0 && a.state_n) {  // after the window: state_n may be the state itself
      float last[MW][VEC];
      row.before(n, last);
      T *out = static_cast<T *>(a.state_n) + (int64_t)b * (w_n - 1) * a.H + h;
#pragma unroll
      for (int k = 1; k < MW; ++k)
        if (k > MW - w_n) store<T, VEC>(out + (int64_t)(k - 1 - (MW - w_n)) * a.H, last[k - 1]);
    }
    int t = t0;
    for (; t < end; t += AHEAD) {
      Word<T, VEC> raw[AHEAD];
#pragma unroll
      for (int q = 0; q < AHEAD; ++q)
        if (t + q < end) raw[q] = *reinterpret_cast<const Word<T, VEC> *>(row.x + (t + q) * row.st);
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        if (t + q >= end) break;
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          win[MW - 1][j] = to_f(raw[q].v[j]);
          v[j] = bias[j];
        }
#pragma unroll
        for (int k = 0; k < MW; ++k)
          if (W || k >= MW - w_n) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = fmaf(w[k][j], win[k][j], v[j]);
          }
        if (a.silu) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[j] *= sigmoid(v[j]);
        }
        store<T, VEC>(y + (t + q) * a.y.st, v);
#pragma unroll
        for (int k = 0; k + 1 < MW; ++k)
#pragma unroll
          for (int j = 0; j < VEC; ++j) win[k][j] = win[k + 1][j];
      }
    }
    const float zero[VEC] = {};
    for (t = max(t0, end); t < t1; ++t) store<T, VEC>(y + t * a.y.st, zero);
  }
}

// A stretch [t0, t1) of dx needs dv up to W - 1 steps past it; the weights' sums
// take the stretch's own dv.  The first stretch also gives the state's gradient:
// dx at the steps from -(W - 1) on.
template <typename T, int W, int VEC>
__global__ void __launch_bounds__(NT) conv_bwd_kernel(const ConvBwd a, const Split sp, float *part,
                                                      int *err) {
  constexpr int MW = taps<W>(), READ = 4;
  const int w_n = W ? W : a.W;
  const int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (id >= sp.threads()) return;
  const int h = (int)(id % sp.groups) * VEC, run = (int)(id / sp.groups % sp.runs);
  const int seg = (int)(id / sp.groups / sp.runs);
  float w[MW][VEC], bias[VEC], dw[MW][VEC] = {}, db[VEC] = {};
  load_taps<W, VEC>(a.weight, a.bias, h, w_n, w, bias);
  const int t0 = seg * sp.len, t1 = min(t0 + sp.len, a.T);
  const int last_b = min((run + 1) * sp.per, a.B);
  for (int b = run * sp.per; b < last_b; ++b) {
    const int n = row_length(a.lengths, b, a.T, err), end = min(t1, n);
    const Row<T, VEC> row = row_of<T, VEC>(a.x, a.state, b, h, w_n, a.H);
    const T *dy = static_cast<const T *>(a.dy.p) + b * a.dy.sb + h;
    T *dx = a.dx.p ? static_cast<T *>(a.dx.p) + b * a.dx.sb + h : nullptr;
    const T *dlast = a.dstate_n ? static_cast<const T *>(a.dstate_n) + (int64_t)b * (w_n - 1) * a.H + h
                                : nullptr;
    T *dstate = a.dstate ? static_cast<T *>(a.dstate) + (int64_t)b * (w_n - 1) * a.H + h : nullptr;
    // steps whose dv is wanted: the stretch and the W - 1 after it; the ones past
    // the row's end have none, and only bring out what is still on its way
    const int stop = t0 < end || seg == 0 ? end + w_n - 1 : t0;
    float win[MW][VEC], grad[MW][VEC] = {};  // x and dv, the newest last
    if (stop > t0 && t0 < n) row.before(t0, win);
    for (int t = t0; t < stop; t += READ) {
      Word<T, VEC> rx[READ], ry[READ];
#pragma unroll
      for (int q = 0; q < READ; ++q)
        if (t + q < stop && t + q < n) {
          rx[q] = *reinterpret_cast<const Word<T, VEC> *>(row.x + (t + q) * row.st);
          ry[q] = *reinterpret_cast<const Word<T, VEC> *>(dy + (t + q) * a.dy.st);
        }
#pragma unroll
      for (int q = 0; q < READ; ++q) {
        if (t + q >= stop) break;
#pragma unroll
        for (int j = 0; j < VEC; ++j) grad[MW - 1][j] = 0.f;
        if (t + q < n) {
          float v[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            win[MW - 1][j] = to_f(rx[q].v[j]);
            v[j] = bias[j];
          }
          if (a.silu) {
#pragma unroll
            for (int k = 0; k < MW; ++k)
              if (W || k >= MW - w_n) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] = fmaf(w[k][j], win[k][j], v[j]);
              }
          }
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float s = sigmoid(v[j]);
            const float slope = a.silu ? s * fmaf(v[j], 1.f - s, 1.f) : 1.f;
            grad[MW - 1][j] = to_f(ry[q].v[j]) * slope;
          }
          if (t + q < t1) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) db[j] += grad[MW - 1][j];
#pragma unroll
            for (int k = 0; k < MW; ++k)
              if (W || k >= MW - w_n) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) dw[k][j] = fmaf(grad[MW - 1][j], win[k][j], dw[k][j]);
              }
          }
        }
        // dx of the step w_n - 1 back: tap k met it at the gradient that stands at
        // MW - 1 - k behind the oldest of the w_n
        const int at = t + q - (w_n - 1);
        if ((at >= t0 || seg == 0) && at < end) {
          float v[VEC] = {};
          if (dlast && at >= n - (w_n - 1)) load<T, VEC>(dlast + (int64_t)(at - n + w_n - 1) * a.H, v);
#pragma unroll
          for (int k = 0; k < MW; ++k)
            if (W || k >= MW - w_n) {
#pragma unroll
              for (int j = 0; j < VEC; ++j) {
                const int newest = MW - 1 - k + (MW - w_n);  // of the gradients in grad
                if (W) {
                  v[j] = fmaf(w[k][j], grad[MW - 1 - k][j], v[j]);
                } else {
#pragma unroll
                  for (int m = 0; m < MW; ++m)
                    if (m == newest) v[j] = fmaf(w[k][j], grad[m][j], v[j]);
                }
              }
            }
          if (at >= 0) {
            if (dx) store<T, VEC>(dx + at * a.dx.st, v);
          } else if (dstate) {
            store<T, VEC>(dstate + (int64_t)(at + w_n - 1) * a.H, v);
          }
        }
#pragma unroll
        for (int k = 0; k + 1 < MW; ++k)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            win[k][j] = win[k + 1][j];
            grad[k][j] = grad[k + 1][j];
          }
      }
    }
    if (dx) {
      const float zero[VEC] = {};
      for (int t = max(t0, end); t < t1; ++t) store<T, VEC>(dx + t * a.dx.st, zero);
    }
  }
  if (!part) return;
  // [stretch, run][h, tap | bias]
  float *out = part + ((int64_t)seg * sp.runs + run) * a.H * (w_n + 1);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
#pragma unroll
    for (int k = 0; k < MW; ++k)
      if (k >= MW - w_n) out[(int64_t)(h + j) * w_n + k - (MW - w_n)] = dw[k][j];
    out[(int64_t)a.H * w_n + h + j] = db[j];
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(NT) conv_step_kernel(const ConvStep a, int *err) {
  const int groups = a.H / VEC;
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
  float v[VEC] = {};
  if (slot >= 0) {
    T *state = static_cast<T *>(a.state) + slot * (a.W - 1) * a.H + h;
    const Word<T, VEC> now =
        *reinterpret_cast<const Word<T, VEC> *>(static_cast<const T *>(a.x) + b * a.ldx + h);
    Word<T, VEC> in[RCU_CONV_MAX_TAPS];
#pragma unroll
    for (int k = 0; k < RCU_CONV_MAX_TAPS; ++k)
      if (k < a.W)
        in[k] = k < a.W - 1 ? *reinterpret_cast<const Word<T, VEC> *>(state + (int64_t)k * a.H) : now;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = a.bias ? a.bias[h + j] : 0.f;
#pragma unroll
    for (int k = 0; k < RCU_CONV_MAX_TAPS; ++k)
      if (k < a.W) {
        if (k) *reinterpret_cast<Word<T, VEC> *>(state + (int64_t)(k - 1) * a.H) = in[k];
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          v[j] = fmaf(a.weight[(int64_t)(h + j) * a.W + k], to_f(in[k].v[j]), v[j]);
      }
    if (a.silu) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] *= sigmoid(v[j]);
    }
  }
  store<T, VEC>(y, v);
}

// Runs f with the kernel's number of taps: those of the usual widths known to the
// compiler, the others (of threads with one channel) not.
constexpr bool usual(int W) { return W >= 2 && W <= 4; }
template <int VEC, typename F>
cudaError_t by_taps(int W, F f) {
  switch (W) {
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    default:
      if constexpr (VEC == 1) return f(std::integral_constant<int, 0>());
      return cudaErrorInvalidValue;
  }
}

// Threads of a kernel that fit on the GPU.
template <typename K>
int64_t room_of(K fn, int nsm) {
  int per = 1;
  cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(&per, fn, NT, 0, 0);
  return (int64_t)std::max(per, 1) * nsm * NT;
}

template <typename T, int VEC>
cudaError_t fwd(const ConvFwd &p, int *err, int nsm, cudaStream_t s) {
  return by_taps<VEC>(p.W, [&](auto w) {
    auto fn = conv_fwd_kernel<T, decltype(w)::value, VEC>;
    static PerDevice<int64_t> room;
    const Split sp = split_of(p.T, p.B, p.H, VEC, room.here([&] { return room_of(fn, nsm); }));
    fn<<<(unsigned)((sp.threads() + NT - 1) / NT), NT, 0, s>>>(p, sp, err);
    return cudaGetLastError();
  });
}
template <typename T, int VEC>
cudaError_t bwd(const ConvBwd &p, DevMem &ws, int *err, int nsm, cudaStream_t s, int *launches) {
  return by_taps<VEC>(p.W, [&](auto w) {
    auto fn = conv_bwd_kernel<T, decltype(w)::value, VEC>;
    static PerDevice<int64_t> room;
    const Split sp = split_of(p.T, p.B, p.H, VEC, room.here([&] { return room_of(fn, nsm); }));
    const int64_t rows = (int64_t)sp.runs * sp.stretches, cols = (int64_t)p.H * (p.W + 1);
    float *part = nullptr;
    if (p.dweight || p.dbias) {
      const cudaError_t e = ws.get(rows * cols * 4, &part);
      if (e != cudaSuccess) return e;
    }
    fn<<<(unsigned)((sp.threads() + NT - 1) / NT), NT, 0, s>>>(p, sp, part, err);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !part) return e;
    const ColumnSum sum{part, rows, cols, (int64_t)p.H * p.W, p.H, p.dweight, p.dbias, nullptr};
    return launch_column_sum(sum, s, launches);
  });
}

bool fits(const SeqIn &x, const void *state, const void *state_n, int H, int size, int vec) {
  return H % vec == 0 && aligned(x, size, vec) && (!state || aligned(state, H, size, vec)) &&
         (!state_n || aligned(state_n, H, size, vec));
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvFwd &p, int *err, int nsm, bool vec, cudaStream_t s,
                            int *launches) {
  ++*launches;
  const int size = p.dtype == RCU_BF16 ? 2 : 4, n = 16 / size;
  const bool wide = vec && usual(p.W) && fits(p.x, p.state, p.state_n, p.H, size, n) &&
                    aligned(p.y, size, n);
  if (p.dtype == RCU_BF16)
    return wide ? fwd<bf16, 8>(p, err, nsm, s) : fwd<bf16, 1>(p, err, nsm, s);
  return wide ? fwd<float, 4>(p, err, nsm, s) : fwd<float, 1>(p, err, nsm, s);
}

cudaError_t launch_conv_bwd(const ConvBwd &p, DevMem &ws, int *err, int nsm, bool vec,
                            cudaStream_t s, int *launches) {
  ++*launches;
  const int size = p.dtype == RCU_BF16 ? 2 : 4;
  const bool wide = vec && usual(p.W) && fits(p.x, p.state, p.dstate_n, p.H, size, 4) &&
                    fits(p.dy, p.dstate, nullptr, p.H, size, 4) &&
                    (!p.dx.p || aligned(p.dx, size, 4));
  if (p.dtype == RCU_BF16)
    return wide ? bwd<bf16, 4>(p, ws, err, nsm, s, launches) : bwd<bf16, 1>(p, ws, err, nsm, s, launches);
  return wide ? bwd<float, 4>(p, ws, err, nsm, s, launches) : bwd<float, 1>(p, ws, err, nsm, s, launches);
}

cudaError_t launch_conv_step(const ConvStep &p, int *err, int nsm, bool vec, cudaStream_t s,
                             int *launches) {
  ++*launches;
  (void)nsm;
  const int size = p.dtype == RCU_BF16 ? 2 : 4;
  const bool wide = vec && p.H % 4 == 0 && aligned(p.x, p.ldx, size, 4) &&
                    aligned(p.y, p.ldy, size, 4) && aligned(p.state, p.H, size, 4);
  const int64_t threads = (int64_t)(wide ? p.H / 4 : p.H) * p.B;
  const unsigned blocks = (unsigned)((threads + NT - 1) / NT);
  if (p.dtype == RCU_BF16) {
    if (wide) conv_step_kernel<bf16, 4><<<blocks, NT, 0, s>>>(p, err);
    else conv_step_kernel<bf16, 1><<<blocks, NT, 0, s>>>(p, err);
  } else {
    if (wide) conv_step_kernel<float, 4><<<blocks, NT, 0, s>>>(p, err);
    else conv_step_kernel<float, 1><<<blocks, NT, 0, s>>>(p, err);
  }
  return cudaGetLastError();
}

}  // namespace rcu
