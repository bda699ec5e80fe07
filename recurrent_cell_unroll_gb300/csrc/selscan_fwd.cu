// Selective scan, forward (selscan.cuh has the mathematics and the layout).
#include <type_traits>

#include "per_device.h"
#include "selscan.cuh"

namespace rcu {
namespace {

using namespace selscan;

// MAIN: outputs.  ENDS: a segment's last states from states of 0 (and its sum of
// delta).  GRADS: the same backwards in time of the states' gradients,
//   e <- 2^(delta A2) (e + gy c),  gy = dy, or dy silu(z).
enum Mode { MAIN, ENDS, GRADS };

struct Args {
  ScanIn in;
  SeqIn dy;        // GRADS
  const float *h0; // MAIN: the states that enter segment 0, [n][B][H][N] with more
  SeqOut y;
  float *h_n, *states;
  Meeting m;
  int groups;
  bool wide_states;
};

// Warps of a block: channels of a block are 32 / LANES of each.
template <int LANES>
constexpr int warps() { return LANES == 1 ? 2 : LANES == 2 ? 4 : 8; }

template <typename T, int LANES, int VE, Mode MODE>
__global__ void __launch_bounds__(32 * warps<LANES>()) scan_kernel(const Args a, int *err) {
  constexpr int NT = 32 * warps<LANES>(), CC = NT / LANES, NP = S * LANES;
  __shared__ float2 step_in[TILE][CC];                      // delta, delta x (or gy)
  __shared__ float2 gate[MODE == MAIN ? TILE : 1][CC];      // silu(z), d x silu(z)
  __shared__ alignas(16) float in_w[TILE][NP];              // b (GRADS: c)
  __shared__ alignas(16) float out_w[MODE == MAIN ? TILE : 1][NP];  // c
  const ScanIn &p = a.in;
  const int group = blockIdx.x % a.groups;
  const int b = (int)(blockIdx.x / a.groups % p.B), seg = (int)(blockIdx.x / a.groups / p.B);
  const int tid = threadIdx.x, l = tid % LANES, cl = tid / LANES;
  const int ch0 = group * CC, ch = ch0 + cl, n0 = l * S;
  const bool live = ch < p.H;
  const int here = live ? min(max(p.N - n0, 0), S) : 0;  // states that exist
  const int64_t row = (int64_t)b * p.H + ch;             // of [B][H]
  const int64_t at = row * p.N + n0;                     // of [B][H][N]
  const int64_t table = (int64_t)p.B * p.H * p.N;
  const int n = row_length(p.lengths, b, p.T, err);
  const int t0 = seg * a.m.seg.len, t1 = min(t0 + a.m.seg.len, p.T), end = min(t1, n);

  F2 A2[S / 2], h[S / 2];
  {
    float v[S];
    load_states(p.a_log + (int64_t)ch * p.N + n0, here, a.wide_states && live, v);
#pragma unroll
    for (int k = 0; k < S; ++k) v[k] = k < here ? rate2(v[k]) : 0.f;
#pragma unroll
    for (int k = 0; k < S / 2; ++k) A2[k] = f2(v[2 * k], v[2 * k + 1]);
#pragma unroll
    for (int k = 0; k < S; ++k) v[k] = 0.f;
    if (MODE == MAIN && a.h0 && live)
      load_states(a.h0 + (a.m.seg.n > 1 ? seg * table : 0) + at, here, a.wide_states, v);
#pragma unroll
    for (int k = 0; k < S / 2; ++k) h[k] = f2(v[2 * k], v[2 * k + 1]);
  }
  auto keep = [&](float *to) {
    float v[S];
#pragma unroll
    for (int k = 0; k < S / 2; ++k) v[2 * k] = lo(h[k]), v[2 * k + 1] = hi(h[k]);
    if (live) store_states(to + at, here, a.wide_states, v);
  };

  const T *x = static_cast<const T *>(p.x.p) + b * p.x.sb;
  const T *dt = static_cast<const T *>(p.dt.p) + b * p.dt.sb;
  const T *z = p.z.p ? static_cast<const T *>(p.z.p) + b * p.z.sb : nullptr;
  const T *dy = MODE == GRADS ? static_cast<const T *>(a.dy.p) + b * a.dy.sb : nullptr;
  const SeqIn &wi = MODE == GRADS ? p.c : p.b;
  const T *w1 = static_cast<const T *>(wi.p) + b * wi.sb;
  const T *w2 = static_cast<const T *>(p.c.p) + b * p.c.sb;
  T *y = MODE == MAIN ? static_cast<T *>(a.y.p) + b * a.y.sb : nullptr;

  const bool use_z = z && MODE != ENDS;
  Ahead<T, NT, CC, VE> rx, rdt, rz;
  AheadRows<T, NT, NP> r1, r2;
  auto read = [&](int t) {
    rdt.read(dt, p.dt.st, t, end, ch0, p.H);
    if (MODE == GRADS) rx.read(dy, a.dy.st, t, end, ch0, p.H);
    else rx.read(x, p.x.st, t, end, ch0, p.H);
    if (use_z) rz.read(z, p.z.st, t, end, ch0, p.H);
    r1.read(w1, wi.st, t, end, p.N);
    if (MODE == MAIN) r2.read(w2, p.c.st, t, end, p.N);
  };
  float total = 0.f;  // of delta
  const int tiles = t0 < end ? ceil_div(end - t0, TILE) : 0;
  auto tile_at = [&](int k) { return t0 + (MODE == GRADS ? tiles - 1 - k : k) * TILE; };
  if (tiles) read(tile_at(0));
  for (int k = 0; k < tiles; ++k) {
    const int base = tile_at(k);
    __syncthreads();  // the tile before is done with
#pragma unroll
    for (int q = 0; q < Ahead<T, NT, CC, VE>::EV; ++q) {
      const int t = rx.row(q), c = rx.col(q);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        float2 in = make_float2(0.f, 0.f), g = make_float2(0.f, 0.f);
        if (base + t < end && ch0 + c + j < p.H) {
          const float v = to_f(rx.w[q].v[j]);
          const float delta =
              softplus(to_f(rdt.w[q].v[j]) + (p.dt_bias ? p.dt_bias[ch0 + c + j] : 0.f));
          float silu = 1.f;
          if (use_z) {
            const float zv = to_f(rz.w[q].v[j]);
            silu = zv * sigmoid(zv);
          }
          in = make_float2(delta, MODE == GRADS ? v * silu : delta * v);
          if (MODE == MAIN) g = make_float2(silu, p.d ? p.d[ch0 + c + j] * v * silu : 0.f);
        }
        step_in[t][c + j] = in;
        if (MODE == MAIN) gate[t][c + j] = g;
      }
    }
    r1.put(in_w, base, end, p.N);
    if (MODE == MAIN) r2.put(out_w, base, end, p.N);
    if (k + 1 < tiles) read(tile_at(k + 1));
    __syncthreads();
    if (MODE == MAIN && a.states) keep(a.states + (base / TILE) * table);
    const int steps = min(TILE, end - base);
    if (MODE == MAIN) {
      for (int t = 0; t < steps; t += LANES) {  // steps past the end have delta 0
        float v[LANES];
#pragma unroll
        for (int j = 0; j < LANES; ++j) {
          const float2 in = step_in[t + j][cl];
          F2 bw[S / 2], cw[S / 2], sum;
          load_pairs(&in_w[t + j][n0], bw);
          load_pairs(&out_w[t + j][n0], cw);
          const F2 d2 = f2(in.x), u2 = f2(in.y);
#pragma unroll
          for (int q = 0; q < S / 2; ++q) {
            h[q] = fma2(ex2_2(mul2(d2, A2[q])), h[q], mul2(u2, bw[q]));
            sum = q ? fma2(h[q], cw[q], sum) : mul2(h[q], cw[q]);
          }
          v[j] = lo(sum) + hi(sum);
        }
        const float s = sum_over_lanes<LANES>(v, l);
        if (t + l < steps && live) {
          const float2 g = gate[t + l][cl];
          y[(base + t + l) * a.y.st + ch] = from_f<T>(fmaf(s, g.x, g.y));
        }
      }
    } else {
#pragma unroll 4
      for (int j = 0; j < steps; ++j) {
        const int t = MODE == GRADS ? steps - 1 - j : j;
        const float2 in = step_in[t][cl];
        F2 w[S / 2];
        load_pairs(&in_w[t][n0], w);
        const F2 d2 = f2(in.x), u2 = f2(in.y);
        total += in.x;
#pragma unroll
        for (int q = 0; q < S / 2; ++q) {
          const F2 decay = ex2_2(mul2(d2, A2[q]));
          h[q] = MODE == GRADS ? mul2(decay, fma2(u2, w[q], h[q])) : fma2(decay, h[q], mul2(u2, w[q]));
        }
      }
    }
  }
  if (MODE != MAIN) {
    keep(a.m.end + seg * table);
    if (live && l == 0) a.m.sums[(int64_t)seg * p.B * p.H + row] = total;
    return;
  }
  // what lies past the row's end
  if (a.states)
    for (int t = t0 + tiles * TILE; t < t1; t += TILE) keep(a.states + (t / TILE) * table);
  if (a.h_n && seg == a.m.seg.n - 1) keep(a.h_n);
  if (live)
    for (int t = max(t0, end) + l; t < t1; t += LANES) y[t * a.y.st + ch] = from_f<T>(0.f);
}

// The states that enter each segment, in the place of those that it ended with
// from states of 0: a thread a state.
template <bool BACKWARDS>
__global__ void __launch_bounds__(128) chain_kernel(const float *a_log, const float *first, Meeting m,
                                                    int B, int H, int N) {
  wait_for_previous();
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x, table = (int64_t)B * H * N;
  if (i >= table) return;
  const int64_t row = i / N, rows = (int64_t)B * H;
  const float A2 = rate2(a_log[i % ((int64_t)H * N)]);
  float h = first ? first[i] : 0.f;
  for (int k = 0; k < m.seg.n; ++k) {
    const int s = BACKWARDS ? m.seg.n - 1 - k : k;
    const float own = m.end[s * table + i], decay = ex2(A2 * m.sums[s * rows + row]);
    m.end[s * table + i] = h;
    h = fmaf(decay, h, own);
  }
}

template <typename T, int LANES, int VE, Mode MODE>
cudaError_t run(Args a, int *err, cudaStream_t s, int *launches) {
  constexpr int NT = 32 * warps<LANES>();
  a.groups = ceil_div(a.in.H, NT / LANES);
  ++*launches;
  const int64_t blocks = (int64_t)a.groups * a.in.B * a.m.seg.n;
  scan_kernel<T, LANES, VE, MODE><<<(unsigned)blocks, NT, 0, s>>>(a, err);
  return cudaGetLastError();
}

template <Mode MODE>
cudaError_t dispatch(const Args &a, bool vec, int *err, cudaStream_t s, int *launches) {
  const ScanIn &p = a.in;
  const int size = p.dtype == RCU_BF16 ? 2 : 4;
  const bool wide = vec && p.H % 4 == 0 && aligned(p.x, size, 4) && aligned(p.dt, size, 4) &&
                    (!p.z.p || aligned(p.z, size, 4)) && (MODE != GRADS || aligned(a.dy, size, 4));
  return by_lanes(p.N, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    if (p.dtype == RCU_BF16)
      return wide ? run<bf16, L, 4, MODE>(a, err, s, launches) : run<bf16, L, 1, MODE>(a, err, s, launches);
    return wide ? run<float, L, 4, MODE>(a, err, s, launches) : run<float, L, 1, MODE>(a, err, s, launches);
  });
}

bool wide_states(const ScanIn &p, bool vec, std::initializer_list<const void *> tables) {
  if (!vec || p.N % S) return false;
  for (const void *t : tables)
    if (t && !aligned(t, 4, 4, 4)) return false;
  return true;
}

}  // namespace

namespace selscan {

cudaError_t launch_local(const ScanIn &p, bool backwards, const SeqIn &dy, const float *first,
                         const Meeting &m, int *err, bool vec, cudaStream_t s, int *launches) {
  Args a{};
  a.in = p;
  a.dy = dy;
  a.m = m;
  a.wide_states = wide_states(p, vec, {p.a_log, m.end});
  const cudaError_t e = backwards ? dispatch<GRADS>(a, vec, err, s, launches)
                                  : dispatch<ENDS>(a, vec, err, s, launches);
  if (e != cudaSuccess) return e;
  ++*launches;
  const dim3 grid((unsigned)(((int64_t)p.B * p.H * p.N + 127) / 128));
  return launch_after(backwards ? chain_kernel<true> : chain_kernel<false>, grid, 128, s, p.a_log,
                      first, m, p.B, p.H, p.N);
}

}  // namespace selscan

cudaError_t launch_scan_fwd(const ScanFwd &p, DevMem &ws, int *err, int nsm, bool vec,
                            cudaStream_t s, int *launches) {
  const ScanIn &in = p.in;
  const int64_t table = (int64_t)in.B * in.H * in.N;
  Args a{};
  a.in = in;
  a.h0 = p.h0;
  a.y = p.y;
  a.h_n = p.h_n;
  a.states = p.states;
  // a block holds 64 channels (32 of those with more than 32 states)
  const int64_t blocks = (int64_t)ceil_div(in.H, in.N > 32 ? 32 : 64) * in.B;
  a.m.seg = segments_of(in.T, blocks, 4 * (int64_t)nsm);
  if (a.m.seg.n > 1) {
    const cudaError_t e = ws.get((size_t)a.m.seg.n * (table + (int64_t)in.B * in.H) * 4, &a.m.end);
    if (e != cudaSuccess) return e;
    a.m.sums = a.m.end + a.m.seg.n * table;
    const cudaError_t l = launch_local(in, false, SeqIn{}, p.h0, a.m, err, vec, s, launches);
    if (l != cudaSuccess) return l;
    a.h0 = a.m.end;
  }
  a.wide_states = wide_states(in, vec, {in.a_log, a.h0, p.h_n, p.states});
  return dispatch<MAIN>(a, vec, err, s, launches);
}

}  // namespace rcu
