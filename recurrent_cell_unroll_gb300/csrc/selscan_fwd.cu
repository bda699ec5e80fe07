// Selective scan, forward (selscan.cuh has the mathematics and the layout).
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
  bool wide_states, wide_bc;
};

// A thread has S states of K neighbouring channels, as pairs of channels; the LANES
// threads that hold a channel's N stand side by side in a warp.  With four channels a
// thread, what it reads of shared memory (their steps and inputs, and b and c of its
// states: a 16-byte read takes four cycles, whoever shares it) is one word a state and
// step; with two it was 2.5, and the reads bound the kernel (T=300 B=64 H=2048 263 us,
// 217 with four).  Tiles are of half a chunk: seven blocks then fit an SM, three with
// whole ones (201 and 286 us).
//
// Measured, bf16, N=16: T=300 B=64 H=2048 203 us, 3.1e12 states a second, where the
// special function unit would take 83 and the issue of 118 instructions a channel and
// step 120; T=2048 B=8 H=2048 285 us, in four segments (some 110 of them for their ends);
// T=65536 B=1 H=512 297.
constexpr int S = 4, K = 4, P = K / 2, TILE = CHUNK / 2;
template <int LANES>
struct Shape {
  static constexpr int WARPS = LANES / 2;  // of a block
  static constexpr int NT = 32 * WARPS, CC = NT / LANES * K, NP = S * LANES;
  // sums over a channel's states come in PARTS, added as they are read; the first two
  // are where the steps' delta and input stood
  static constexpr int PARTS = LANES < 4 ? LANES : 4;
  static constexpr int BUF = TILE * CC + 8;  // floats: parts 8 banks apart
};
template <typename T, int LANES, bool ALIGNED, Mode MODE>
constexpr int shared_bytes() {
  typedef Shape<LANES> Sh;
  typedef Fetch<T, Sh::NT, TILE, Sh::CC, ALIGNED> F;
  return (MODE == MAIN ? Sh::PARTS : 2) * Sh::BUF * 4 + (MODE == MAIN ? 2 : 1) * TILE * Sh::NP * 4 +
         2 * (MODE == ENDS ? 2 : 3) * TILE * F::RS * (int)sizeof(T);
}

// WHOLE: the lanes' states are all a channel's (or no sums over them are asked for).
template <typename T, int LANES, bool ALIGNED, Mode MODE, bool WHOLE>
__global__ void __launch_bounds__(Shape<LANES>::NT, LANES == 4 ? 7 : 1) scan_kernel(const Args a, int *err) {
  typedef Shape<LANES> Sh;
  constexpr int NT = Sh::NT, CC = Sh::CC, NP = Sh::NP, BUF = Sh::BUF, PARTS = Sh::PARTS;
  constexpr int U = 4;                 // steps worked on together
  constexpr int RAW = MODE == ENDS ? 2 : 3;
  constexpr int ROW = CC / 4, EV = (TILE * ROW + NT - 1) / NT;  // words of four of a thread, of the same channels
  constexpr bool IDLE = TILE * ROW < NT;  // some threads have none
  typedef Fetch<T, NT, TILE, CC, ALIGNED> F;
  constexpr int RS = F::RS;
  constexpr bool SHIFTS = F::SHIFTS;
  extern __shared__ float4 shared4[];
  float *buf = reinterpret_cast<float *>(shared4);                     // [PARTS][BUF]: delta, input
  float(*in_w)[NP] = reinterpret_cast<float(*)[NP]>(buf + (MODE == MAIN ? PARTS : 2) * BUF);  // b (GRADS: c)
  float(*out_w)[NP] = in_w + TILE;                                    // MAIN: c
  T(*raw)[TILE][RS] = reinterpret_cast<T(*)[TILE][RS]>(MODE == MAIN ? out_w + TILE : in_w + TILE);
  const ScanIn &p = a.in;
  const int group = blockIdx.x % a.groups;
  // GRADS: of all segments but the first; ENDS: but the last (by the grid)
  const int b = (int)(blockIdx.x / a.groups % p.B), seg = (int)(blockIdx.x / a.groups / p.B) + (MODE == GRADS);
  const int tid = threadIdx.x, l = tid % LANES, own = tid / LANES * K;  // own: of the block's channels
  const int ch0 = group * CC, n0 = l * S;
  const int64_t table = (int64_t)p.B * p.H * p.N;
  const int n = row_length(p.lengths, b, p.T, err);
  const int t0 = seg * a.m.seg.len, t1 = min(t0 + a.m.seg.len, p.T), end = min(t1, n);

  const SeqIn &sx = MODE == GRADS ? a.dy : p.x, &sw = MODE == GRADS ? p.c : p.b;
  const F fdt(static_cast<const T *>(p.dt.p) + b * p.dt.sb, p.dt.st, ch0, p.H);
  const F fx(static_cast<const T *>(sx.p) + b * sx.sb, sx.st, ch0, p.H);
  const bool use_z = p.z.p && MODE != ENDS;
  const F fz(static_cast<const T *>(p.z.p) + (use_z ? b * p.z.sb : 0), p.z.st, ch0, p.H);
  const bool words = sizeof(T) == 4 && a.wide_bc;
  Weights<T, NT, TILE, NP> r1(static_cast<const T *>(sw.p) + b * sw.sb, sw.st, p.N, words);
  Weights<T, NT, TILE, NP> r2(static_cast<const T *>(p.c.p) + b * p.c.sb, p.c.st, p.N, words);
  T *y = MODE == MAIN ? static_cast<T *>(a.y.p) + b * a.y.sb : nullptr;

  const int tiles = t0 < end ? ceil_div(end - t0, TILE) : 0;
  auto tile_at = [&](int k) { return t0 + (MODE == GRADS ? tiles - 1 - k : k) * TILE; };
  // tile k's rows, into the buffers of its parity
  auto start = [&](int k) {
    T(*to)[TILE][RS] = raw + k % 2 * RAW;
    const int t = tile_at(k);
    fdt.start(to[0], t, end);
    fx.start(to[1], t, end);
    if (use_z) fz.start(to[RAW - 1], t, end);
    r1.read(t, end);
    if (MODE == MAIN) r2.read(t, end);
  };
  if (tiles) start(0);

  int here[K];          // states that exist
  const int exist = p.N - n0;  // the same of a channel that exists
  F2 A2[P][S], h[P][S]; // of pairs of channels
#pragma unroll
  for (int c = 0; c < K; c += 2) {
    float r[2][S], v[2][S];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int ch = ch0 + own + c + j;
      here[c + j] = ch < p.H ? min(max(p.N - n0, 0), S) : 0;
      load_states(p.a_log + (int64_t)ch * p.N + n0, here[c + j], a.wide_states, r[j]);
#pragma unroll
      for (int k = 0; k < S; ++k) {
        r[j][k] = k < here[c + j] ? rate2(r[j][k]) : 0.f;
        v[j][k] = 0.f;
      }
      if (MODE == MAIN && a.h0)
        load_states(a.h0 + (a.m.seg.n > 1 ? seg * table : 0) + ((int64_t)b * p.H + ch) * p.N + n0, here[c + j],
                    a.wide_states, v[j]);
    }
#pragma unroll
    for (int k = 0; k < S; ++k) A2[c / 2][k] = f2(r[0][k], r[1][k]), h[c / 2][k] = f2(v[0][k], v[1][k]);
  }
  auto keep = [&](float *to) {
    to += ((int64_t)b * p.H + ch0 + own) * p.N + n0;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      float v[S];
#pragma unroll
      for (int k = 0; k < S; ++k) v[k] = c % 2 ? hi(h[c / 2][k]) : lo(h[c / 2][k]);
      store_states(to + (int64_t)c * p.N, here[c], a.wide_states, v);
    }
  };
  const int col = tid % ROW * 4, row0 = tid / ROW;  // of the thread's words: rows NT / ROW apart
  const Four bias = constants(p.dt_bias, ch0 + col, p.H);
  const Four skip = constants(MODE == MAIN ? p.d : nullptr, ch0 + col, p.H);
  F2 total[P] = {};  // of delta

  for (int k = 0; k < tiles; ++k) {
    const int base = tile_at(k), steps = min(TILE, end - base);
    T(*now)[TILE][RS] = raw + k % 2 * RAW;
    if (k == 0) {
      fetched();
      __syncthreads();
    }
    F2 probe = f2(0.f);  // !WHOLE: NaN where an input of the states is not finite
#pragma unroll
    for (int q = 0; q < EV; ++q) {
      const int r = row0 + q * (NT / ROW);
      if (IDLE && r >= TILE) break;
      Four v = four<SHIFTS>(now[0][r], col, fdt.shift(base, r)), u = four<SHIFTS>(now[1][r], col, fx.shift(base, r));
      v.a = softplus(add2(v.a, bias.a)), v.b = softplus(add2(v.b, bias.b));
      if (MODE != GRADS) {
        u.a = mul2(v.a, u.a), u.b = mul2(v.b, u.b);
      } else if (use_z) {
        const Four g = four<SHIFTS>(now[RAW - 1][r], col, fz.shift(base, r));
        u.a = mul2(u.a, silu(g.a)), u.b = mul2(u.b, silu(g.b));
      }
      // steps past the end have delta and input 0, and so leave the states alone
      if (steps < TILE && r >= steps) v = u = {f2(0.f), f2(0.f)};
      put_four(buf + r * CC + col, v);
      put_four(buf + BUF + r * CC + col, u);
      if (!WHOLE) probe = fma2(u.b, f2(0.f), fma2(u.a, f2(0.f), probe));
    }
    r1.put(in_w);
    if (MODE == MAIN) r2.put(out_w);
    // A state that does not exist has weights of 0, and stays 0 but for infinite inputs: then
    // it must be kept out of the sums, where it would be NaN.  (Selects at every step, with all
    // inputs, N=16 T=300 B=64 H=2048 bf16 206 -> 241 us.)
    bool careful = false;
    if (WHOLE) __syncthreads();
    else careful = __syncthreads_or(isnan(lo(probe)) || isnan(hi(probe)));
    if (k + 1 < tiles) start(k + 1);
    if (MODE == MAIN && a.states && base % CHUNK == 0) keep(a.states + (base / CHUNK) * table);

    const int groups = ceil_div(steps, U);
    auto work = [&](auto care) {
      constexpr bool CAREFUL = decltype(care)::value;
      for (int g = 0; g < groups; ++g) {
        F2 decay[U][P][S], add[U][P][S];
        const int first = MODE == GRADS ? (groups - 1 - g) * U : g * U;
#pragma unroll
        for (int j = 0; j < U; ++j) {
          F2 d[P], in[P];
          float w[S];
          load_pairs<P>(buf + (first + j) * CC + own, d);
          load_pairs<P>(buf + BUF + (first + j) * CC + own, in);
          load_row(in_w[first + j] + n0, w);
#pragma unroll
          for (int c = 0; c < P; ++c) {
            if (MODE != MAIN) total[c] = add2(total[c], d[c]);
#pragma unroll
            for (int q = 0; q < S; ++q) {
              decay[j][c][q] = ex2_2(mul2(d[c], A2[c][q]));
              add[j][c][q] = mul2(in[c], f2(w[q]));
            }
          }
        }
        F2 v[U][P];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int j = MODE == GRADS ? U - 1 - i : i;
          float w[S];
          if (MODE == MAIN) load_row(out_w[first + j] + n0, w);
#pragma unroll
          for (int c = 0; c < P; ++c)
#pragma unroll
            for (int q = 0; q < S; ++q) {
              F2 &s = h[c][q];
              if (MODE == GRADS) s = mul2(decay[j][c][q], add2(add[j][c][q], s));
              else s = fma2(decay[j][c][q], s, add[j][c][q]);
              if (MODE != MAIN) continue;
              if (CAREFUL && q >= exist) s = f2(0.f);
              v[j][c] = q ? fma2(s, f2(w[q]), v[j][c]) : mul2(s, f2(w[q]));
            }
        }
        if (MODE == MAIN) {
          // down to PARTS lanes: of 8, every half of them takes two of the steps, of 16, a
          // quarter one
          int at = 0, count = U * P;
          F2 *sum = &v[0][0];
#pragma unroll
          for (int o = LANES / 2; o >= PARTS; o /= 2) {
            count /= 2;
            const bool upper = l & o;
            at += upper ? count : 0;
#pragma unroll
            for (int j = 0; j < U * P / 2; ++j)
              if (j < count) {
                const F2 mine = upper ? sum[j + count] : sum[j], other = upper ? sum[j] : sum[j + count];
                sum[j] = add2(mine, __shfl_xor_sync(0xffffffffu, other, o));
              }
          }
          __syncwarp();  // the parts stand where the warp's other lanes have read from
          float *to = buf + l % PARTS * BUF + (first + at / P) * CC + own;
          if (count >= P) {
#pragma unroll
            for (int j = 0; j < U; ++j)
              if (j * P < count)
                *reinterpret_cast<float4 *>(to + j * CC) = make_float4(lo(v[j][0]), hi(v[j][0]), lo(v[j][1]), hi(v[j][1]));
          } else {
            *reinterpret_cast<F2 *>(to + at % P * 2) = sum[0];
          }
        }
      }
    };
    if (!WHOLE && careful) work(std::true_type());
    else work(std::false_type());
    fetched();
    __syncthreads();
    if (MODE == MAIN) {
      // y = (sum + d x) silu(z)
#pragma unroll
      for (int q = 0; q < EV; ++q) {
        const int r = row0 + q * (NT / ROW);
        if (r >= steps) break;
        Four v = four(buf + r * CC + col);
#pragma unroll
        for (int k2 = 1; k2 < PARTS; ++k2) {
          const Four more = four(buf + k2 * BUF + r * CC + col);
          v.a = add2(v.a, more.a), v.b = add2(v.b, more.b);
        }
        if (p.d) {
          const Four xs = four<SHIFTS>(now[1][r], col, fx.shift(base, r));
          v.a = fma2(skip.a, xs.a, v.a), v.b = fma2(skip.b, xs.b, v.b);
        }
        if (use_z) {
          const Four g = four<SHIFTS>(now[RAW - 1][r], col, fz.shift(base, r));
          v.a = mul2(v.a, silu(g.a)), v.b = mul2(v.b, silu(g.b));
        }
        T *to = y + (base + r) * a.y.st + ch0 + col;
        if (ALIGNED) {
          if (ch0 + col < p.H) put_four(to, v);
        } else {
          const float out[4] = {lo(v.a), hi(v.a), lo(v.b), hi(v.b)};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (ch0 + col + j < p.H) to[j] = from_f<T>(out[j]);
        }
      }
    }
  }
  if (MODE != MAIN) {
    keep(a.m.end + seg * table);
    if (l == 0) {
      float *to = a.m.sums + ((int64_t)seg * p.B + b) * p.H + ch0 + own;
#pragma unroll
      for (int c = 0; c < K; ++c)
        if (here[c]) to[c] = c % 2 ? hi(total[c / 2]) : lo(total[c / 2]);
    }
    return;
  }
  // what lies past the row's end
  if (a.states)
    for (int t = t0 + round_up(tiles * TILE, CHUNK); t < t1; t += CHUNK) keep(a.states + (t / CHUNK) * table);
  if (a.h_n && seg == a.m.seg.n - 1) keep(a.h_n);
  const int past = max(t0, end);
  for (int64_t i = tid; i < (int64_t)(t1 - past) * CC; i += NT) {
    const int c = ch0 + (int)(i % CC);
    if (c < p.H) y[(past + i / CC) * a.y.st + c] = from_f<T>(0.f);
  }
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
  constexpr int READ = 16;  // segments in flight
  for (int k0 = 0; k0 < m.seg.n; k0 += READ) {
    float own[READ], sum[READ];
#pragma unroll
    for (int k = 0; k < READ; ++k) {
      const int s = BACKWARDS ? m.seg.n - 1 - k0 - k : k0 + k;
      if (k0 + k < m.seg.n - 1) own[k] = m.end[s * table + i], sum[k] = m.sums[s * rows + row];
    }
#pragma unroll
    for (int k = 0; k < READ; ++k) {
      if (k0 + k >= m.seg.n) break;
      m.end[(BACKWARDS ? m.seg.n - 1 - k0 - k : k0 + k) * table + i] = h;
      if (k0 + k == m.seg.n - 1) break;  // nothing follows the last
      float decay = A2 * sum[k];
      // an infinite state is kept infinite by decays above 0, though their product be 0 in fp32
      if (isinf(h) && !isinf(decay)) decay = fmaxf(decay, -100.f);
      h = fmaf(ex2(decay), h, own[k]);
    }
  }
}

template <typename T, int LANES, bool ALIGNED, Mode MODE, bool WHOLE>
cudaError_t run(Args a, int *err, cudaStream_t s, int *launches) {
  typedef Shape<LANES> Sh;
  constexpr int bytes = shared_bytes<T, LANES, ALIGNED, MODE>();
  auto fn = scan_kernel<T, LANES, ALIGNED, MODE, WHOLE>;
  static PerDevice<cudaError_t> ready;
  const cudaError_t set =
      ready.here([&] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
  if (set != cudaSuccess) return set;
  a.groups = ceil_div(a.in.H, Sh::CC);
  ++*launches;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)a.groups * a.in.B * (a.m.seg.n - (MODE != MAIN))));
  cfg.blockDim = dim3(Sh::NT);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, fn, a, err);
}

template <typename T, Mode MODE, int LANES>
cudaError_t of_lanes(const Args &a, bool aligned, int *err, cudaStream_t s, int *launches) {
  if constexpr (MODE == MAIN)
    if (a.in.N < Shape<LANES>::NP)
      return aligned ? run<T, LANES, true, MODE, false>(a, err, s, launches)
                     : run<T, LANES, false, MODE, false>(a, err, s, launches);
  return aligned ? run<T, LANES, true, MODE, true>(a, err, s, launches)
                 : run<T, LANES, false, MODE, true>(a, err, s, launches);
}
template <typename T, Mode MODE>
cudaError_t of_type(const Args &a, bool aligned, int *err, cudaStream_t s, int *launches) {
  const int N = a.in.N;
  // of four states or fewer, half of the lanes' are idle: a kernel for those alone was no
  // faster (N=4 T=512 H=1024: bf16 B=16 82 us, 74 so, B=64 197 and 155)
  if (N <= 8) return of_lanes<T, MODE, 2>(a, aligned, err, s, launches);
  if (N <= 16) return of_lanes<T, MODE, 4>(a, aligned, err, s, launches);
  if (N <= 32) return of_lanes<T, MODE, 8>(a, aligned, err, s, launches);
  return of_lanes<T, MODE, 16>(a, aligned, err, s, launches);
}
template <Mode MODE>
cudaError_t dispatch(Args a, bool vec, int *err, cudaStream_t s, int *launches) {
  const ScanIn &p = a.in;
  const int size = p.dtype == RCU_BF16 ? 2 : 4, n = 16 / size;
  const bool wide = vec && p.H % n == 0 && aligned(p.x, size, n) && aligned(p.dt, size, n) &&
                    (!p.z.p || aligned(p.z, size, n)) && (MODE != GRADS || aligned(a.dy, size, n)) &&
                    (MODE != MAIN || aligned(a.y, size, n));
  // fp32 by words (T=512 N=16 H=1024: B=16 107 -> 103 us, B=64 232 -> 226); bf16 value by value,
  // with no other way in its kernels (T=300 B=64 H=2048 204 us, by words 226)
  a.wide_bc = vec && p.dtype == RCU_F32 && p.N % 4 == 0 && aligned(MODE == GRADS ? p.c : p.b, 4, 4) &&
              (MODE != MAIN || aligned(p.c, 4, 4));
  return p.dtype == RCU_BF16 ? of_type<bf16, MODE>(a, wide, err, s, launches)
                             : of_type<float, MODE>(a, wide, err, s, launches);
}

bool wide_states(const ScanIn &p, bool vec, std::initializer_list<const void *> tables) {
  if (!vec || p.N % 4) return false;
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
  const int64_t blocks = (int64_t)ceil_div(in.H, 64) * in.B;
  a.m.seg = segments_of(in.T, blocks, nsm, 8);
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
