// Gated linear recurrence, backward, for short sequences of many rows: a warp has a
// row's channels to itself.
//
// The tiled kernel gives each of its warps 8 of a tile's 64 steps, which short
// sequences leave idle, and joins them with a barrier a tile.  Here a warp runs all
// steps, first forwards, keeping the states in shared memory, then backwards with
// the gates made again; nothing is exchanged.  It stays with its channels, whose
// constants it keeps, from one batch row to the next.  Making the gates twice tells
// with the length: bf16 B=250 H=2048 takes 90 us here and 120 tiled at 20 steps, 164
// and 124 at 40.
//
// How far it pays goes by the rows: those that TMA cannot address cost the tiled kernel
// more, and this one only where a lane's values are not a word.  In us, here and tiled:
//   bf16   T=20: B=188 H=1920 72 and 73, H=1922 75 and 115; B=80 H=1984 38 and 38;
//          split words: B=188 H=1921 T=9 108 and 113, T=10 118 and 113; B=700 H=1023
//          T=8 160 and 183; B=80 H=1985 T=8 34 and 51
//          from 8 bits: B=188 H=1920 T=9 77 and 86, T=10 88 and 87; B=700 H=1024 T=8
//          125 and 163, T=11 170 and 165; B=80 H=1984 T=14 43 and 47
//   fp32   T=20: B=188 H=1920 86 and 100, B=60 H=1984 36 and 52; B=700 H=1024 T=17 149
//          and 246; T=44, off TMA: B=188 H=1921 172 and 204, B=60 H=1985 70 and 70
#include "linrec_bwd.cuh"

namespace rcu {
namespace {

using namespace linrec;

constexpr int NW = 4, NT = 32 * NW, N = 4;  // N: steps whose reads are in flight together
// the most steps: at all; of pairs from 8 bits; of fp32 rows off TMA; of split words; and
// of pairs from 8 bits or split words by steps_within(), where warps have many rows each
constexpr int SHORT_T = 20, SHORT_Q8 = 16, SHORT_LOOSE = 44, SHORT_SPLIT = 12, SHORT_MANY = 12;

// Of a block's states.  Below what a launch may have without asking: what a kernel is
// allowed beyond that is one setting for all the process's threads.
template <typename T>
constexpr size_t state_bytes(int steps) {
  return (size_t)NW * steps * 32 * sizeof(typename Lane<T>::V);
}
template <typename T>
constexpr int most_steps() {
  return sizeof(T) == 4 ? std::max(SHORT_T, SHORT_LOOSE) : std::max({SHORT_T, SHORT_Q8, SHORT_SPLIT});
}
static_assert(std::max(state_bytes<float>(most_steps<float>()), state_bytes<bf16>(most_steps<bf16>())) <=
                  48 << 10,
              "a block's states fit the default limit");

template <typename IT, typename T>
__global__ void __launch_bounds__(NT, 3)
    linrec_bwd_short_kernel(const LinrecBwd p, const int groups, const int each,
                            float *__restrict__ partial, const int words, int *err) {
  constexpr int CPT = Shape<T>::CPT, CW = Shape<T>::CW;
  constexpr bool Q8 = sizeof(IT) == 1;
  typedef typename Lane<T>::V V;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  V *before = reinterpret_cast<V *>(smem) + (size_t)warp * p.T * 32 + lane;  // the state before t
  const int w = blockIdx.x * NW + warp, c0 = w % groups * CW;
  if (w >= each * groups) return;
  const int ch = c0 + lane * CPT, live = min(max(p.H - ch, 0), CPT);
  const int nb8 = ceil_div(p.H, BLOCK8);
  V k2, nk, zero, minus;
  set(zero, 0.f);
  set(minus, -1.f);
  rate(p.lambda + ch, p.c, live, k2);
  const Limits lim = limits(k2);
  const bool small = __all_sync(0xffffffffu, small_rate(k2));
  set(nk, -1.f / LOG2E);
  nk = mul_v(nk, k2);  // -K

  uint32_t raw[3][N], rawd[N];
  float scale[3][N];
  int top = FREE_EXP;  // the largest of the gates' exponents
  auto load = [&](int64_t b, int t0, int len, bool with_dy) {
    top = FREE_EXP;
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const int64_t t = t0 + s;
      const int on = t < len ? live : 0;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const SeqIn &in = (&p.x)[k];
        raw[k][s] = global_raw<IT, CPT>(static_cast<const IT *>(in.p) + t * in.st + b * in.sb + ch,
                                        on, words >> k & 1);
        if (Q8) {
          const int e = on ? (int)__ldg(in.e + (t * p.et + b * p.eb) * nb8 + c0 / BLOCK8) : FREE_EXP;
          if (k) top = max(top, e);
          scale[k][s] = power2(e) * (k ? -LOG2E : 1.f);
        }
      }
      if (with_dy)
        rawd[s] = global_raw<T, CPT>(static_cast<const T *>(p.dy.p) + t * p.dy.st + b * p.dy.sb + ch,
                                     on, words >> 3 & 1);
    }
  };
  V em1[N], nb[N], ns[N], ng[N];
  auto make_gates = [&](int t0, int len) {
    if (small && top <= FREE_EXP) gates<IT, true, 2>(raw, scale, k2, lim, em1, nb, ns, ng);
    else gates<IT, false, 2>(raw, scale, k2, lim, em1, nb, ns, ng);
    if (Q8) spoil_codes<CPT>(raw, em1, nb, ns, ng);
    if (t0 + N > len) {
#pragma unroll
      for (int s = 0; s < N; ++s)
        if (t0 + s >= len) em1[s] = nb[s] = ns[s] = ng[s] = 0;
    }
  };
  for (int64_t b = w / groups; b < p.B; b += each) {
    const int64_t row = b * p.H + ch;
    const int len = row_length(p.lengths, (int)b, p.T, err);
    V h, nc = zero, sum = zero;
    load_v(p.states + row, live, h);
    if (p.dh_n) load_v(p.dh_n + row, live, nc);
    nc = neg_v(nc);
    load(b, 0, len, false);
    for (int t0 = 0; t0 < len; t0 += N) {
      make_gates(t0, len);
      if (t0 + N < len) load(b, t0 + N, len, false);
#pragma unroll
      for (int s = 0; s < N; ++s) {
        if (t0 + s < len) before[(t0 + s) * 32] = h;
        h = fma_v(nb[s], minus, fma_v(em1[s], h, h));
      }
    }
    T *out[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const SeqOut &o = (&p.dx)[k];
      out[k] = static_cast<T *>(o.p) + b * o.sb + ch;
    }
    auto store = [&](int k, int64_t t, V v) {
      const SeqOut &o = (&p.dx)[k];
      if (o.p) store_raw(out[k] + t * o.st, v, live, words >> (4 + k) & 1);
    };
    for (int t = p.T - 1; t >= len; --t)
#pragma unroll
      for (int k = 0; k < 3; ++k) store(k, t, zero);
    int t0 = len > 0 ? (len - 1) / N * N : -N;
    if (t0 >= 0) load(b, t0, len, true);
    for (; t0 >= 0; t0 -= N) {
      make_gates(t0, len);
      V dy[N];
#pragma unroll
      for (int s = 0; s < N; ++s) dy[s] = Decode<T, V>::x(rawd[s], 0.f);
      if (t0 > 0) load(b, t0 - N, len, true);
#pragma unroll
      for (int s = N - 1; s >= 0; --s) {
        if (t0 + s >= len) continue;
        const V ne = fma_v(dy[s], minus, nc);
        nc = fma_v(em1[s], ne, ne);
        V hp = before[(t0 + s) * 32], gx, gr, gi, gl;
        grads(em1[s], nb[s], ns[s], ng[s], nk, ne, hp, gx, gr, gi, gl);
        sum = add_v(sum, gl);
        store(0, t0 + s, gx);
        store(1, t0 + s, gr);
        store(2, t0 + s, gi);
      }
    }
    if (p.dh0) store_v(p.dh0 + row, neg_v(nc), live);
    if (p.dlambda) store_v(partial + row, sum, live);
  }
}

template <typename IT, typename T>
Warps warps(const LinrecBwd &p) {
  static PerDevice<int> rooms;
  const int room = rooms.here([] {
    return resident_blocks(linrec_bwd_short_kernel<IT, T>, NT, state_bytes<T>(most_steps<T>()));
  });
  return warps_of(p.B, ceil_div(p.H, Shape<T>::CW), room, NW);
}

template <typename IT, typename T>
cudaError_t run(const LinrecBwd &p, DevMem &ws, int *err, cudaStream_t s, int *launches) {
  const int groups = ceil_div(p.H, Shape<T>::CW);
  const size_t smem = state_bytes<T>(p.T);
  auto fn = linrec_bwd_short_kernel<IT, T>;
  const Warps w = warps<IT, T>(p);
  const SeqIn *in[4] = {&p.x, &p.r, &p.i, &p.dy};
  const SeqOut *out[3] = {&p.dx, &p.dr, &p.di};
  auto whole = [](const void *q, int64_t st, int64_t sb, int size) {
    const int bytes = Shape<T>::CPT * size;
    return reinterpret_cast<uintptr_t>(q) % bytes == 0 && st * size % bytes == 0 &&
           sb * size % bytes == 0;
  };
  int words = 0;
  for (int k = 0; k < 4; ++k)
    words |= whole(in[k]->p, in[k]->st, in[k]->sb, k < 3 ? sizeof(IT) : sizeof(T)) << k;
  for (int k = 0; k < 3; ++k)
    words |= whole(out[k]->p, out[k]->st, out[k]->sb, sizeof(T)) << (4 + k);
  float *partial = nullptr;
  if (p.dlambda) {
    const cudaError_t e = ws.get((size_t)p.B * p.H * 4, &partial);
    if (e != cudaSuccess) return e;
  }
  fn<<<w.blocks, NT, smem, s>>>(p, groups, w.each, partial, words, err);
  ++*launches;
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.dlambda) return e;
  ++*launches;
  return launch_dlambda(partial, p.B, p, s);
}

}  // namespace

bool linrec::short_bwd_pays(const LinrecBwd &p, int resident_blocks, bool vec) {
  const bool half = p.dtype == RCU_BF16;
  const int groups = ceil_div(p.H, half ? Shape<bf16>::CW : Shape<float>::CW);
  if (p.T > SHORT_LOOSE || (int64_t)p.B * groups < resident_blocks) return false;
  // whether the inputs' rows start on multiples of `bytes` (8-bit ones of `bytes8`)
  auto aligned = [&](int bytes, int bytes8) {
    const SeqIn *in[4] = {&p.x, &p.r, &p.i, &p.dy};
    for (int k = 0; k < 4; ++k) {
      const bool q8 = k < 3 && p.saved == RCU_I8;
      const int size = q8 ? 1 : half ? 2 : 4, to = q8 ? bytes8 : bytes;
      if (reinterpret_cast<uintptr_t>(in[k]->p) % to || in[k]->st * size % to ||
          in[k]->sb * size % to)
        return false;
    }
    return true;
  };
  if (!half) return p.T <= (vec && aligned(16, 16) ? SHORT_T : SHORT_LOOSE);
  const bool q8 = p.saved == RCU_I8;
  const bool whole = aligned(4, 2);
  if (!q8 && whole) return p.T <= SHORT_T;
  if (p.T > (whole ? SHORT_Q8 : SHORT_SPLIT)) return false;
  const Warps w = q8 ? warps<int8_t, bf16>(p) : warps<bf16, bf16>(p);
  return p.B <= 2 * w.each || steps_within(p.T, p.B, w, SHORT_MANY);
}

cudaError_t linrec::launch_short_bwd(const LinrecBwd &p, DevMem &ws, int *err, cudaStream_t s,
                                     int *launches) {
  const bool q8 = p.saved == RCU_I8;
  if (p.dtype == RCU_BF16)
    return q8 ? run<int8_t, bf16>(p, ws, err, s, launches)
              : run<bf16, bf16>(p, ws, err, s, launches);
  return q8 ? run<int8_t, float>(p, ws, err, s, launches)
            : run<float, float>(p, ws, err, s, launches);
}

}  // namespace rcu
