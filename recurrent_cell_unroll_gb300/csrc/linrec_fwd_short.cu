// Gated linear recurrence, forward, for short sequences of many rows: a warp has a
// row's channels to itself.
//
// The tiled kernel gives each of its warps 16 of a tile's 64 steps, which short
// sequences leave idle, and runs every step twice.  Here a warp runs them once, one
// after another; nothing is exchanged, and N steps' reads are in flight together.
// It stays with its channels, whose constants it keeps, from one batch row to the
// next.  Bound by the reads' latency: 24 warps an SM with 12 words each in flight (8
// steps at once and 16 warps took 32 us where this took 25, bf16 T=20 B=250 H=2048).
//
// How far it pays goes by the rows, as for the backward.  In us, here and tiled:
//   bf16   B=250 H=2048 T=4 20 and 40, T=20 29 and 45, T=32 41 and 43; B=900 H=1024 T=32
//          65 and 86; off TMA, T=64: B=250 H=2046 77 and 92, B=100 H=1922 35 and 41;
//          split words: B=250 H=2047 T=12 66 and 70, T=16 87 and 74; B=900 H=1023 T=16
//          117 and 133; B=100 H=1921 T=20 24 and 35
//   fp32   B=250 H=2048 T=20 39 and 64, T=32 57 and 62; off TMA, T=64: B=250 H=2047 105
//          and 116, B=60 H=1985 31 and 33
#include "linrec_bwd.cuh"

namespace rcu {
namespace {

using namespace linrec;

constexpr int NW = 4, NT = 32 * NW, N = 4, PER_SM = 6;  // N: steps whose reads are in flight together
// the most steps: of TMA's rows; of others; of split words, by steps_within()
constexpr int SHORT_T = 32, SHORT_LOOSE = CHUNK, SHORT_SPLIT = 20;

// each: warps that share a group's rows; words: bit k: input k's (x, r, i) values of a lane are one word; bit 3: the output's
template <typename T>
__global__ void __launch_bounds__(NT, PER_SM)
    linrec_fwd_short_kernel(const LinrecFwd p, const int groups, const int each, const int words,
                            int *err) {
  constexpr int CPT = Shape<T>::CPT, CW = Shape<T>::CW;
  constexpr int BATCH = CPT == 2 ? N : N / 2;  // the N steps at once: pairs of channels, or of steps
  typedef typename Lane<T>::V V;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int w = blockIdx.x * NW + warp, c0 = w % groups * CW;
  if (w >= each * groups) return;
  const int ch = c0 + lane * CPT, live = min(max(p.H - ch, 0), CPT);
  V k2, zero, minus;
  set(zero, 0.f);
  set(minus, -1.f);
  rate(p.lambda + ch, p.c, live, k2);
  const Limits lim = limits(k2);
  const bool small = __all_sync(0xffffffffu, small_rate(k2));
  const float scale[3][N] = {};

  uint32_t raw[3][N];
  auto load = [&](int64_t b, int t0, int len) {
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const int64_t t = t0 + s;
      const int on = t < len ? live : 0;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const SeqIn &in = (&p.x)[k];
        raw[k][s] = global_raw<T, CPT>(static_cast<const T *>(in.p) + t * in.st + b * in.sb + ch, on,
                                       words >> k & 1);
      }
    }
  };
  for (int64_t b = w / groups; b < p.B; b += each) {
    const int64_t row = b * p.H + ch;
    const int len = row_length(p.lengths, (int)b, p.T, err);
    load(b, 0, len);
    V h = zero;
    if (p.h0) load_v(p.h0 + row, live, h);
    if (p.states) store_v(p.states + row, h, live);  // one: T is at most a chunk
    T *y = static_cast<T *>(p.y.p) + b * p.y.sb + ch;
    for (int t0 = 0; t0 < p.T; t0 += N) {
      V em1[N], nb[N], ns[N], ng[N];
      if (small) gates<T, true, BATCH>(raw, scale, k2, lim, em1, nb, ns, ng);
      else gates<T, false, BATCH>(raw, scale, k2, lim, em1, nb, ns, ng);
      if (t0 + N < len) load(b, t0 + N, len);
#pragma unroll
      for (int s = 0; s < N; ++s) {
        if (t0 + s < len) h = fma_v(nb[s], minus, fma_v(em1[s], h, h));
        if (t0 + s < p.T) store_raw(y, t0 + s < len ? h : zero, live, words >> 3 & 1);
        y += p.y.st;
      }
    }
    if (p.h_n) store_v(p.h_n + row, h, live);
  }
}

template <typename T>
Warps warps(const LinrecFwd &p) {
  static PerDevice<int> rooms;
  const int room = rooms.here([] { return resident_blocks(linrec_fwd_short_kernel<T>, NT, 0); });
  return warps_of(p.B, ceil_div(p.H, Shape<T>::CW), room, NW);
}

template <typename T>
cudaError_t run(const LinrecFwd &p, int *err, cudaStream_t s, int *launches) {
  const int groups = ceil_div(p.H, Shape<T>::CW);
  const Warps w = warps<T>(p);
  auto whole = [](const void *q, int64_t st, int64_t sb) {
    constexpr int bytes = Shape<T>::CPT * (int)sizeof(T);
    return reinterpret_cast<uintptr_t>(q) % bytes == 0 && st * (int)sizeof(T) % bytes == 0 &&
           sb * (int)sizeof(T) % bytes == 0;
  };
  const int words = whole(p.x.p, p.x.st, p.x.sb) | whole(p.r.p, p.r.st, p.r.sb) << 1 |
                    whole(p.i.p, p.i.st, p.i.sb) << 2 | whole(p.y.p, p.y.st, p.y.sb) << 3;
  linrec_fwd_short_kernel<T><<<w.blocks, NT, 0, s>>>(p, groups, w.each, words, err);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace

bool linrec::short_fwd_pays(const LinrecFwd &p, int resident_blocks, bool vec) {
  const bool half = p.dtype == RCU_BF16;
  const int groups = ceil_div(p.H, half ? Shape<bf16>::CW : Shape<float>::CW);
  if (p.T > SHORT_LOOSE || (int64_t)p.B * groups < resident_blocks) return false;
  // whether all rows start on multiples of `to` bytes
  auto aligned = [&](int to) {
    const SeqIn y{p.y.p, p.y.st, p.y.sb, nullptr}, *at[4] = {&p.x, &p.r, &p.i, &y};
    const int size = half ? 2 : 4;
    for (const SeqIn *t : at)
      if (reinterpret_cast<uintptr_t>(t->p) % to || t->st * size % to || t->sb * size % to)
        return false;
    return true;
  };
  if (vec && aligned(16)) return p.T <= SHORT_T;
  return aligned(4) || steps_within(p.T, p.B, warps<bf16>(p), SHORT_SPLIT);
}

cudaError_t linrec::launch_short_fwd(const LinrecFwd &p, int *err, cudaStream_t s, int *launches) {
  return p.dtype == RCU_BF16 ? run<bf16>(p, err, s, launches) : run<float>(p, err, s, launches);
}

}  // namespace rcu
