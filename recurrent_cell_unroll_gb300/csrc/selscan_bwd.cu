// Selective scan, backward (selscan.cuh has the mathematics and the layout).
//
//   gy = dy silu(z), s_t = sum_n c h_t + d x,     dz = dy s silu'(z)
//   e_t[n] = gy_t c_t[n] + a_{t+1}[n] e_{t+1}[n]  (the gradient reaching a state)
//   dx = delta sum_n e b + gy d,   ddelta = sum_n e (a A h_{t-1} + b x)
//   db_t[n] = sum_ch e delta x,    dc_t[n] = sum_ch gy h_t,   da_log = A sum e a h_{t-1} delta
//
// A block takes the chunks of 32 steps from the last to the first.  In a chunk it
// runs the states forward from the kept ones, leaving those before every fourth
// step in shared memory, then takes four steps at a time backwards: their states
// once more, in registers, and the gradients against them.
//
// A thread has S states of K neighbouring channels, a warp all states of its own
// channels, so only the sums over channels (db, dc) leave a warp.  They are what
// costs beside the exponentials: a thread adds its two channels' first, the lanes of the
// same states halve theirs with one another (7 shuffles; exchanged in shared memory N=16
// 504 us, 488 so, N=64 1060 and 979), and the warps' sums stand where the checkpoint of the
// four steps was.  Sums over states are left in parts by the lanes, and added by the lanes
// that compute the outputs, as words of two channels.
//
// Two channels a thread and not four, though those read less of shared memory: 8 warps
// an SM in the place of 6 (bf16, N=16, T=2048 B=8 H=1024 1190 -> 802 us, 544 now).  Three blocks
// an SM, at 168 registers, were no faster (the decays kept 1015 us, computed again 928,
// two blocks 755).
//
// Measured, N=16: bf16 T=8192 B=2 H=1024 (19 segments) 480 us, of which 100 for their ends
// and 32 for chaining and sums; fp32 T=500 B=32 H=512, mixed lengths, 194.  Bf16 T=512 B=16
// H=1024: N=8 227, 16 277, 32 436, 64 969.  Issue bound: 27 instructions a state and step
// at 2.0 a cycle.
#include "selscan.cuh"

namespace rcu {
namespace {

using namespace selscan;

constexpr int TILE = CHUNK;                // steps of a tile: those between two kept states
constexpr int SUB = 4, SUBS = TILE / SUB;  // steps in registers, and groups of them in a chunk
constexpr int S = 4, K = 2;                // states and channels (a pair) of a thread
constexpr int SLOT = 32 * K * S;           // floats of a warp's checkpoint

struct Args {
  ScanBwd p;
  int groups;            // blocks of channels
  Segments seg;
  const float *enter;    // [seg][B][H][N]: gradients that enter each segment, or dh_n
  float *part_bc;        // [groups][T][B][2][N], or NULL
  float *part;           // [B * seg][H N | H | H], or NULL
  bool wide_states, wide_bc;
};

template <int LANES>
struct Shape {
  static constexpr int NP = S * LANES;
  static constexpr int WC = 32 / LANES * K;                    // channels of a warp
  static constexpr int WARPS = LANES == 2 ? 2 : 4;             // of a block
  static constexpr int NT = 32 * WARPS, CC = WC * WARPS;
  // Checkpoints of a chunk, one of the first steps only where the sums over channels
  // of two groups of steps do not fit into one.
  static constexpr int SLOTS = NP > 16 ? SUBS : SUBS - 1;
  // Floats of a warp's sums over channels that a checkpoint does not hold: of more than
  // 32 states, those of the last two of four steps.  (With all of them outside, 16 kB a
  // warp, an SM had one block in the place of two: N=64 T=512 B=16 H=1024 bf16 1494 us.)
  static constexpr int SUMS = NP > 32 ? TILE / 2 * 2 * NP : 0;
  static constexpr int PARTS = LANES < 4 ? LANES : 4;
  static constexpr int WORDS = SUB * WC / K;                   // pairs of a warp's four steps
  static constexpr int MINE = (WORDS + 31) / 32;               // of them, of a lane
  static constexpr int PART = SUB * WC + 8;                    // floats: parts 8 banks apart
  // floats of a warp: checkpoints, parts of three sums
  static constexpr int WARP = SLOTS * SLOT + SUMS + 3 * PARTS * PART;
  // What the outputs need of the tile's inputs is kept for them, x, dt, dy and z as read
  // (read again, N=32 467 us, 450 so; fewer states leave no room, see AHEAD).
  static constexpr bool KEPT = LANES > 4;
  template <typename T>
  static constexpr int shared() {
    return 4 * (WARPS * WARP + 3 * TILE * CC + 2 * TILE * NP + 2 * CC) + (KEPT ? 4 * TILE * CC * (int)sizeof(T) : 0);
  }
};

// Four channels' values of a row, by a word where rows are aligned.
template <bool ALIGNED, typename T>
__device__ __forceinline__ Word<T, 4> load_four(const T *p, int left) {
  Word<T, 4> w;
  if constexpr (ALIGNED) {
    w = *reinterpret_cast<const Word<T, 4> *>(p);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) w.v[j] = j < left ? p[j] : from_f<T>(0.f);
  }
  return w;
}
template <typename T>
__device__ __forceinline__ Four pairs_of(const Word<T, 4> &w) {
  return {f2(to_f(w.v[0]), to_f(w.v[1])), f2(to_f(w.v[2]), to_f(w.v[3]))};
}
__device__ __forceinline__ Four operator*(const Four &x, const Four &y) {
  return {mul2(x.a, y.a), mul2(x.b, y.b)};
}
__device__ __forceinline__ Four operator+(const Four &x, const Four &y) {
  return {add2(x.a, y.a), add2(x.b, y.b)};
}
__device__ __forceinline__ Four sigmoid(const Four &v) {
  return {f2(ssm::sigmoid(lo(v.a)), ssm::sigmoid(hi(v.a))), f2(ssm::sigmoid(lo(v.b)), ssm::sigmoid(hi(v.b)))};
}

// Two channels' values of a row.
template <bool ALIGNED, typename T>
__device__ __forceinline__ Word<T, 2> load_two(const T *p, int left) {
  Word<T, 2> w;
  if (ALIGNED) return *reinterpret_cast<const Word<T, 2> *>(p);
  w.v[0] = p[0];
  w.v[1] = left > 1 ? p[1] : from_f<T>(0.f);
  return w;
}
template <typename T>
__device__ __forceinline__ F2 pair_of(const Word<T, 2> &w) { return f2(to_f(w.v[0]), to_f(w.v[1])); }
template <bool ALIGNED, typename T>
__device__ __forceinline__ void store_two(T *p, int left, F2 v) {
  Word<T, 2> w;
  w.v[0] = from_f<T>(lo(v)), w.v[1] = from_f<T>(hi(v));
  if (ALIGNED) {
    *reinterpret_cast<Word<T, 2> *>(p) = w;
    return;
  }
  p[0] = w.v[0];
  if (left > 1) p[1] = w.v[1];
}
__device__ __forceinline__ F2 sigmoid2(F2 v) { return f2(ssm::sigmoid(lo(v)), ssm::sigmoid(hi(v))); }
__device__ __forceinline__ F2 pair_at(const float *p) { return *reinterpret_cast<const F2 *>(p); }

__device__ __forceinline__ void prefetch(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// WHOLE: the lanes' states and channels are all there.  Blocks of eight warps an SM in all; left to
// itself the compiler takes 168 registers for N=32 and up and spills (N=32 503 us, 445 so).
template <typename T, int LANES, bool ALIGNED, bool WHOLE>
__global__ void __launch_bounds__(Shape<LANES>::NT, 256 / Shape<LANES>::NT) scan_bwd_kernel(const Args a, int *err) {
  typedef Shape<LANES> Sh;
  constexpr int NP = Sh::NP, WC = Sh::WC, NT = Sh::NT, CC = Sh::CC, SLOTS = Sh::SLOTS, PARTS = Sh::PARTS;
  constexpr int PART = Sh::PART, ROW = CC / 4;
  // What the outputs need of the inputs, and the first states a second time, come by
  // asynchronous copies into checkpoints that have been read: a plain read would be
  // waited for, some 1700 cycles, by six warps an SM.  Of 16 states a channel, which
  // leave the upper halves of the checkpoints free.
  constexpr bool AHEAD = LANES == 4 && ALIGNED;
  constexpr bool GUARD = WHOLE && LANES == 16;  // the row's end, at every step (below)
  const ScanBwd &p = a.p;
  const ScanIn &in = p.in;
  extern __shared__ float4 shared4[];
  float *shared = reinterpret_cast<float *>(shared4);
  float *s_delta = shared + Sh::WARPS * Sh::WARP;  // [TILE][CC]
  float *s_u = s_delta + TILE * CC;
  float *s_gy = s_u + TILE * CC;
  float(*s_b)[NP] = reinterpret_cast<float(*)[NP]>(s_gy + TILE * CC);
  float(*s_c)[NP] = s_b + TILE;
  float *s_bias = &s_c[TILE][0], *s_skip = s_bias + CC;  // dt_bias, d
  constexpr bool KEPT = Sh::KEPT;
  T(*s_in)[TILE][CC] = reinterpret_cast<T(*)[TILE][CC]>(s_skip + CC);  // KEPT

  const int group = blockIdx.x % a.groups;
  const int b = (int)(blockIdx.x / a.groups % in.B), seg = (int)(blockIdx.x / a.groups / in.B);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, l = lane % LANES, cl = lane / LANES;
  const int ch0 = group * CC, own = warp * WC + cl * K;  // the thread's channels in the block
  const int n0 = l * S;
  const int64_t table = (int64_t)in.B * in.H * in.N;
  const int64_t at0 = ((int64_t)b * in.H + ch0 + own) * in.N + n0;  // of [B][H][N]
  const int n = row_length(in.lengths, b, in.T, err);
  const int t0 = seg * a.seg.len, t1 = min(t0 + a.seg.len, in.T), end = min(t1, n);
  float *check = shared + warp * Sh::WARP;    // [SLOTS][SLOT]
  float *parts = check + SLOTS * SLOT + Sh::SUMS;  // [3][PARTS][PART]

  auto here = [&](int c) { return ch0 + own + c < in.H ? min(max(in.N - n0, 0), S) : 0; };
  auto load_all = [&](const float *from, F2 (&v)[S]) {
    float x[S], y[S];
    load_states(from, here(0), a.wide_states, x);
    load_states(from + in.N, here(1), a.wide_states, y);
#pragma unroll
    for (int k = 0; k < S; ++k) v[k] = f2(x[k], y[k]);
  };
  auto store_all = [&](float *to, const F2 (&v)[S]) {
#pragma unroll
    for (int c = 0; c < K; ++c) {
      float x[S];
#pragma unroll
      for (int k = 0; k < S; ++k) x[k] = c ? hi(v[k]) : lo(v[k]);
      store_states(to + (int64_t)c * in.N, here(c), a.wide_states, x);
    }
  };

  F2 A2[S], e[S], dA[S];
  load_all(in.a_log + (int64_t)(ch0 + own) * in.N + n0, A2);
#pragma unroll
  for (int k = 0; k < S; ++k) {
    A2[k] = f2(k < here(0) ? rate2(lo(A2[k])) : 0.f, k < here(1) ? rate2(hi(A2[k])) : 0.f);
    e[k] = dA[k] = f2(0.f);
  }
  if (a.enter) load_all(a.enter + (a.seg.n > 1 ? seg * table : 0) + at0, e);

  const T *x = static_cast<const T *>(in.x.p) + b * in.x.sb;
  const T *dt = static_cast<const T *>(in.dt.p) + b * in.dt.sb;
  const T *z = in.z.p ? static_cast<const T *>(in.z.p) + b * in.z.sb : nullptr;
  const T *dy = static_cast<const T *>(p.dy.p) + b * p.dy.sb;
  T *dx = p.dx.p ? static_cast<T *>(p.dx.p) + b * p.dx.sb : nullptr;
  T *ddt = p.ddt.p ? static_cast<T *>(p.ddt.p) + b * p.ddt.sb : nullptr;
  T *dz = p.dz.p ? static_cast<T *>(p.dz.p) + b * p.dz.sb : nullptr;
  Weights<T, NT, TILE, NP> rb(static_cast<const T *>(in.b.p) + b * in.b.sb, in.b.st, in.N, a.wide_bc);
  Weights<T, NT, TILE, NP> rc(static_cast<const T *>(in.c.p) + b * in.c.sb, in.c.st, in.N, a.wide_bc);

  // words of four channels of the tile's inputs (rows NT / ROW apart), and of two of the
  // warp's outputs (a lane's are of the same channels)
  const int in_col = tid % ROW * 4, in_row = tid / ROW, in_left = in.H - ch0 - in_col;
  constexpr int OUT = WC / K;  // words of an output row
  const int out_col = warp * WC + lane % OUT * K, out_row = lane / OUT, out_left = in.H - ch0 - out_col;
  for (int c = tid; c < CC; c += NT) {
    s_bias[c] = in.dt_bias && ch0 + c < in.H ? in.dt_bias[ch0 + c] : 0.f;
    s_skip[c] = in.d && ch0 + c < in.H ? in.d[ch0 + c] : 0.f;
  }
  __syncthreads();
  F2 dd = f2(0.f), ddtb = f2(0.f);  // of the lane's outputs

  // h after step t of the tile, from the state before it
  auto step = [&](int t, F2 (&h)[S]) {
    const F2 d = pair_at(s_delta + t * CC + own), u = pair_at(s_u + t * CC + own);
    float w[S];
    load_row(s_b[t] + n0, w);
#pragma unroll
    for (int q = 0; q < S; ++q) h[q] = fma2(ex2_2(mul2(d, A2[q])), h[q], mul2(u, f2(w[q])));
  };
  auto save = [&](int slot, const F2 (&h)[S]) {
    ulonglong2 *to = reinterpret_cast<ulonglong2 *>(check + slot * SLOT) + lane;
#pragma unroll
    for (int q = 0; q < S / 2; ++q) to[q * 32] = make_ulonglong2(h[2 * q], h[2 * q + 1]);
  };
  auto restore = [&](int slot, F2 (&h)[S]) {
    const ulonglong2 *from = reinterpret_cast<const ulonglong2 *>(check + slot * SLOT) + lane;
#pragma unroll
    for (int q = 0; q < S / 2; ++q) {
      const ulonglong2 v = from[q * 32];
      h[2 * q] = v.x, h[2 * q + 1] = v.y;
    }
  };
  auto copy = [](const F2 (&from)[S], F2 (&to)[S]) {
#pragma unroll
    for (int q = 0; q < S; ++q) to[q] = from[q];
  };
  // where the warp's db and dc of step j of a group of four are: in the place of its
  // checkpoint; of the first group, where it has none, behind those of the second
  auto sums_of = [&](float *from, int sub, int j) {
    const int slot = sub + SLOTS - SUBS;
    if (Sh::SUMS && j >= SUB / 2) return from + SLOTS * SLOT + (sub * SUB / 2 + j - SUB / 2) * 2 * NP;
    return from + (slot < 0 ? SUB * 2 * NP : slot * SLOT) + j * 2 * NP;
  };

  const int tiles = t0 < end ? ceil_div(end - t0, TILE) : 0;
  for (int k = tiles - 1; k >= 0; --k) {
    const int base = t0 + k * TILE, steps = min(TILE, end - base), subs = ceil_div(steps, SUB);
    rb.read(base, end);
    rc.read(base, end);
    const float *first = p.states + (base / TILE) * table + at0;  // the states before the tile
    F2 h[S];
    load_all(first, h);
    F2 probe = f2(0.f);  // NaN where an input of the states or of their gradients is not finite
    constexpr int PASS = NT / ROW, MOST = 4;
    constexpr int BATCH = TILE / PASS < MOST ? TILE / PASS : MOST;  // words in flight, of rows PASS apart
#pragma unroll 1
    for (int r0 = in_row; r0 < TILE; r0 += BATCH * PASS) {
      Word<T, 4> wx[BATCH], wt[BATCH], wy[BATCH], wz[BATCH];
#pragma unroll
      for (int q = 0; q < BATCH; ++q) {
        const int64_t t = base + r0 + q * PASS;
        if (r0 + q * PASS >= steps || in_left <= 0) break;
        wx[q] = load_four<ALIGNED>(x + t * in.x.st + ch0 + in_col, in_left);
        wt[q] = load_four<ALIGNED>(dt + t * in.dt.st + ch0 + in_col, in_left);
        wy[q] = load_four<ALIGNED>(dy + t * p.dy.st + ch0 + in_col, in_left);
        if (z) wz[q] = load_four<ALIGNED>(z + t * in.z.st + ch0 + in_col, in_left);
      }
#pragma unroll
      for (int q = 0; q < BATCH; ++q) {
        const int r = r0 + q * PASS;
        Four v{}, u{}, g{};  // 0 past the row's end
        if (r < steps && in_left > 0) {
          v = pairs_of(wt[q]) + four(s_bias + in_col);
          v = {softplus(v.a), softplus(v.b)};
          u = v * pairs_of(wx[q]);
          if constexpr (KEPT) {
            auto keep = [&](int i, const Word<T, 4> &w) { *reinterpret_cast<Word<T, 4> *>(&s_in[i][r][in_col]) = w; };
            keep(0, wx[q]), keep(1, wt[q]);
            if (z) keep(2, wy[q]), keep(3, wz[q]);
          }
          g = pairs_of(wy[q]);
          if (z) {
            const Four zs = pairs_of(wz[q]);
            g = g * zs * sigmoid(zs);
          }
        }
        put_four(s_delta + r * CC + in_col, v);
        put_four(s_u + r * CC + in_col, u);
        put_four(s_gy + r * CC + in_col, g);
        if (!WHOLE) probe = fma2(u.b, f2(0.f), fma2(u.a, f2(0.f), probe));
        if (!WHOLE) probe = fma2(g.b, f2(0.f), fma2(g.a, f2(0.f), probe));
      }
    }
    const float probe_bc = rb.put(s_b) + rc.put(s_c);
    // States and channels that do not exist have weights or inputs of 0, and stay 0 (their
    // gradients too) but for infinite inputs of those that do.
    int met = 0;
    if (WHOLE) __syncthreads();
    else met = __syncthreads_or(isnan(lo(probe)) || isnan(hi(probe)) || isnan(probe_bc));
    if (k > 0) {  // the tile before, into the second-level cache
      constexpr int LINE = 128 / sizeof(T);  // values
      for (int i = tid; i < TILE * ((CC + LINE - 1) / LINE); i += NT) {
        const int64_t t = base - TILE + i % TILE;
        const int c = ch0 + i / TILE * LINE;
        if (c >= in.H) break;
        prefetch(x + t * in.x.st + c);
        prefetch(dt + t * in.dt.st + c);
        prefetch(dy + t * p.dy.st + c);
        if (z) prefetch(z + t * in.z.st + c);
      }
      const float *before = p.states + (base / TILE - 1) * table + ((int64_t)b * in.H + ch0) * in.N;
      for (int i = tid * 32; i < min(CC, in.H - ch0) * in.N; i += NT * 32) prefetch(before + i);
    }
    if (SLOTS == SUBS) save(0, h);
    for (int t = 0; t < (subs - 1) * SUB; ++t) {
      step(t, h);
      if (t % SUB == SUB - 1) save(t / SUB + SLOTS - (SUBS - 1), h);
    }
    // Four steps backwards.  CAREFUL: what does not exist must not get into the sums, where an
    // infinity would make it NaN.
    auto back_over = [&](int sub, auto care) {
      constexpr bool CAREFUL = decltype(care)::value;
      auto keep_there = [&](int q, F2 &v) { v = f2(q < here(0) ? lo(v) : 0.f, q < here(1) ? hi(v) : 0.f); };
      const int slot = sub + SLOTS - SUBS;
      // AHEAD: the upper half of a slot, 16 bytes a lane; the first states are in those of
      // slots 2 and 3
      auto upper = [&](int of) { return check + of * SLOT + SLOT / 2; };
      auto first_at = [&](int c) { return upper(2 + c) + lane * 4; };
      if (AHEAD && a.wide_states && sub == 1) {
#pragma unroll
        for (int c = 0; c < K; ++c)
          if (here(c) == S) copy_async<16>(first_at(c), first + (int64_t)c * in.N);
          else *reinterpret_cast<float4 *>(first_at(c)) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      Word<T, 2> wx, wt, wy, wz;
      auto read = [&](int r) {  // the words of the outputs at row r of the tile
        const int64_t t = base + r;
        if (r >= steps || out_left <= 0 || (Sh::WORDS < 32 && out_row >= SUB)) return;
        if constexpr (KEPT) {
          auto kept = [&](int i) { return *reinterpret_cast<const Word<T, 2> *>(&s_in[i][r][out_col]); };
          wx = kept(0), wt = kept(1);
          if (z) wy = kept(2), wz = kept(3);
          return;
        }
        wx = load_two<ALIGNED>(x + t * in.x.st + ch0 + out_col, out_left);
        wt = load_two<ALIGNED>(dt + t * in.dt.st + ch0 + out_col, out_left);
        if (z) {
          wy = load_two<ALIGNED>(dy + t * p.dy.st + ch0 + out_col, out_left);
          wz = load_two<ALIGNED>(z + t * in.z.st + ch0 + out_col, out_left);
        }
      };
      // AHEAD: where the i-th of them waits, of fp32 the third and fourth in the next slot
      // (the first steps, whose sums are in the upper half of slot 0, take slot 1)
      const bool two_slots = sizeof(T) == 4, rest = !two_slots || slot + 1 < SLOTS;
      auto word_at = [&](int i) {
        const int of = slot < 0 ? 1 : slot;
        float *to = two_slots ? upper(of + i / 2) + i % 2 * 64 + lane * 2 : upper(of) + i * 32 + lane;
        return reinterpret_cast<Word<T, 2> *>(to);
      };
      auto read_ahead = [&]() {
        const int r = sub * SUB + out_row;
        const int64_t t = base + r;
        if (r >= steps || out_left <= 0) return;
        copy_async<sizeof(wx)>(word_at(0), x + t * in.x.st + ch0 + out_col);
        copy_async<sizeof(wx)>(word_at(1), dt + t * in.dt.st + ch0 + out_col);
        if (z && rest) {
          copy_async<sizeof(wx)>(word_at(2), dy + t * p.dy.st + ch0 + out_col);
          copy_async<sizeof(wx)>(word_at(3), z + t * in.z.st + ch0 + out_col);
        }
      };
      auto start = [&](F2 (&h)[S]) {  // the states before the four steps
        if (slot >= 0) {
          restore(slot, h);
        } else if (AHEAD && a.wide_states && subs > 1) {
          float v[K][S];
          load_row(first_at(0), v[0]);
          load_row(first_at(1), v[1]);
#pragma unroll
          for (int q = 0; q < S; ++q) h[q] = f2(v[0][q], v[1][q]);
        } else {
          load_all(first, h);
        }
      };
      constexpr int OUTS = LANES > 4 ? LANES / 4 : 1;  // sums over channels of a lane, at a step
      float bc[SUB][OUTS];
      F2 before[SUB][S];
      auto back = [&](int j) {  // step j backwards; h after it
        const int t = sub * SUB + j;
        const F2 d = pair_at(s_delta + t * CC + own), u = pair_at(s_u + t * CC + own);
        const F2 g = pair_at(s_gy + t * CC + own);
        float w[S], v[S], db[S], dc[S];
        load_row(s_b[t] + n0, w);
        load_row(s_c[t] + n0, v);
        F2 so, sd, sl;
#pragma unroll
        for (int q = 0; q < S; ++q) {
          e[q] = fma2(g, f2(v[q]), e[q]);
          if (CAREFUL && !WHOLE) keep_there(q, e[q]), keep_there(q, h[q]), keep_there(q, before[j][q]);
          so = q ? fma2(h[q], f2(v[q]), so) : mul2(h[q], f2(v[q]));
          sd = q ? fma2(e[q], f2(w[q]), sd) : mul2(e[q], f2(w[q]));
          db[q] = fmaf(hi(e[q]), hi(u), lo(e[q]) * lo(u));
          dc[q] = fmaf(hi(h[q]), hi(g), lo(h[q]) * lo(g));
          e[q] = mul2(e[q], ex2_2(mul2(d, A2[q])));
          if (CAREFUL && !WHOLE) keep_there(q, e[q]);
          const F2 r = mul2(e[q], before[j][q]);
          sl = q ? fma2(r, A2[q], sl) : mul2(r, A2[q]);
          if (!(CAREFUL || GUARD) || t < steps) dA[q] = fma2(r, d, dA[q]);
          h[q] = before[j][q];
        }
        // sums over the states, down to PARTS lanes
#pragma unroll
        for (int o = LANES / 2; o >= PARTS; o /= 2) {
          so = add2(so, __shfl_xor_sync(0xffffffffu, so, o));
          sd = add2(sd, __shfl_xor_sync(0xffffffffu, sd, o));
          sl = add2(sl, __shfl_xor_sync(0xffffffffu, sl, o));
        }
        float *to = parts + l % PARTS * PART + j * WC + cl * K;
        if (LANES <= 4 || l < 4) {
          *reinterpret_cast<F2 *>(to) = so;
          *reinterpret_cast<F2 *>(to + PARTS * PART) = sd;
          *reinterpret_cast<F2 *>(to + 2 * PARTS * PART) = sl;
        }
        // sums over the warp's channels: its lanes of the same states halve with one another
        // what they hold, by b and c first
        float v8[2 * S];
#pragma unroll
        for (int q = 0; q < S; ++q) v8[q] = db[q], v8[S + q] = dc[q];
        int count = 2 * S;
#pragma unroll
        for (int o = 16; o >= LANES; o /= 2) {
          if (count == 1) {
            v8[0] += __shfl_xor_sync(0xffffffffu, v8[0], o);
            continue;
          }
          count /= 2;
          const bool upper = lane & o;
#pragma unroll
          for (int q = 0; q < S; ++q)
            if (q < count) {
              const float mine = upper ? v8[q + count] : v8[q], other = upper ? v8[q] : v8[q + count];
              v8[q] = mine + __shfl_xor_sync(0xffffffffu, other, o);
            }
        }
#pragma unroll
        for (int m = 0; m < OUTS; ++m) bc[j][m] = v8[m];
      };
      if (AHEAD && sub == 0) fetched();
      if (sub < subs - 1) start(h);  // the last ones are at hand
      if (AHEAD) {
        __syncwarp();  // all lanes have what was there
        read_ahead();
      }
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        copy(h, before[j]);
        step(sub * SUB + j, h);
      }
      // (rolled up where registers are full, so that the other body is not the one that spills:
      // N=33 T=512 B=16 H=1024 fp32 833 us, 785 so)
      if constexpr (CAREFUL && LANES == 16) {
#pragma unroll 1
        for (int j = SUB - 1; j >= 0; --j) back(j);
      } else {
#pragma unroll
        for (int j = SUB - 1; j >= 0; --j) back(j);
      }
      if (a.part_bc) {
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
          float *to = sums_of(check, sub, j);
#pragma unroll
          for (int m = 0; m < OUTS; ++m) {
            const int i = lane / (LANES < 4 ? 4 : LANES) * OUTS + m;  // of LANES 2, every other pair's
            if (LANES >= 4 || lane % 4 < LANES) to[(i >> 2) * NP + n0 + (i & 3)] = bc[j][m];
          }
        }
      }
      __syncwarp();
      // the outputs: dx = delta sd + gy d, ddt = (sl A + sd x) sigmoid(dt), dz = dy (so + d x) silu'(z)
#pragma unroll
      for (int i = 0; i < Sh::MINE; ++i) {
        const int j = out_row + i * (32 / OUT), r = sub * SUB + j;
        const int64_t t = base + r;
        if (AHEAD) {
          fetched();
          wx = *word_at(0), wt = *word_at(1);
          if (z && rest) wy = *word_at(2), wz = *word_at(3);
        }
        if (r >= steps || out_left <= 0 || (Sh::WORDS < 32 && j >= SUB)) continue;
        if (!AHEAD) {
          read(r);
        } else if (z && !rest) {
          wy = load_two<ALIGNED>(dy + t * p.dy.st + ch0 + out_col, out_left);
          wz = load_two<ALIGNED>(z + t * in.z.st + ch0 + out_col, out_left);
        }
        const float *from = parts + j * WC + out_col - warp * WC;
        F2 so = pair_at(from), sd = pair_at(from + PARTS * PART), sl = pair_at(from + 2 * PARTS * PART);
#pragma unroll
        for (int m = 1; m < PARTS; ++m) {
          so = add2(so, pair_at(from + m * PART));
          sd = add2(sd, pair_at(from + (PARTS + m) * PART));
          sl = add2(sl, pair_at(from + (2 * PARTS + m) * PART));
        }
        const F2 delta = pair_at(s_delta + r * CC + out_col), gy = pair_at(s_gy + r * CC + out_col);
        const F2 skip = pair_at(s_skip + out_col), xv = pair_of(wx);
        if (dx) {
          F2 v = mul2(sd, delta);
          if (in.d) v = fma2(gy, skip, v);
          store_two<ALIGNED>(dx + t * p.dx.st + ch0 + out_col, out_left, v);
        }
        // A2 is in units of log2(e)
        const F2 gdt = mul2(fma2(sl, f2(1.f / LOG2E), mul2(sd, xv)),
                            sigmoid2(add2(pair_of(wt), pair_at(s_bias + out_col))));
        if (ddt) store_two<ALIGNED>(ddt + t * p.ddt.st + ch0 + out_col, out_left, gdt);
        if (dz) {
          const F2 zs = pair_of(wz), sg = sigmoid2(zs);
          if (in.d) so = fma2(skip, xv, so);
          const F2 slope = mul2(sg, fma2(zs, fma2(sg, f2(-1.f), f2(1.f)), f2(1.f)));
          store_two<ALIGNED>(dz + t * p.dz.st + ch0 + out_col, out_left, mul2(mul2(pair_of(wy), so), slope));
        }
        ddtb = add2(ddtb, gdt);
        dd = fma2(gy, xv, dd);
      }
      __syncwarp();  // before the next steps' parts
    };
    // With care: all where an infinity was met, else the last four steps, where the row ends
    // in the midst of them.  For those, of 64 states a select at every step is faster than a
    // second body (T=512 B=16 H=1024 bf16 972 us, 997), of fewer the body is (N=16 T=300 B=64
    // H=2048 938 us, 981).  (The vote has the flag in a register of its own: without
    // it N=16 T=512 B=16 H=1001 bf16 317 us, 309 so.)
    const bool careful = !WHOLE && __any_sync(0xffffffffu, met);
    int sub = subs - 1;
#pragma unroll 1
    for (const int last = careful ? 0 : GUARD ? subs : steps / SUB; sub >= last; --sub) back_over(sub, std::true_type());
#pragma unroll 1
    for (; sub >= 0; --sub) back_over(sub, std::false_type());
    __syncthreads();
    if (a.part_bc) {
      // four neighbouring sums of a step at a time: [steps][2][N]
      float *to = a.part_bc + (((int64_t)group * in.T + base) * in.B + b) * 2 * in.N;
      const int64_t row = (int64_t)in.B * 2 * in.N;
      constexpr int QUADS = 2 * NP / 4;
      for (int i = tid; i < steps * QUADS; i += NT) {
        const int t = i / QUADS, m = i % QUADS * 4, q = m % NP;
        const float *from = sums_of(shared, t / SUB, t % SUB) + m;
        Four v = four(from);
#pragma unroll
        for (int w = 1; w < Sh::WARPS; ++w) v = v + four(from + w * Sh::WARP);
        float *at = to + t * row + (m / NP) * in.N + q;
        const float out[4] = {lo(v.a), hi(v.a), lo(v.b), hi(v.b)};
        if (in.N % 4 == 0) {
          if (q < in.N) *reinterpret_cast<float4 *>(at) = make_float4(out[0], out[1], out[2], out[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (q + j < in.N) at[j] = out[j];
        }
      }
      __syncthreads();
    }
  }
  // past the row's end
  const int past = max(t0, end);
  for (int64_t i = tid; i < (int64_t)(t1 - past) * CC; i += NT) {
    const int64_t t = past + i / CC;
    const int c = ch0 + (int)(i % CC);
    if (c >= in.H) continue;
    if (dx) dx[t * p.dx.st + c] = from_f<T>(0.f);
    if (ddt) ddt[t * p.ddt.st + c] = from_f<T>(0.f);
    if (dz) dz[t * p.dz.st + c] = from_f<T>(0.f);
  }
  if (seg == 0 && p.dh0) store_all(p.dh0 + at0, e);
  if (!a.part) return;
  float *to = a.part + ((int64_t)seg * in.B + b) * in.H * (in.N + 2);
#pragma unroll
  for (int q = 0; q < S; ++q) {
    const F2 v = mul2(dA[q], mul2(A2[q], f2(1.f / LOG2E)));
    float *at = to + (int64_t)(ch0 + own) * in.N + n0 + q;
    if (q < here(0)) at[0] = lo(v);
    if (q < here(1)) at[in.N] = hi(v);
  }
  // lanes with the same channels of the outputs
#pragma unroll
  for (int o = OUT; o < 32; o *= 2) {
    dd = add2(dd, __shfl_xor_sync(0xffffffffu, dd, o));
    ddtb = add2(ddtb, __shfl_xor_sync(0xffffffffu, ddtb, o));
  }
  if (out_row == 0) {
    to += (int64_t)in.H * in.N + ch0 + out_col;
    if (out_left > 0) to[0] = lo(dd), to[in.H] = lo(ddtb);
    if (out_left > 1) to[1] = hi(dd), to[in.H + 1] = hi(ddtb);
  }
}

// db and dc from the blocks' sums, [groups][T][B][2][N]: a thread a value.
template <typename T>
__global__ void __launch_bounds__(256) sum_bc_kernel(const float *part, int groups, int T_, int B, int N,
                                                     const int32_t *lengths, SeqOut db, SeqOut dc) {
  wait_for_previous();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)T_ * B * 2 * N;
  if (i >= all) return;
  const int m = (int)(i % (2 * N)), b = (int)(i / (2 * N) % B);
  const int64_t t = i / (2 * N) / B;
  const SeqOut &to = m < N ? db : dc;
  if (!to.p) return;
  float s = 0.f;
  if (!lengths || t < lengths[b])
    for (int g = 0; g < groups; ++g) s += part[g * all + i];
  static_cast<T *>(to.p)[t * to.st + b * to.sb + m % N] = from_f<T>(s);
}

template <typename T, int LANES, bool ALIGNED, bool WHOLE>
cudaError_t run(Args a, int *err, cudaStream_t s, int *launches) {
  typedef Shape<LANES> Sh;
  auto fn = scan_bwd_kernel<T, LANES, ALIGNED, WHOLE>;
  static PerDevice<cudaError_t> ready;
  const cudaError_t set = ready.here(
      [&] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::template shared<T>()); });
  if (set != cudaSuccess) return set;
  ++*launches;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)a.groups * a.p.in.B * a.seg.n));
  cfg.blockDim = dim3(Sh::NT);
  cfg.dynamicSmemBytes = Sh::template shared<T>();
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, fn, a, err);
}

// Of four states or fewer a channel, half of the lanes' are idle: a kernel for those alone,
// with one warp a block and six an SM, was slower (N=4 bf16 T=512 B=16 H=1024 315 us, 248).
template <typename F>
cudaError_t by_lanes(int N, F f) {
  if (N <= 8) return f(std::integral_constant<int, 2>());
  if (N <= 16) return f(std::integral_constant<int, 4>());
  if (N <= 32) return f(std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 16>());
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanBwd &p, DevMem &ws, int *err, int nsm, bool vec,
                            cudaStream_t s, int *launches) {
  const ScanIn &in = p.in;
  const int64_t table = (int64_t)in.B * in.H * in.N, rows = (int64_t)in.B * in.H;
  Args a{};
  a.p = p;
  by_lanes(in.N, [&](auto lanes) {
    a.groups = ceil_div(in.H, Shape<decltype(lanes)::value>::CC);
    return cudaSuccess;
  });
  a.seg = segments_of(in.T, (int64_t)a.groups * in.B, nsm, 4);
  const bool bc = p.db.p || p.dc.p, sums = p.da_log || p.dd || p.ddt_bias;
  const int64_t n_bc = bc ? (int64_t)a.groups * in.T * in.B * 2 * in.N : 0;
  const int64_t n_part = sums ? (int64_t)a.seg.n * in.B * in.H * (in.N + 2) : 0;
  const int64_t n_seg = a.seg.n > 1 ? a.seg.n * (table + rows) : 0;
  float *mem = nullptr;
  auto up = [](int64_t v) { return (v + 31) / 32 * 32; };
  if (n_bc + n_part + n_seg) {
    const cudaError_t e = ws.get((size_t)(up(n_bc) + up(n_part) + up(n_seg)) * 4, &mem);
    if (e != cudaSuccess) return e;
  }
  if (bc) a.part_bc = mem;
  if (sums) a.part = mem + up(n_bc);
  a.enter = p.dh_n;
  if (n_seg) {
    Meeting m{a.seg, mem + up(n_bc) + up(n_part), nullptr};
    m.sums = m.end + a.seg.n * table;
    const cudaError_t e = launch_local(in, true, p.dy, p.dh_n, m, err, vec, s, launches);
    if (e != cudaSuccess) return e;
    a.enter = m.end;
  }
  a.wide_states = vec && in.N % S == 0 && aligned(in.a_log, 4, 4, 4) && aligned(p.states, 4, 4, 4) &&
                  (!a.enter || aligned(a.enter, 4, 4, 4)) && (!p.dh0 || aligned(p.dh0, 4, 4, 4));
  const int size = in.dtype == RCU_BF16 ? 2 : 4;
  a.wide_bc = vec && in.N % 4 == 0 && aligned(in.b, size, 4) && aligned(in.c, size, 4);
  auto fits = [&](const auto &t) { return !t.p || aligned(t, size, 4); };
  const bool wide = vec && in.H % 4 == 0 && fits(in.x) && fits(in.dt) && fits(in.z) && fits(p.dy) &&
                    fits(p.dx) && fits(p.ddt) && fits(p.dz);
  cudaError_t e = by_lanes(in.N, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const bool whole = in.N == Shape<L>::NP && in.H % Shape<L>::CC == 0;
    auto of_type = [&](auto value) {
      typedef decltype(value) V;
      if (whole) return wide ? run<V, L, true, true>(a, err, s, launches) : run<V, L, false, true>(a, err, s, launches);
      return wide ? run<V, L, true, false>(a, err, s, launches) : run<V, L, false, false>(a, err, s, launches);
    };
    return in.dtype == RCU_BF16 ? of_type(bf16()) : of_type(float());
  });
  if (e != cudaSuccess) return e;
  if (sums) {
    const ColumnSum c{a.part, a.seg.n * (int64_t)in.B, (int64_t)in.H * (in.N + 2), (int64_t)in.H * in.N,
                      in.H, p.da_log, p.dd, p.ddt_bias};
    e = launch_column_sum(c, s, launches);
    if (e != cudaSuccess) return e;
  }
  if (bc) {
    const dim3 grid((unsigned)(((int64_t)in.T * in.B * 2 * in.N + 255) / 256));
    ++*launches;
    auto fn = in.dtype == RCU_BF16 ? sum_bc_kernel<bf16> : sum_bc_kernel<float>;
    e = launch_after(fn, grid, 256, s, (const float *)a.part_bc, a.groups, in.T, in.B, in.N, in.lengths,
                     p.db, p.dc);
  }
  return e;
}

}  // namespace rcu
