// Gated linear recurrence, backward: the gradients of x, r, i, lambda and h0.
//
// The gradient that reaches a state follows the same recurrence backwards in
// time, e_t = dy_t + a_{t+1} e_{t+1}, so the tiles run from the last to the
// first and each warp publishes two maps of its steps: h -> P h + E forwards
// and c -> P c + R backwards (c = a e; the factor is the same).  The state
// that enters a tile comes from the forward's states, so only the backward
// carry crosses tiles.  Per element: four values read and three written, once;
// em1, b and both sigmoids stay in registers between the two runs.
//
// Bound by the issue of instructions, 65 to 70 an element (bf16) at 2.3 a cycle,
// which is what 16 warps an SM reach at 128 registers a thread: DRAM is half busy.
// Measured: bf16 T=512 B=256 H=1024 344 us, T=8192 B=4 H=2048 236 us (944 MB,
// 4.0 TB/s); fp32 T=500 B=64 H=512 with mixed lengths 71 us (348 MB, 4.9 TB/s).
// From 8 bits it issues nearly 80, the codes' scaling among them: T=1000 B=32
// H=1024 114 us for 364 MB.
#include "linrec_bwd.cuh"

namespace rcu {
namespace {

using namespace linrec;

// Eight warps of 8 steps: the tile is what one kept state covers, and 16 steps a
// lane would need more than the 255 registers a thread can have.  Two blocks an SM
// (128 registers); bf16 rows that TMA cannot address take more, and beside a cluster's
// exchange one block is faster there (T=15731 B=1 H=2133: 258 us, 280 with two; with
// shares two are: T=521 B=86 H=748 178 us, 280 with one).
constexpr int NW = 8, NT = 32 * NW, S = CHUNK / NW, STEPS = CHUNK, STAGES = 2, PER_SM = 2;
constexpr int MAXCS = 8;  // blocks of a cluster
constexpr int BATCH = 4;  // pairs whose gates are computed together

template <typename V>
struct Smem {
  typename Slot<V>::type part[2][NW][32];     // the warps' P and R, by parity of the tile
  V fwd[2][NW][32];                           // and their E
  typename Slot<V>::type peer[2][MAXCS][32];  // the blocks' P and R, by parity of the round
  V sum[NW][32];  // of dlambda, over the row or, with shares, all the block's rows
  uint64_t full[STAGES];
  uint64_t met[2];  // every block's map of a round is here, by parity of the round
  int abort;
  Next next;
  struct {
    V k2, nk;  // the channel's rate, as rate() has it, and -K
    Limits lim;
  } chan[32];
};

// Bytes of a tile of a saved input (IT) and of all four.
template <typename IT, typename T, bool TMA>
constexpr int in_bytes() {
  return STEPS * (TMA ? Shape<T>::CW * (int)sizeof(IT) : Loose<IT, Shape<T>::CPT>::PITCH);
}
template <typename IT, typename T, bool TMA>
constexpr int tensor_bytes() { return 3 * in_bytes<IT, T, TMA>() + in_bytes<T, T, TMA>(); }
// and with the states that enter the tile
template <typename IT, typename T, bool TMA>
constexpr int stage_bytes() { return tensor_bytes<IT, T, TMA>() + Shape<T>::CW * 4; }

// A lane's values of one step (CPT channels) in a tile that TMA brought
template <typename IT, int CPT>
__device__ __forceinline__ uint32_t tile_raw(const uint8_t *row, int lane) {
  constexpr int N = CPT * (int)sizeof(IT);
  row += lane * N;
  if (N == 4) return *reinterpret_cast<const uint32_t *>(row);
  if (N == 2) return *reinterpret_cast<const unsigned short *>(row);
  return *row;
}

// MAPS: only the backward map (P, R) of each segment but the first, from r and dy
// alone, into `mem`, which the launch after it starts its segments from.  (With
// SHARES, mem has their carries.)
template <typename IT, typename T, bool TMA, Mode M>
__global__ void __launch_bounds__(NT, TMA || sizeof(T) == 4 || M == SHARES ? PER_SM : 1)
    linrec_bwd_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mr,
                      const __grid_constant__ CUtensorMap mi, const __grid_constant__ CUtensorMap mdy,
                      const LinrecBwd p, const Cut cut, void *mem, float *__restrict__ partial,
                      const bool words, const bool bulk_states, int *err) {
  constexpr bool MAP = M == MAPS;
  constexpr int CPT = Shape<T>::CPT, CW = Shape<T>::CW;
  constexpr int IN = in_bytes<IT, T, TMA>(), TENSORS = tensor_bytes<IT, T, TMA>();
  constexpr int STAGE = stage_bytes<IT, T, TMA>();
  constexpr int IN_ROW = IN / STEPS, DY_ROW = in_bytes<T, T, TMA>() / STEPS;
  constexpr bool Q8 = sizeof(IT) == 1;
  // fp32 copies its next tile after a tile's stores, not before them: T=512 B=128 H=1024
  // 300 us, 325 the other way round (bf16 368 and 353)
  constexpr bool LATE = TMA && !MAP && sizeof(IT) == 4;
  typedef typename Lane<T>::V V;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *ring = smem;
  Smem<V> &sh = *reinterpret_cast<Smem<V> *>(smem + STAGES * STAGE);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cs = M == UNITS ? (int)tc::cluster_nctarank() : 1;
  const int rank = M == UNITS ? (int)tc::cluster_ctarank() : 0;
  const int stride = M == SHARES ? 1 : gridDim.x / cs, u0 = M == SHARES ? 0 : blockIdx.x / cs;
  const int units = count_units<M>(cut, p.B);

  // the inputs' rows lie alike
  const bool same = !TMA && p.x.st == p.r.st && p.x.st == p.i.st && p.x.sb == p.r.sb &&
                    p.x.sb == p.i.sb && alike(p.x.p, p.r.p) && alike(p.x.p, p.i.p);
  // Copies of the live tiles of this block, the last steps first: by TMA (thread
  // 0, the whole tile) or by each warp its own rows.
  // With TMA it is one thread that copies: what it keeps for that is in shared memory,
  // as its registers would be every thread's (bf16 T=512 B=256 H=1024: 345 us, 353 with
  // registers).  Clusters, with more to do between two tiles, lose by it (238, 249) but
  // for pairs from 8 bits (T=8192 B=4 H=2048 291, 298).
  constexpr bool ONE = TMA && (M != UNITS || (Q8 && CPT == 2));
  Next own;
  Next &next = ONE ? sh.next : own;
  if (!ONE || threadIdx.x == 0) {
    next.u = u0 - stride, next.issued = 0;
    next.tile = -1, next.v.first = 0;
  }
  auto issue = [&] {
    Unit v = next.v;
    int tile = next.tile;
    while (tile < v.first) {
      if (next.u >= units - stride) {
        if (!TMA) copy_commit();
        return;
      }
      v = next.v = unit_of<M, true>(cut, p.B, next.u += stride, CW);
      next.len = row_length(p.lengths, v.b, p.T, err);
      tile = v.last - 1 - rank;
      const int dead = tile - (ceil_div(next.len, STEPS) - 1);  // tiles past the row's end
      if (dead > 0) tile -= ceil_div(dead, cs) * cs;
      next.tile = tile;
    }
    next.tile = tile - cs;
    const int issued = next.issued++;
    uint8_t *dst = ring + issued % STAGES * STAGE;
    if (TMA) {
      uint64_t *bar = &sh.full[issued % STAGES];
      const bool kept = bulk_states && !MAP && RCU_DCHECK(tile >= 0 && tile * STEPS < p.T, err);
      const int states = kept ? min(CW, p.H - v.c0) * 4 : 0;
      tc::mbar_arrive_expect_tx(bar, (MAP ? TENSORS - 2 * IN : TENSORS) + states);
      if (states)
        tc::bulk_load(dst + TENSORS, p.states + ((int64_t)tile * p.B + v.b) * p.H + v.c0, states,
                      bar);
      tma_load_3d(dst + IN, &mr, bar, v.c0, v.b, tile * STEPS);
      if (!MAP) {
        tma_load_3d(dst, &mx, bar, v.c0, v.b, tile * STEPS);
        tma_load_3d(dst + 2 * IN, &mi, bar, v.c0, v.b, tile * STEPS);
      }
      tma_load_3d(dst + 3 * IN, &mdy, bar, v.c0, v.b, tile * STEPS);
    } else {
      const int tw = tile * STEPS + warp * S;
      const int rows = RCU_DCHECK(tile >= 0 && v.b < p.B && v.c0 < p.H && next.len <= p.T, err)
                           ? min(next.len - tw, S)
                           : 0;
      const int width = min(CW, p.H - v.c0);
      auto pos = [&](const SeqIn &in, int size) {
        return ((int64_t)tw * in.st + (int64_t)v.b * in.sb + v.c0) * size;
      };
      uint8_t *to = dst + warp * S * IN_ROW;
      if (!MAP && same) {
        const void *const base[3] = {p.x.p, p.r.p, p.i.p};
        copy_rows<IT, CPT>(to, IN, base, pos(p.x, sizeof(IT)), p.x.st * (int64_t)sizeof(IT), rows,
                           width * (int)sizeof(IT));
      } else {
#pragma unroll 1
        for (int k = MAP ? 1 : 0; k < (MAP ? 2 : 3); ++k) {
          const SeqIn &in = (&p.x)[k];
          const void *const base[1] = {in.p};
          copy_rows<IT, CPT>(to + k * IN, 0, base, pos(in, sizeof(IT)),
                             in.st * (int64_t)sizeof(IT), rows, width * (int)sizeof(IT));
        }
      }
      const void *const base[1] = {p.dy.p};
      copy_rows<T, CPT>(dst + 3 * IN + warp * S * DY_ROW, 0, base, pos(p.dy, sizeof(T)),
                        p.dy.st * (int64_t)sizeof(T), rows, width * (int)sizeof(T));
    }
    if (!TMA) copy_commit();
  };
  if (threadIdx.x == 0) {
    for (int st = 0; st < STAGES; ++st) tc::mbar_init(&sh.full[st], 1);
    for (int q = 0; q < 2; ++q) tc::mbar_init(&sh.met[q], 1);
    sh.abort = 0;
    tc::fence_mbar_init();
  }
  if (!TMA || threadIdx.x == 0) {
#pragma unroll 1
    for (int st = 0; st < STAGES; ++st) issue();
  }
  __syncthreads();
  if (cs > 1) tc::cluster_sync();  // every block of the cluster runs before its memory is written

  set(sh.sum[warp][lane], 0.f);
  int used = 0, parity = 0, round = 0, held = -1;  // held: the channels k2 and so on are of
  bool small = false;
  V k2;
  Limits lim;
  for (int u = u0; u < units; u += stride) {
    const Unit v = unit_of<M, true>(cut, p.B, u, CW);
    const int len = row_length(p.lengths, v.b, p.T, err);
    const int ch = v.c0 + lane * CPT, live = min(max(p.H - ch, 0), CPT);
    const int64_t row = (int64_t)v.b * p.H + ch;
    V nc, sum, zero, minus;
    set(zero, 0.f);
    set(minus, -1.f);
    if (v.c0 != held) {
      held = v.c0;
      rate(p.lambda + ch, p.c, live, k2);
      lim = limits(k2);
      small = __all_sync(0xffffffffu, small_rate(k2));
    }
    const bool whole = v.c0 + CW <= p.H && words;
    set(nc, 0.f);
    if (p.dh_n) load_v(p.dh_n + row, live, nc);
    nc = neg_v(nc);  // the carry, negated: -dL/dh after the steps so far
    if (!MAP && v.seg < cut.nseg - 1)
      nc = apply(chain_segments<V, NW>(mem, cut, p.B, v, CW, cut.nseg - 1, v.seg, -1, sh.part[0],
                                        err),
                 nc);
    if (M == SHARES && v.last < cut.tiles)
      nc = take_carry<V>(mem, blockIdx.x - cut.groups, err, &sh.abort);
    Aff<V> all_map = identity<V>();
    sum = zero;
    // 8 bits: lane 8 k + s has the exponent of tensor k at the warp's step s, read a
    // tile ahead
    int ex = FREE_EXP;
    auto read_exponent = [&](int tile) {
      const int t = tile * STEPS + warp * S + lane % S, k = lane / S;
      ex = FREE_EXP;
      if (k < 3 && tile >= v.first && t < len)
        ex = (int)__ldg((k == 0 ? p.x.e : k == 1 ? p.r.e : p.i.e) +
                        ((int64_t)t * p.et + v.b * p.eb) * ceil_div(p.H, BLOCK8) + v.c0 / BLOCK8);
    };
    if (Q8) read_exponent(v.last - 1 - rank);
    for (int base = v.last - 1; base >= v.first; base -= cs) {
      const int tile = base - rank, tw = tile * STEPS + warp * S;
      const bool on = tile >= v.first && tile * STEPS < len;  // the same for the whole block
      V em1[S], nb[S], ns[S], ng[S], dy[S], h = zero, fe = zero;
      Aff<V> mine = identity<V>();
      if (on) {
        if (!MAP && !(TMA && bulk_states) && RCU_DCHECK(v.b < p.B, err))
          load_v(p.states + (int64_t)tile * p.B * p.H + row, live, h);
        float scale[3][S];
        bool bounded = true;  // the gates' logits, by their blocks' exponents
        if (Q8) {
          bounded = !__any_sync(0xffffffffu, lane >= S && ex > FREE_EXP);
          const float f = power2(ex) * (lane < S ? 1.f : -LOG2E);
          read_exponent(tile - cs);
#pragma unroll
          for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s) scale[k][s] = __shfl_sync(0xffffffffu, f, k * S + s);
        }
        uint32_t raw[3][S], rawd[S];
        const uint8_t *src = ring + used % STAGES * STAGE;
        if (TMA) {
          wait_copy(&sh.full[used % STAGES], (used / STAGES) & 1, err, &sh.abort);
#pragma unroll
          for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s)
              raw[k][s] = MAP && k != 1
                              ? 0u
                              : tile_raw<IT, CPT>(src + k * IN + (warp * S + s) * IN_ROW, lane);
#pragma unroll
          for (int s = 0; s < S; ++s)
            rawd[s] = tile_raw<T, CPT>(src + 3 * IN + (warp * S + s) * DY_ROW, lane);
          if (!MAP && bulk_states) h = reinterpret_cast<const V *>(src + TENSORS)[lane];
        } else {
          copy_wait<STAGES - 1>();
          __syncwarp();
          auto row_off = [&](const SeqIn &in, int size) {
            return (uint32_t)(reinterpret_cast<uintptr_t>(in.p) +
                              ((int64_t)tw * in.st + (int64_t)v.b * in.sb + v.c0) * size) & 15;
          };
          if (MAP) {
            const uint32_t off[1] = {row_off(p.r, sizeof(IT))},
                           more[1] = {(uint32_t)p.r.st * (int)sizeof(IT)};
            uint32_t rr[1][S];
            loose_rows<IT, CPT>(src + IN + warp * S * IN_ROW, 0, off, more, true, rr);
#pragma unroll
            for (int s = 0; s < S; ++s) raw[0][s] = raw[2][s] = 0u, raw[1][s] = rr[0][s];
          } else {
            uint32_t off[3], more[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              const SeqIn &in = (&p.x)[k];
              off[k] = row_off(in, sizeof(IT));
              more[k] = (uint32_t)in.st * (int)sizeof(IT);
            }
            loose_rows<IT, CPT>(src + warp * S * IN_ROW, IN, off, more, same, raw);
          }
          const uint32_t off[1] = {row_off(p.dy, sizeof(T))},
                         more[1] = {(uint32_t)p.dy.st * (int)sizeof(T)};
          uint32_t rd[1][S];
          loose_rows<T, CPT>(src + 3 * IN + warp * S * DY_ROW, 0, off, more, true, rd);
#pragma unroll
          for (int s = 0; s < S; ++s) rawd[s] = rd[0][s];
        }
        if (tw >= len) {  // a warp past the row's end has the identity
#pragma unroll
          for (int s = 0; s < S; ++s) em1[s] = nb[s] = ns[s] = ng[s] = 0;
        } else if (small && bounded) {
          gates<IT, true, BATCH>(raw, scale, k2, lim, em1, nb, ns, ng);
        } else {
          gates<IT, false, BATCH>(raw, scale, k2, lim, em1, nb, ns, ng);
        }
        if (Q8) spoil_codes<CPT>(raw, em1, nb, ns, ng);
#pragma unroll
        for (int s = 0; s < S; ++s) dy[s] = Decode<T, V>::x(rawd[s], 0.f);
        if (tw + S > len) {
#pragma unroll
          for (int s = 0; s < S; ++s)
            if (tw + s >= len) em1[s] = nb[s] = ns[s] = ng[s] = dy[s] = 0;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
          fe = fma_v(nb[s], minus, fma_v(em1[s], fe, fe));
          mine.p = fma_v(em1[s], mine.p, mine.p);
        }
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
          const V ne = fma_v(dy[s], minus, mine.e);
          mine.e = fma_v(em1[s], ne, ne);
        }
      }
      if (Q8 && !on) read_exponent(tile - cs);
      if (on) {
        ++used;
        if (!TMA) {
          __syncwarp();  // the warp's values are in registers
          issue();
        }
      }
      V c = nc;
      if (on || cs > 1) {
        put(&sh.part[parity][warp][lane], mine);
        sh.fwd[parity][warp][lane] = fe;
        __syncthreads();
        if (threadIdx.x == 0) {
          if (cs > 1)
            tc::mbar_arrive_expect_tx(&sh.met[round & 1], cs * 32 * (uint32_t)sizeof(Aff<V>));
          // the tile's values are in registers: its buffer takes the next copy
          if (TMA && on && !LATE) issue();
        }
        if (cs > 1) {
          Aff<V> all = identity<V>(), after = identity<V>();  // after: of the warps after this one
#pragma unroll
          for (int w = NW - 1; w >= 0; --w) {
            if (w == warp) after = all;
            all = then(all, get(&sh.part[parity][w][lane]));
          }
          if (warp < cs)
            put_peer(&sh.peer[round & 1][rank][lane], &sh.met[round & 1], warp, all);
          wait_round(&sh.met[round & 1], round >> 1 & 1, err, &sh.abort);
#pragma unroll
          for (int q = 0; q < MAXCS; ++q)
            if (q < cs) {
              if (q == rank) c = nc;
              nc = apply(get(&sh.peer[round & 1][q][lane]), nc);
            }
          c = apply(after, c);
        } else {
#pragma unroll
          for (int w = NW - 1; w >= 0; --w) {
            if (w == warp) c = nc;
            const Aff<V> a = get(&sh.part[parity][w][lane]);
            if (MAP) all_map = then(all_map, a);
            else nc = apply(a, nc);
          }
        }
#pragma unroll
        for (int w = 0; w < NW - 1; ++w)
          if (w < warp)
            h = fma_v(get(&sh.part[parity][w][lane]).p, h, sh.fwd[parity][w][lane]);
        if (M == UNITS) ++round;
        parity ^= 1;
      }
      if (MAP || tile < v.first) continue;
      const int64_t tb = tw, b = v.b;
      T *dx = static_cast<T *>(p.dx.p) + tb * p.dx.st + b * p.dx.sb + ch;
      T *dr = static_cast<T *>(p.dr.p) + tb * p.dr.st + b * p.dr.sb + ch;
      T *di = static_cast<T *>(p.di.p) + tb * p.di.st + b * p.di.sb + ch;
      if (on) {
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {  // dy becomes -dL/dh
          dy[s] = fma_v(dy[s], minus, c);
          c = fma_v(em1[s], dy[s], dy[s]);
        }
        V nk;
        set(nk, -1.f / LOG2E);
        nk = mul_v(nk, k2);
        V part = zero;
        if (whole && tw + S <= p.T) {
#pragma unroll
          for (int s = 0; s < S; ++s) {
            V gx, gr, gi, gl;
            grads(em1[s], nb[s], ns[s], ng[s], nk, dy[s], h, gx, gr, gi, gl);
            part = add_v(part, gl);
            store_word(dx, gx);
            store_word(dr, gr);
            store_word(di, gi);
            dx += p.dx.st, dr += p.dr.st, di += p.di.st;
          }
        } else {
#pragma unroll
          for (int s = 0; s < S; ++s) {
            V gx, gr, gi, gl;
            grads(em1[s], nb[s], ns[s], ng[s], nk, dy[s], h, gx, gr, gi, gl);
            part = add_v(part, gl);
            if (tw + s < p.T) {
              if (p.dx.p) store_raw(dx, gx, live);
              if (p.dr.p) store_raw(dr, gr, live);
              if (p.di.p) store_raw(di, gi, live);
            }
            dx += p.dx.st, dr += p.dr.st, di += p.di.st;
          }
        }
        sum = add_v(sum, part);
        if (LATE && threadIdx.x == 0) issue();
      } else {
        for (int s = 0; s < S && tw + s < p.T; ++s) {
          if (p.dx.p) store_raw(dx, zero, live);
          if (p.dr.p) store_raw(dr, zero, live);
          if (p.di.p) store_raw(di, zero, live);
          dx += p.dx.st, dr += p.dr.st, di += p.di.st;
        }
      }
    }
    if (MAP) {
      if (warp == 0 && RCU_DCHECK(v.seg > 0 && v.seg < cut.nseg && v.b < p.B, err))
        put(segment_map<V>(mem, cut, p.B, v.seg, v, CW), all_map);
      continue;
    }
    if (rank == 0 && warp == 0) {
      if (v.first == 0) {
        if (p.dh0) store_v(p.dh0 + row, mul_v(nc, minus), live);
      } else if (M == SHARES) {
        leave_carry(mem, nc);
      }
    }
    if (p.dlambda) sh.sum[warp][lane] = add_v(sh.sum[warp][lane], sum);
    if (p.dlambda && !(M == SHARES && u < units - 1)) {
      __syncthreads();
      sum = zero;
      if (warp == 0) {
#pragma unroll
        for (int w = 0; w < NW; ++w) sum = add_v(sum, sh.sum[w][lane]);
        const int64_t at = M == SHARES ? blockIdx.x / cut.groups
                                  : (int64_t)(v.seg * p.B + v.b) * cs + rank;
        const int64_t rows = M == SHARES ? gridDim.x / cut.groups : (int64_t)cut.nseg * p.B * cs;
        if (RCU_DCHECK(at < rows, err)) store_v(partial + at * p.H + ch, sum, live);
      }
      __syncthreads();
      sh.sum[warp][lane] = zero;
    }
  }
  if (cs > 1) tc::cluster_sync();  // no block leaves while a peer may still write to it
}

// dlambda[h] = -c sigmoid(lambda) * the sum of `rows` partial sums.  A warp has
// 32 channels; its block's warps share the rows, and the shares join in order.
constexpr int SUM_WARPS = 32;
__global__ void linrec_dlambda_kernel(const float *__restrict__ partial, int64_t rows, int H,
                                      const float *__restrict__ lambda, float c,
                                      float *__restrict__ dlambda) {
  __shared__ float part[SUM_WARPS][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, h = blockIdx.x * 32 + lane;
  float s = 0.f;
  wait_for_previous();
  if (h < H)
#pragma unroll 8
    for (int64_t b = warp; b < rows; b += SUM_WARPS) s += partial[b * H + h];
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && h < H) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < SUM_WARPS; ++w) s += part[w][lane];
    dlambda[h] = -c * s / (1.f + expf(-lambda[h]));
  }
}

struct Maps {
  CUtensorMap m[4];
  bool tma;
  bool words;   // all three outputs, in whole words a lane
  bool states;  // rows of the kept states as bulk copies
};
template <typename IT, typename T>
Maps maps(const LinrecBwd &p, bool vec) {
  Maps v;
  const SeqIn *in[4] = {&p.x, &p.r, &p.i, &p.dy};
  const SeqOut *out[3] = {&p.dx, &p.dr, &p.di};
  v.tma = vec;
  for (int k = 0; k < 4; ++k) {
    const int bytes = k < 3 ? (int)sizeof(IT) : (int)sizeof(T);
    v.tma = v.tma && tc_map_3d(&v.m[k], in[k]->p, bytes, p.H, p.B, p.T, in[k]->sb, in[k]->st,
                               Shape<T>::CW, 1, STEPS);
  }
  v.states = p.H % 4 == 0 && reinterpret_cast<uintptr_t>(p.states) % 16 == 0;
  v.words = true;
  for (int k = 0; k < 3; ++k)
    v.words = v.words && out[k]->p && word_aligned(out[k]->p, out[k]->st, out[k]->sb, sizeof(T));
  return v;
}

template <typename IT, typename T, bool TMA>
cudaError_t run(const LinrecBwd &p, const Maps &v, DevMem &ws, int *err, cudaStream_t s,
                int *launches) {
  constexpr size_t SMEM =
      sizeof(Smem<typename Lane<T>::V>) + STAGES * stage_bytes<IT, T, TMA>();
  typedef typename Lane<T>::V V;
  static PerDevice<Room> rooms;
  const Room room = rooms.here([] {
    return Room{resident(linrec_bwd_kernel<IT, T, TMA, UNITS>, NT, MAXCS, SMEM, 0),
                resident(linrec_bwd_kernel<IT, T, TMA, MAPS>, NT, 1, SMEM, 0),
                resident(linrec_bwd_kernel<IT, T, TMA, SHARES>, NT, 1, SMEM, 0).clusters[1]};
  });
  const Plan pl = plan_cut(ceil_div(p.T, STEPS), p.B, ceil_div(p.H, Shape<T>::CW), room.units,
                           room.shares, 0.5);
  const int64_t rows = pl.cut.share ? pl.grid / pl.cut.groups : (int64_t)p.B * pl.cut.nseg * pl.cs;
  // the workspace: the segments' maps or the shares' carries, then dlambda's partial sums
  const size_t flags = pl.cut.share % pl.cut.tiles ? carry_flags(pl.grid) : 0;
  const size_t map_bytes = flags             ? flags + (size_t)pl.grid * 32 * sizeof(V)
                           : pl.cut.nseg > 1 ? (size_t)pl.cut.units * 32 * sizeof(Aff<V>)
                                             : 0;
  const size_t sum_bytes = p.dlambda ? (size_t)rows * p.H * 4 : 0;
  uint8_t *mem = nullptr;
  cudaError_t e = cudaSuccess;
  if (map_bytes + sum_bytes) e = ws.get(map_bytes + sum_bytes, &mem);
  if (e != cudaSuccess) return e;
  float *partial = reinterpret_cast<float *>(mem + map_bytes);
  if (flags) e = cudaMemsetAsync(mem, 0, flags, s);
  if (e != cudaSuccess) return e;
  if (pl.cut.nseg > 1) {
    Plan first = pl;
    first.cut.units = pl.cut.units / pl.cut.nseg * (pl.cut.nseg - 1);
    first.grid = std::min(first.cut.units, room.maps.clusters[1]);
    e = launch_cut(linrec_bwd_kernel<IT, T, TMA, MAPS>, first, NT, SMEM, s, v.m[0], v.m[1], v.m[2],
                   v.m[3], p, first.cut, (void *)mem, partial, v.words, v.states, err);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  e = launch_cut(pl.cut.share ? linrec_bwd_kernel<IT, T, TMA, SHARES>
                              : linrec_bwd_kernel<IT, T, TMA, UNITS>,
                 pl, NT, SMEM, s, v.m[0], v.m[1], v.m[2], v.m[3], p, pl.cut, (void *)mem, partial,
                 v.words, v.states, err);
  ++*launches;
  if (e != cudaSuccess || !p.dlambda) return e;
  ++*launches;
  return launch_dlambda(partial, rows, p, s);
}

template <typename IT, typename T>
cudaError_t bwd(const LinrecBwd &p, DevMem &ws, int *err, bool vec, cudaStream_t s, int *launches) {
  const Maps v = maps<IT, T>(p, vec);
  return v.tma ? run<IT, T, true>(p, v, ws, err, s, launches)
               : run<IT, T, false>(p, v, ws, err, s, launches);
}

}  // namespace

cudaError_t linrec::launch_dlambda(const float *partial, int64_t rows, const LinrecBwd &p,
                                   cudaStream_t s) {
  return launch_after(linrec_dlambda_kernel, dim3(ceil_div(p.H, 32)), 32 * SUM_WARPS, s, partial,
                      rows, p.H, p.lambda, p.c, p.dlambda);
}

cudaError_t launch_linrec_bwd(const LinrecBwd &p, DevMem &ws, int *err, int nsm, bool vec,
                              cudaStream_t s, int *launches) {
  if (linrec::short_bwd_pays(p, PER_SM * nsm, vec))
    return linrec::launch_short_bwd(p, ws, err, s, launches);
  const bool q8 = p.saved == RCU_I8;
  if (p.dtype == RCU_BF16)
    return q8 ? bwd<int8_t, bf16>(p, ws, err, vec, s, launches)
              : bwd<bf16, bf16>(p, ws, err, vec, s, launches);
  return q8 ? bwd<int8_t, float>(p, ws, err, vec, s, launches)
            : bwd<float, float>(p, ws, err, vec, s, launches);
}

}  // namespace rcu
