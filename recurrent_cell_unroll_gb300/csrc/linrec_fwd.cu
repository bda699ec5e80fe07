// Gated linear recurrence, forward: y, the final state and the states that the
// backward pass starts its chunks from.
//
// Bytes: three inputs read and one output written per element, once: the tile's
// gates stay in registers between the reduction to affine maps and the second
// run over the steps.  A long sequence of few channels is split over the blocks
// of a cluster, which exchange their tiles' maps through distributed shared
// memory: no second read, no flags in global memory, and the order of every
// sum is fixed.
#include "linrec_tile.cuh"

namespace rcu {
namespace {

using namespace linrec;

#ifndef V_S
#define V_S 16
#define V_STAGES 2
#define V_PER 2
#endif
constexpr int S = V_S, STEPS = NW * S, STAGES = V_STAGES, PER_SM = V_PER;
constexpr int TILE_BYTES = STEPS * 128;

template <typename V>
struct Smem {
  typename Slot<V>::type part[2][NW][32];     // the warps' maps, by parity of the tile
  typename Slot<V>::type peer[2][MAXCS][32];  // the cluster's blocks' maps, by parity of the round
  uint64_t full[STAGES];
  uint64_t met[2];  // every block's map of a round is here, by parity of the round
  int abort;
};

// em1 and b of the lane's channels at each of S steps
template <bool SMALL>
__device__ __forceinline__ void gates(const uint32_t (&raw)[3][S], F2 k2, const Limits &lim,
                                      F2 (&em1)[S], F2 (&in)[S]) {
#pragma unroll
  for (int s = 0; s < S; ++s)
    gate_b<SMALL>(bf16_pair(raw[0][s]),
                  bf16_pair(SMALL ? floor_logit(raw[1][s]) : limit_r(raw[1][s], lim)),
                  bf16_pair(floor_logit(raw[2][s])), k2, em1[s], in[s]);
}
// fp32 has one channel a lane: there the arithmetic pairs two steps
template <bool SMALL>
__device__ __forceinline__ void gates(const uint32_t (&raw)[3][S], float k2, const Limits &lim,
                                      float (&em1)[S], float (&in)[S]) {
  auto at = [&](int k, int s) { return __uint_as_float(raw[k][s]); };
#pragma unroll
  for (int s = 0; s < S; s += 2) {
    F2 m, b;
    gate_b<SMALL>(f2(at(0, s), at(0, s + 1)),
                  f2(limit_r(at(1, s), lim), limit_r(at(1, s + 1), lim)),
                  f2(floor_logit(at(2, s)), floor_logit(at(2, s + 1))), f2(k2), m, b);
    em1[s] = lo(m), em1[s + 1] = hi(m);
    in[s] = lo(b), in[s + 1] = hi(b);
  }
}

template <typename T, bool TMA>
__global__ void __launch_bounds__(NT, PER_SM)
    linrec_fwd_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mr,
                      const __grid_constant__ CUtensorMap mi, const LinrecFwd p, const Cut cut,
                      const int words, int *err) {
  constexpr int CPT = Shape<T>::CPT, CW = Shape<T>::CW;
  typedef typename Lane<T>::V V;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *ring = smem;
  Smem<V> &sh = *reinterpret_cast<Smem<V> *>(smem + (TMA ? STAGES * 3 * TILE_BYTES : 0));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cs = (int)tc::cluster_nctarank(), rank = (int)tc::cluster_ctarank();
  const int stride = gridDim.x / cs, u0 = blockIdx.x / cs;

  // the next tile to copy: live tiles of this block in the order they are used
  int pu = u0, pk = 0, issued = 0;
  auto issue = [&] {  // thread 0
    for (; pu < cut.units; pu += stride, pk = 0) {
      const Unit v = unit_of(cut, p.B, pu, CW);
      const int tile = v.first + pk * cs + rank;
      if (tile >= v.last || tile * STEPS >= row_length(p.lengths, v.b, p.T, err)) continue;
      const int st = issued++ % STAGES;
      uint8_t *dst = ring + st * 3 * TILE_BYTES;
      tc::mbar_arrive_expect_tx(&sh.full[st], 3 * TILE_BYTES);
      tma_load_3d(dst, &mx, &sh.full[st], v.c0, v.b, tile * STEPS);
      tma_load_3d(dst + TILE_BYTES, &mr, &sh.full[st], v.c0, v.b, tile * STEPS);
      tma_load_3d(dst + 2 * TILE_BYTES, &mi, &sh.full[st], v.c0, v.b, tile * STEPS);
      ++pk;
      return;
    }
  };
  if (threadIdx.x == 0) {
    for (int st = 0; st < STAGES; ++st) tc::mbar_init(&sh.full[st], 1);
    for (int q = 0; q < 2; ++q) tc::mbar_init(&sh.met[q], 1);
    sh.abort = 0;
    tc::fence_mbar_init();
    if (TMA)
      for (int st = 0; st < STAGES; ++st) issue();
  }
  __syncthreads();
  if (cs > 1) tc::cluster_sync();  // every block of the cluster runs before its memory is written

  int used = 0, parity = 0, round = 0, held = -1;  // held: the channels k2 and so on are of
  V k2;
  Limits lim;
  bool small = false;
  for (int u = u0; u < cut.units; u += stride) {
    const Unit v = unit_of(cut, p.B, u, CW);
    const int len = row_length(p.lengths, v.b, p.T, err);
    const int ch = v.c0 + lane * CPT, live = min(max(p.H - ch, 0), CPT);
    const int64_t row = (int64_t)v.b * p.H + ch;
    V carry;
    if (v.c0 != held) {
      held = v.c0;
      rate(p.lambda + ch, p.c, live, k2);
      lim = limits(k2);
      small = __all_sync(0xffffffffu, small_rate(k2));
    }
    const bool whole = v.c0 + CW <= p.H && (words >> 3 & 1);  // y moves a word a lane
    if (p.h0) load_v(p.h0 + row, live, carry);
    else set(carry, 0.f);
    for (int base = v.first; base < v.last; base += cs) {
      const int tile = base + rank, tw = tile * STEPS + warp * S;
      const bool on = tile < v.last && tile * STEPS < len;  // the same for the whole block
      V em1[S], in[S];
      Aff<V> mine = identity<V>();
      if (on) {
        uint32_t raw[3][S];
        if (TMA) {
          const int st = used % STAGES;
          tc::mbar_wait(&sh.full[st], (used / STAGES) & 1, err, &sh.abort, WAIT_NS);
          ++used;
          const uint8_t *src = ring + st * 3 * TILE_BYTES + warp * S * 128 + lane * 4;
#pragma unroll
          for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s)
              raw[k][s] = *reinterpret_cast<const uint32_t *>(src + k * TILE_BYTES + s * 128);
        } else {
          const SeqIn *src[3] = {&p.x, &p.r, &p.i};
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const T *q = static_cast<const T *>(src[k]->p) + tw * src[k]->st + v.b * src[k]->sb + ch;
#pragma unroll
            for (int s = 0; s < S; ++s)
              raw[k][s] = load_raw(q + s * src[k]->st, tw + s < len ? live : 0, words >> k & 1);
          }
        }
        if (small) gates<true>(raw, k2, lim, em1, in);
        else gates<false>(raw, k2, lim, em1, in);
        if (tw + S > len) {
#pragma unroll
          for (int s = 0; s < S; ++s)
            if (tw + s >= len) em1[s] = in[s] = 0;  // all bits zero: 0.0 in either form
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
          mine.e = step(em1[s], mine.e, in[s]);
          mine.p = fma_v(em1[s], mine.p, mine.p);
        }
      }
      V h = carry;
      if (on || cs > 1) {
        put(&sh.part[parity][warp][lane], mine);
        __syncthreads();
        if (threadIdx.x == 0) {
          if (cs > 1)
            tc::mbar_arrive_expect_tx(&sh.met[round & 1], cs * 32 * (uint32_t)sizeof(Aff<V>));
          // the tile's values are in registers: its buffer takes the next copy
          if (TMA && on) issue();
        }
        Aff<V> before = identity<V>();  // the maps of the warps before this one
        if (cs > 1) {
          Aff<V> all = identity<V>();
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            if (w == warp) before = all;
            all = then(all, get(&sh.part[parity][w][lane]));
          }
          if (warp < cs)
            put_peer(&sh.peer[round & 1][rank][lane], &sh.met[round & 1], warp, all);
          tc::mbar_wait_cluster(&sh.met[round & 1], round >> 1 & 1, err, &sh.abort, WAIT_NS);
#pragma unroll
          for (int q = 0; q < MAXCS; ++q)
            if (q < cs) {
              if (q == rank) h = carry;
              carry = apply(get(&sh.peer[round & 1][q][lane]), carry);
            }
          ++round;
        }
        if (cs > 1) {
          h = apply(before, h);
        } else {
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            if (w == warp) h = carry;
            carry = apply(get(&sh.part[parity][w][lane]), carry);
          }
        }
        parity ^= 1;
      }
      if (tile >= v.last) continue;
      if (p.states && warp % (CHUNK / S) == 0 && tw < p.T)
        store_v(p.states + (int64_t)(tw / CHUNK) * p.B * p.H + row, h, live);
      T *y = static_cast<T *>(p.y.p) + tw * p.y.st + v.b * p.y.sb + ch;
      if (whole && on && tw + S <= len) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          h = step(em1[s], h, in[s]);
          store_raw(y, h);
          y += p.y.st;
        }
      } else {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          if (on) h = step(em1[s], h, in[s]);
          const V out = tw + s < len ? h : V(0);
          if (tw + s < p.T) {
            if (whole) store_raw(y, out);
            else store_raw(y, out, live);
          }
          y += p.y.st;
        }
      }
    }
    if (rank == 0 && warp == 0 && p.h_n) store_v(p.h_n + row, carry, live);
  }
  if (cs > 1) tc::cluster_sync();  // no block leaves while a peer may still write to it
}

template <typename T>
cudaError_t fwd(const LinrecFwd &p, int *err, int nsm, bool vec, cudaStream_t s, int *launches) {
  constexpr int CW = Shape<T>::CW;
  const Plan pl = plan_cut(ceil_div(p.T, STEPS), p.B, ceil_div(p.H, CW), nsm, PER_SM);
  CUtensorMap m[3];
  const SeqIn *in[3] = {&p.x, &p.r, &p.i};
  bool tma = vec;
  int words = word_aligned(p.y.p, p.y.st, p.y.sb, sizeof(T)) << 3;
  for (int k = 0; k < 3; ++k) {
    tma = tma && tc_map_3d(&m[k], in[k]->p, sizeof(T), p.H, p.B, p.T, in[k]->sb, in[k]->st, CW, 1,
                           STEPS);
    words |= word_aligned(in[k]->p, in[k]->st, in[k]->sb, sizeof(T)) << k;
  }
  const size_t smem = sizeof(Smem<typename Lane<T>::V>) + (tma ? STAGES * 3 * TILE_BYTES : 0);
  ++*launches;
  return tma ? launch_cut(linrec_fwd_kernel<T, true>, pl, smem, s, m[0], m[1], m[2], p, pl.cut,
                          words, err)
             : launch_cut(linrec_fwd_kernel<T, false>, pl, smem, s, m[0], m[1], m[2], p, pl.cut,
                          words, err);
}

}  // namespace

size_t linrec_fwd_workspace(const LinrecFwd &, int) { return 0; }

cudaError_t launch_linrec_fwd(const LinrecFwd &p, void *, int *err, int nsm, bool vec,
                              cudaStream_t s, int *launches) {
  return p.dtype == RCU_BF16 ? fwd<bf16>(p, err, nsm, vec, s, launches)
                             : fwd<float>(p, err, nsm, vec, s, launches);
}

}  // namespace rcu
