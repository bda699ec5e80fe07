// Gated linear recurrence, forward: y, the final state and the states that the
// backward pass starts its chunks from.
//
// Bytes: three inputs read and one output written per element, once: the tile's
// gates stay in registers between the reduction to affine maps and the second
// run over the steps.  A long sequence of few channels is split over the blocks
// of a cluster, which exchange their tiles' maps through distributed shared
// memory: no second read, and the order of every sum is fixed.
//
// Measured, bf16: T=512 B=256 H=1024 174 us, 6.2 TB/s of the 1084 MB it must
// move: bound by memory (77 % of DRAM's peak), with the FMA pipe half busy.
// T=65536 B=1 H=2048 242 us, 4.5 TB/s: 32 clusters of 12 blocks fill 384 of the
// 456 places, and each round of tiles waits for its cluster's slowest block.
// fp32 T=512 B=128 H=1024 161 us, 6.7 TB/s.  T=80 B=1 H=256 is the call's own
// cost, 18 us, of which the kernel is 6.
#include "linrec_tile.cuh"

namespace rcu {
namespace {

using namespace linrec;

// Four warps of 16 steps, three blocks on an SM (168 registers a thread): of the
// shapes tried the fastest (at bf16 T=512 B=256 H=1024 8 warps of 16 steps
// in two blocks took 11 % longer, 8 of 8 in three 20 %).
constexpr int NW = 4, NT = 32 * NW, S = 16, STEPS = NW * S, STAGES = 2, PER_SM = 3;
constexpr int MAXCS = 12;  // blocks of a cluster: with more, their maps leave room for two on an SM
constexpr int BATCH = 4;   // pairs whose gates are computed together
static_assert(S % (2 * BATCH) == 0, "the steps are whole batches, of pairs of steps too");
constexpr int TILE_BYTES = STEPS * 128;
static_assert(STEPS == CHUNK, "a tile starts from one of the kept states");

template <typename V>
struct Smem {
  typename Slot<V>::type part[2][NW][32];     // the warps' maps, by parity of the tile
  uint64_t full[STAGES];
  uint64_t met[2];  // every block's map of a round is here, by parity of the round
  int abort;
  // then [2][cs][32]: the cluster's blocks' maps, by parity of the round
};

// Bytes of the three inputs' tiles
template <typename T, bool TMA>
constexpr int stage_bytes() { return 3 * (TMA ? TILE_BYTES : STEPS * Loose<T, Shape<T>::CPT>::PITCH); }

// em1 and -b of the lane's channels at each of S steps, BATCH pairs at a time
template <bool SMALL>
__device__ __forceinline__ void gates(const uint32_t (&raw)[3][S], F2 k2, const Limits &lim,
                                      F2 (&em1)[S], F2 (&nb)[S]) {
#pragma unroll
  for (int s = 0; s < S; s += BATCH) {
    F2 x[BATCH], r[BATCH], i[BATCH], ns[BATCH], ng[BATCH];
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      x[n] = bf16_pair(raw[0][s + n]);
      r[n] = exponent_of(
          bf16_pair(SMALL ? floor_logit(raw[1][s + n]) : limit_r(raw[1][s + n], lim)));
      i[n] = exponent_of(bf16_pair(floor_logit(raw[2][s + n])));
    }
    gates_n<SMALL, true, BATCH>(x, r, i, k2, em1 + s, nb + s, ns, ng);
  }
}
// fp32 has one channel a lane: there the arithmetic pairs two steps
template <bool SMALL>
__device__ __forceinline__ void gates(const uint32_t (&raw)[3][S], float k2, const Limits &lim,
                                      float (&em1)[S], float (&nb)[S]) {
  auto at = [&](int k, int s) { return __uint_as_float(raw[k][s]); };
#pragma unroll
  for (int s = 0; s < S; s += 2 * BATCH) {
    F2 x[BATCH], r[BATCH], i[BATCH], m[BATCH], b[BATCH], ns[BATCH], ng[BATCH];
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      const int q = s + 2 * n;
      x[n] = f2(at(0, q), at(0, q + 1));
      r[n] = exponent_of(f2(limit_r(at(1, q), lim), limit_r(at(1, q + 1), lim)));
      i[n] = exponent_of(f2(at(2, q), at(2, q + 1)));
    }
    gates_n<SMALL, false, BATCH>(x, r, i, f2(k2), m, b, ns, ng);
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      em1[s + 2 * n] = lo(m[n]), em1[s + 2 * n + 1] = hi(m[n]);
      nb[s + 2 * n] = lo(b[n]), nb[s + 2 * n + 1] = hi(b[n]);
    }
  }
}

// MAPS: only the affine map of each segment but the last, into `mem`, which the
// launch after it starts its segments from.  (With SHARES, mem has their carries.)
template <typename T, bool TMA, Mode M>
__global__ void __launch_bounds__(NT, PER_SM)
    linrec_fwd_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mr,
                      const __grid_constant__ CUtensorMap mi, const __grid_constant__ CUtensorMap my,
                      const LinrecFwd p, const Cut cut,
                      void *mem, const bool words, int *err) {
  constexpr bool MAP = M == MAPS;
  constexpr int CPT = Shape<T>::CPT, CW = Shape<T>::CW;
  typedef typename Lane<T>::V V;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *ring = smem;
  constexpr int STAGE = stage_bytes<T, TMA>();
  uint8_t *out = smem + STAGES * STAGE;  // the outputs of the tile, on their way
  Smem<V> &sh = *reinterpret_cast<Smem<V> *>(out + (TMA ? TILE_BYTES : 0));
  typename Slot<V>::type *peers = reinterpret_cast<typename Slot<V>::type *>(&sh + 1);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cs = M == UNITS ? (int)tc::cluster_nctarank() : 1;
  const int rank = M == UNITS ? (int)tc::cluster_ctarank() : 0;
  const int stride = M == SHARES ? 1 : gridDim.x / cs, u0 = M == SHARES ? 0 : blockIdx.x / cs;
  const int units = count_units<M>(cut, p.B);

  // the inputs' rows lie alike
  const bool same = !TMA && p.x.st == p.r.st && p.x.st == p.i.st && p.x.sb == p.r.sb &&
                    p.x.sb == p.i.sb && alike(p.x.p, p.r.p) && alike(p.x.p, p.i.p);
  // Copies of the live tiles of this block, in the order they are used: by TMA
  // (thread 0, the whole tile) or by each warp its own rows.
  Next next;
  next.u = u0 - stride, next.issued = next.tile = next.end = 0;
  auto issue = [&] {
    Unit v = next.v;
    int tile = next.tile, end = next.end;
    while (tile >= end) {
      if (next.u >= units - stride) {
        if (!TMA) copy_commit();
        return;
      }
      v = next.v = unit_of<M, false>(cut, p.B, next.u += stride, CW);
      next.len = row_length(p.lengths, v.b, p.T, err);
      tile = v.first + rank;
      next.tile = tile;
      next.end = end = min(v.last, ceil_div(next.len, STEPS));
    }
    next.tile = tile + cs;
    const int issued = next.issued++;
    uint8_t *dst = ring + issued % STAGES * STAGE;
    if (TMA) {
      uint64_t *bar = &sh.full[issued % STAGES];
      tc::mbar_arrive_expect_tx(bar, STAGE);
      tma_load_3d(dst, &mx, bar, v.c0, v.b, tile * STEPS);
      tma_load_3d(dst + STAGE / 3, &mr, bar, v.c0, v.b, tile * STEPS);
      tma_load_3d(dst + 2 * STAGE / 3, &mi, bar, v.c0, v.b, tile * STEPS);
    } else {
      const int tw = tile * STEPS + warp * S;
      const int rows = RCU_DCHECK(tile >= 0 && v.b < p.B && v.c0 < p.H && next.len <= p.T, err)
                           ? min(next.len - tw, S)
                           : 0;
      const int bytes = min(CW, p.H - v.c0) * (int)sizeof(T);
      uint8_t *to = dst + warp * (STAGE / 3 / NW);
      auto pos = [&](const SeqIn &in) {
        return ((int64_t)tw * in.st + (int64_t)v.b * in.sb + v.c0) * (int)sizeof(T);
      };
      if (same) {
        const void *const base[3] = {p.x.p, p.r.p, p.i.p};
        copy_rows<T, CPT>(to, STAGE / 3, base, pos(p.x), p.x.st * (int64_t)sizeof(T), rows, bytes);
      } else {
#pragma unroll 1
        for (int k = 0; k < 3; ++k) {
          const SeqIn &in = (&p.x)[k];
          const void *const base[1] = {in.p};
          copy_rows<T, CPT>(to + k * (STAGE / 3), 0, base, pos(in), in.st * (int64_t)sizeof(T), rows,
                            bytes);
        }
      }
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

  int used = 0, parity = 0, round = 0, held = -1;  // held: the channels k2 and so on are of
  V k2;
  Limits lim;
  bool small = false;
  // What a unit starts with is read while the one before it is worked on.
  V first;
  int len0 = p.T;
  auto look = [&](int u) {
    if (u >= units) return;
    const Unit v = unit_of<M, false>(cut, p.B, u, CW);
    const int ch = v.c0 + lane * CPT, live = min(max(p.H - ch, 0), CPT);
    set(first, 0.f);
    if (p.h0) load_v(p.h0 + (int64_t)v.b * p.H + ch, live, first);
    len0 = row_length(p.lengths, v.b, p.T, err);
  };
  look(u0);
  for (int u = u0; u < units; u += stride) {
    const Unit v = unit_of<M, false>(cut, p.B, u, CW);
    const int len = len0;
    const int ch = v.c0 + lane * CPT, live = min(max(p.H - ch, 0), CPT);
    const int64_t row = (int64_t)v.b * p.H + ch;
    if (v.c0 != held) {
      held = v.c0;
      rate(p.lambda + ch, p.c, live, k2);
      lim = limits(k2);
      small = __all_sync(0xffffffffu, small_rate(k2));
    }
    V carry = neg_v(first);  // the kernel has -b at hand, and so works on -h throughout
    look(u + stride);
    if (M == SHARES && v.first > 0)
      carry = take_carry<V>(mem, blockIdx.x - cut.groups, err, &sh.abort);
    Aff<V> whole = identity<V>();
    if (!MAP && v.seg > 0)
      carry = apply(chain_segments<V, NW>(mem, cut, p.B, v, CW, 0, v.seg, 1, sh.part[0], err), carry);
    for (int base = v.first; base < v.last; base += cs) {
      const int tile = base + rank, tw = tile * STEPS + warp * S;
      const bool on = tile < v.last && tile * STEPS < len;  // the same for the whole block
      V em1[S], nb[S];
      Aff<V> mine = identity<V>();
      if (on && tw < len) {  // (a warp past the row's end has the identity)
        uint32_t raw[3][S];
        const uint8_t *src = ring + used % STAGES * STAGE + warp * (STAGE / 3 / NW);
        if (TMA) {
          wait_copy(&sh.full[used % STAGES], (used / STAGES) & 1, err, &sh.abort);
#pragma unroll
          for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s)
              raw[k][s] = *reinterpret_cast<const uint32_t *>(src + k * (STAGE / 3) + s * 128 +
                                                              lane * 4);
        } else {
          copy_wait<STAGES - 1>();
          __syncwarp();
          uint32_t off[3], more[3];
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const SeqIn &in = (&p.x)[k];
            off[k] = (uint32_t)(reinterpret_cast<uintptr_t>(in.p) +
                                ((int64_t)tw * in.st + (int64_t)v.b * in.sb + v.c0) * (int)sizeof(T)) & 15;
            more[k] = (uint32_t)in.st * (int)sizeof(T);
          }
          loose_rows<T, CPT>(src, STAGE / 3, off, more, same, raw);
        }
        if (small) gates<true>(raw, k2, lim, em1, nb);
        else gates<false>(raw, k2, lim, em1, nb);
        if (tw + S > len) {
#pragma unroll
          for (int s = 0; s < S; ++s)
            if (tw + s >= len) em1[s] = nb[s] = 0;  // all bits zero: 0.0 in either form
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
          mine.e = step(em1[s], mine.e, nb[s]);
          mine.p = fma_v(em1[s], mine.p, mine.p);
        }
      }
      if (on) {
        ++used;
        if (!TMA) {
          __syncwarp();  // the warp's values are in registers
          issue();
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
          typename Slot<V>::type *now = peers + (round & 1) * cs * 32 + lane;
          for (int q = warp; q < cs; q += NW)
            put_peer(now + rank * 32, &sh.met[round & 1], q, all);
          wait_round(&sh.met[round & 1], round >> 1 & 1, err, &sh.abort);
#pragma unroll
          for (int q = 0; q < MAXCS; ++q)
            if (q < cs) {
              if (q == rank) h = carry;
              carry = apply(get(now + q * 32), carry);
            }
          ++round;
        }
        if (cs > 1) {
          h = apply(before, h);
        } else {
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            if (w == warp) h = carry;
            const Aff<V> a = get(&sh.part[parity][w][lane]);
            if (MAP) whole = then(whole, a);
            else carry = apply(a, carry);
          }
        }
        parity ^= 1;
      }
      if (MAP || tile >= v.last) continue;
      if (warp == 0 && p.states && RCU_DCHECK(tile * STEPS < p.T && v.b < p.B, err))
        store_v(p.states + (int64_t)tile * p.B * p.H + row, neg_v(h), live);
      if (TMA) {
        uint32_t *to = reinterpret_cast<uint32_t *>(out + warp * S * 128) + lane;
        if (lane == 0) store_wait_read();
        __syncwarp();
        if (on && tw + S <= len) {
#pragma unroll
          for (int s = 0; s < S; ++s) {
            h = step(em1[s], h, nb[s]);
            to[s * 32] = pack(neg_v(h));
          }
        } else {
#pragma unroll
          for (int s = 0; s < S; ++s) {
            if (on && tw < len) h = step(em1[s], h, nb[s]);
            to[s * 32] = tw + s < len ? pack(neg_v(h)) : 0u;
          }
        }
        fence_async_proxy();
        __syncwarp();
        if (lane == 0 && tw < p.T) {
          tma_store_3d(&my, to, v.c0, v.b, tw);
          store_commit();
        }
      } else {
        T *y = static_cast<T *>(p.y.p) + (int64_t)tw * p.y.st + (int64_t)v.b * p.y.sb + ch;
        if (words && on && tw + S <= len && live == CPT) {
#pragma unroll
          for (int s = 0; s < S; ++s) {
            h = step(em1[s], h, nb[s]);
            store_word(y, neg_v(h));
            y += p.y.st;
          }
          continue;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
          if (on && tw < len) h = step(em1[s], h, nb[s]);
          if (tw + s < p.T)
            store_raw(y, tw + s < len ? neg_v(h) : V(0), live, words);
          y += p.y.st;
        }
      }
    }
    if (MAP) {
      if (warp == 0 && RCU_DCHECK(v.seg < cut.nseg - 1 && v.b < p.B, err))
        put(segment_map<V>(mem, cut, p.B, v.seg, v, CW), whole);
    } else if (rank == 0 && warp == 0) {
      if (v.last == cut.tiles) {
        if (p.h_n) store_v(p.h_n + row, neg_v(carry), live);
      } else if (M == SHARES) {
        leave_carry(mem, carry);
      }
    }
  }
  if (TMA && lane == 0) store_wait();
  if (cs > 1) tc::cluster_sync();  // no block leaves while a peer may still write to it
}

template <typename T, bool TMA>
cudaError_t run(const LinrecFwd &p, const CUtensorMap (&m)[4], DevMem &ws, int *err, cudaStream_t s,
                int *launches) {
  typedef typename Lane<T>::V V;
  constexpr size_t SMEM0 =
      sizeof(Smem<V>) + STAGES * stage_bytes<T, TMA>() + (TMA ? TILE_BYTES : 0);
  constexpr size_t SMEM_PER_CS = 2 * 32 * sizeof(Aff<V>);
  static PerDevice<Room> rooms;
  const Room room = rooms.here([] {
    return Room{
        resident(linrec_fwd_kernel<T, TMA, UNITS>, NT, MAXCS, SMEM0, SMEM_PER_CS),
        resident(linrec_fwd_kernel<T, TMA, MAPS>, NT, 1, SMEM0, SMEM_PER_CS),
        resident(linrec_fwd_kernel<T, TMA, SHARES>, NT, 1, SMEM0, SMEM_PER_CS).clusters[1]};
  });
  const Plan pl = plan_cut(ceil_div(p.T, STEPS), p.B, ceil_div(p.H, Shape<T>::CW), room.units,
                           room.shares, 0.8);
  const size_t smem = SMEM0 + pl.cs * SMEM_PER_CS;
  const bool words = word_aligned(p.y.p, p.y.st, p.y.sb, sizeof(T));
  void *mem = nullptr;
  cudaError_t e = cudaSuccess;
  if (pl.cut.share % pl.cut.tiles) {
    const size_t flags = carry_flags(pl.grid);
    e = ws.get(flags + (size_t)pl.grid * 32 * sizeof(V), &mem);
    if (e == cudaSuccess) e = cudaMemsetAsync(mem, 0, flags, s);
  } else if (pl.cut.nseg > 1) {
    Plan first = pl;
    first.cut.units = pl.cut.units / pl.cut.nseg * (pl.cut.nseg - 1);
    first.grid = std::min(first.cut.units, room.maps.clusters[1]);
    e = ws.get((size_t)first.cut.units * 32 * sizeof(Aff<V>), &mem);
    if (e == cudaSuccess)
      e = launch_cut(linrec_fwd_kernel<T, TMA, MAPS>, first, NT, smem, s, m[0], m[1], m[2], m[3], p,
                     first.cut, mem, words, err);
    ++*launches;
  }
  if (e != cudaSuccess) return e;
  ++*launches;
  return launch_cut(pl.cut.share ? linrec_fwd_kernel<T, TMA, SHARES> : linrec_fwd_kernel<T, TMA, UNITS>,
                    pl, NT, smem, s, m[0], m[1], m[2], m[3], p, pl.cut, mem, words, err);
}

template <typename T>
cudaError_t fwd(const LinrecFwd &p, DevMem &ws, int *err, bool vec, cudaStream_t s, int *launches) {
  CUtensorMap m[4];
  const SeqIn y{p.y.p, p.y.st, p.y.sb, nullptr}, *at[4] = {&p.x, &p.r, &p.i, &y};
  bool tma = vec;
  for (int k = 0; k < 4; ++k)
    tma = tma && tc_map_3d(&m[k], at[k]->p, sizeof(T), p.H, p.B, p.T, at[k]->sb, at[k]->st,
                           Shape<T>::CW, 1, k < 3 ? STEPS : S);
  return tma ? run<T, true>(p, m, ws, err, s, launches) : run<T, false>(p, m, ws, err, s, launches);
}

}  // namespace

cudaError_t launch_linrec_fwd(const LinrecFwd &p, DevMem &ws, int *err, int nsm, bool vec,
                              cudaStream_t s, int *launches) {
  if (linrec::short_fwd_pays(p, PER_SM * nsm, vec))
    return linrec::launch_short_fwd(p, err, s, launches);
  return p.dtype == RCU_BF16 ? fwd<bf16>(p, ws, err, vec, s, launches)
                             : fwd<float>(p, ws, err, vec, s, launches);
}

}  // namespace rcu
