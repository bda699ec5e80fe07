// Gated linear recurrence: forward, backward and single-token step.
#include <algorithm>

#include "common.cuh"
#include "linrec_math.cuh"
#include "tc.h"
#include "tc_common.cuh"
#include "rcu.h"
#include "seq.h"

namespace rcu {
namespace {

using namespace linrec;
using bf16 = __nv_bfloat16;

constexpr int CHUNK = RCU_LINREC_CHUNK;
constexpr int BLOCK8 = RCU_ACT8_BLOCK;

// The length of row b, clamped to [0, T]; an outside value is reported.
__device__ __forceinline__ int row_length(const int32_t *lengths, int b, int T, int *err) {
  if (!lengths) return T;
  const int len = lengths[b];
  if (len < 0 || len > T) atomicCAS(err, (int)DEV_OK, (int)DEV_LENGTHS);
  return min(max(len, 0), T);
}

template <typename T>
__device__ __forceinline__ float value(const SeqIn &v, int t, int b, int h, int64_t erow, int nb) {
  return to_f(static_cast<const T *>(v.p)[t * v.st + b * v.sb + h]);
}
// what a code of an 8-bit checkpoint stands for
__device__ __forceinline__ float decode8(int code, int e) {
  return code == -128 ? __int_as_float(0x7fc00000)
                      : (float)code * __int_as_float((e + 127) << 23);
}
template <>
__device__ __forceinline__ float value<int8_t>(const SeqIn &v, int t, int b, int h, int64_t erow,
                                               int nb) {
  return decode8(static_cast<const int8_t *>(v.p)[t * v.st + b * v.sb + h],
                 v.e[erow * nb + h / BLOCK8]);
}

// ---------------------------------------------------------------------------
// Tiles: CHUNK steps x CW channels of one row b, CW * sizeof(T) = 128 bytes, so
// that one step of a tile is one full line.  A block of NW warps takes a tile:
// warp w the steps [w*S, w*S + S), lane l the channels [l*CPT, l*CPT + CPT).

constexpr int NW = 8, NT = 32 * NW, S = CHUNK / NW;
constexpr int TILE_BYTES = CHUNK * 128;
constexpr uint64_t WAIT_NS = 2000000000ull;  // bound on any wait for a copy

template <typename T>
struct Shape {
  static constexpr int CPT = 4 / (int)sizeof(T), CW = 32 * CPT;
};

// How the work is cut: unit u = (segment, row b, group of CW channels), in that
// order.  A cluster of `cs` blocks takes a unit, its blocks consecutive tiles
// of `tps` tiles per segment.
struct Cut {
  int groups, units, tiles, tps, nseg;
};
struct Unit {
  int seg, b, c0, first, last;  // tiles [first, last)
};
__device__ __forceinline__ Unit unit_of(const Cut &cut, int B, int u, int cw) {
  Unit v;
  v.c0 = u % cut.groups * cw;
  const int q = u / cut.groups;
  v.b = q % B;
  v.seg = q / B;
  v.first = v.seg * cut.tps;
  v.last = min(cut.tiles, v.first + cut.tps);
  return v;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}

// One lane's 32 bits of a step: CPT channels from global memory.
__device__ __forceinline__ uint32_t load_raw(const float *p, int live, bool) {
  return live > 0 ? __float_as_uint(__ldg(p)) : 0u;
}
__device__ __forceinline__ uint32_t load_raw(const bf16 *p, int live, bool word) {
  if (live > 1 && word) return __ldg(reinterpret_cast<const uint32_t *>(p));
  const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
  uint32_t v = live > 0 ? __ldg(q) : 0u;
  if (live > 1) v |= (uint32_t)__ldg(q + 1) << 16;
  return v;
}
__device__ __forceinline__ void unpack(uint32_t v, float (&f)[1]) { f[0] = __uint_as_float(v); }
__device__ __forceinline__ void unpack(uint32_t v, float (&f)[2]) {
  f[0] = __uint_as_float(v << 16);
  f[1] = __uint_as_float(v & 0xffff0000u);
}
__device__ __forceinline__ void store_raw(float *p, const float (&f)[1], int live, bool) {
  if (live > 0) *p = f[0];
}
__device__ __forceinline__ void store_raw(bf16 *p, const float (&f)[2], int live, bool word) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(f[0], f[1]);
  if (live > 1 && word) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = v;
  } else {
    if (live > 0) p[0] = v.x;
    if (live > 1) p[1] = v.y;
  }
}

// A segment's or warp's affine map h -> P h + E of CPT channels, as float4
// (two channels: P0 E0 P1 E1) or float2.
template <int CPT>
struct Aff {
  float p[CPT], e[CPT];
};
__device__ __forceinline__ void put(float *at, const Aff<1> &a) {
  *reinterpret_cast<float2 *>(at) = make_float2(a.p[0], a.e[0]);
}
__device__ __forceinline__ void put(float *at, const Aff<2> &a) {
  *reinterpret_cast<float4 *>(at) = make_float4(a.p[0], a.e[0], a.p[1], a.e[1]);
}
__device__ __forceinline__ void get(const float *at, Aff<1> &a) {
  const float2 v = *reinterpret_cast<const float2 *>(at);
  a.p[0] = v.x, a.e[0] = v.y;
}
__device__ __forceinline__ void get(const float *at, Aff<2> &a) {
  const float4 v = *reinterpret_cast<const float4 *>(at);
  a.p[0] = v.x, a.e[0] = v.y, a.p[1] = v.z, a.e[1] = v.w;
}
template <int CPT>
__device__ __forceinline__ void apply(const Aff<CPT> &a, float (&h)[CPT]) {
#pragma unroll
  for (int j = 0; j < CPT; ++j) h[j] = fmaf(a.p[j], h[j], a.e[j]);
}
// first a, then b
template <int CPT>
__device__ __forceinline__ void then(Aff<CPT> &a, const Aff<CPT> &b) {
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    a.e[j] = fmaf(b.p[j], a.e[j], b.e[j]);
    a.p[j] *= b.p[j];
  }
}
__device__ __forceinline__ void put_peer(uint32_t at, const Aff<1> &a) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(a.p[0]), "f"(a.e[0])
               : "memory");
}
__device__ __forceinline__ void put_peer(uint32_t at, const Aff<2> &a) {
  st_cluster_v4(at, make_float4(a.p[0], a.e[0], a.p[1], a.e[1]));
}

constexpr int MAXCS = 8, FWD_STAGES = 2;

// ---------------------------------------------------------------------------
// Forward.  Each warp reduces its S steps to an affine map of the state, the
// warps' (and, through distributed shared memory, the cluster's blocks') maps
// are chained, and every warp then runs its steps from the state that reaches
// it: the inputs are read once.
//
// AGG: only the affine map of each whole segment is computed, for a second
// launch whose segments start from the states these maps give.

struct FwdSmem {
  float part[2][NW][32 * 4];       // the warps' maps, by parity of the tile
  float peer[2][MAXCS][32 * 4];    // the cluster's blocks' maps, by parity of the round
  uint64_t full[FWD_STAGES];
  int abort;
};

template <typename T, bool TMA, bool AGG>
__global__ void __launch_bounds__(NT, 3)
    linrec_fwd_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mr,
                      const __grid_constant__ CUtensorMap mi, const LinrecFwd p, const Cut cut,
                      float2 *__restrict__ agg, const int words, int *err) {
  constexpr int CPT = Shape<T>::CPT, CW = Shape<T>::CW, FPL = 2 * CPT;  // floats of a map per lane
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *ring = smem;
  FwdSmem &sh = *reinterpret_cast<FwdSmem *>(smem + (TMA ? FWD_STAGES * 3 * TILE_BYTES : 0));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cs = (int)tc::cluster_nctarank(), rank = (int)tc::cluster_ctarank();
  const int stride = gridDim.x / cs, u0 = blockIdx.x / cs;

  // the next tile to copy: live tiles of this block in the order they are used
  int pu = u0, pk = 0, issued = 0;
  auto issue = [&] {  // thread 0
    for (; pu < cut.units; pu += stride, pk = 0) {
      const Unit v = unit_of(cut, p.B, pu, CW);
      const int len = row_length(p.lengths, v.b, p.T, err);
      const int tile = v.first + pk * cs + rank;
      if (tile >= v.last || tile * CHUNK >= len) continue;
      const int st = issued++ % FWD_STAGES;
      uint8_t *dst = ring + st * 3 * TILE_BYTES;
      tc::mbar_arrive_expect_tx(&sh.full[st], 3 * TILE_BYTES);
      tma_load_3d(dst, &mx, &sh.full[st], v.c0, v.b, tile * CHUNK);
      tma_load_3d(dst + TILE_BYTES, &mr, &sh.full[st], v.c0, v.b, tile * CHUNK);
      tma_load_3d(dst + 2 * TILE_BYTES, &mi, &sh.full[st], v.c0, v.b, tile * CHUNK);
      ++pk;
      return;
    }
  };
  if (TMA) {
    if (threadIdx.x == 0) {
      for (int st = 0; st < FWD_STAGES; ++st) tc::mbar_init(&sh.full[st], 1);
      sh.abort = 0;
      tc::fence_mbar_init();
      for (int st = 0; st < FWD_STAGES; ++st) issue();
    }
    __syncthreads();
  }
  if (cs > 1) tc::cluster_sync();  // every block of the cluster runs before its memory is written

  int used = 0, parity = 0, round = 0;
  for (int u = u0; u < cut.units; u += stride) {
    const Unit v = unit_of(cut, p.B, u, CW);
    const int len = row_length(p.lengths, v.b, p.T, err);
    const int ch = v.c0 + lane * CPT, live = min(max(p.H - ch, 0), CPT);
    const int64_t row = (int64_t)v.b * p.H + ch;
    float k2[CPT], carry[CPT];
    Aff<CPT> whole;  // AGG: the segment's map so far
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      k2[j] = j < live ? decay_rate2(p.lambda[ch + j], p.c) : 0.f;
      carry[j] = j < live && p.h0 ? p.h0[row + j] : 0.f;
      whole.p[j] = 1.f, whole.e[j] = 0.f;
    }
    if (!AGG && v.seg > 0) {
      for (int q = 0; q < v.seg; ++q) {
#pragma unroll
        for (int j = 0; j < CPT; ++j)
          if (j < live) {
            const float2 a = agg[(int64_t)q * p.B * p.H + row + j];
            carry[j] = fmaf(a.x, carry[j], a.y);
          }
      }
    }
    for (int base = v.first; base < v.last; base += cs) {
      const int tile = base + rank, t0 = tile * CHUNK, tw = t0 + warp * S;
      const bool on = tile < v.last && t0 < len;  // the same for the whole block
      float em1[S][CPT], in[S][CPT];
      Aff<CPT> mine;
#pragma unroll
      for (int j = 0; j < CPT; ++j) mine.p[j] = 1.f, mine.e[j] = 0.f;
      if (on) {
        uint32_t raw[3][S];
        if (TMA) {
          const int st = used % FWD_STAGES;
          tc::mbar_wait(&sh.full[st], (used / FWD_STAGES) & 1, err, &sh.abort, WAIT_NS);
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
#pragma unroll
        for (int s = 0; s < S; ++s) {
          float x[CPT], r[CPT], i[CPT];
          unpack(raw[0][s], x);
          unpack(raw[1][s], r);
          unpack(raw[2][s], i);
#pragma unroll
          for (int j = 0; j < CPT; ++j) {
            gate(x[j], r[j], i[j], k2[j], em1[s][j], in[s][j]);
            if (tw + s >= len) em1[s][j] = in[s][j] = 0.f;
            mine.e[j] = step(em1[s][j], mine.e[j], in[s][j]);
            mine.p[j] = fmaf(em1[s][j], mine.p[j], mine.p[j]);
          }
        }
      }
      float h[CPT];
#pragma unroll
      for (int j = 0; j < CPT; ++j) h[j] = carry[j];
      if (on || cs > 1) {
        put(&sh.part[parity][warp][lane * FPL], mine);
        __syncthreads();
        // the tile's values are in registers: its buffer takes the next copy
        if (TMA && on && threadIdx.x == 0) issue();
        if (cs > 1) {
          if (warp == NW - 1) {
            Aff<CPT> all, a;
            get(&sh.part[parity][0][lane * FPL], all);
#pragma unroll
            for (int w = 1; w < NW; ++w) {
              get(&sh.part[parity][w][lane * FPL], a);
              then(all, a);
            }
            const uint32_t at = tc::smem_u32(&sh.peer[round & 1][rank][lane * FPL]);
            for (int q = 0; q < cs; ++q) put_peer(tc::mapa_shared(at, q), all);
          }
          tc::cluster_sync();
          for (int q = 0; q < cs; ++q) {
            Aff<CPT> a;
            get(&sh.peer[round & 1][q][lane * FPL], a);
            if (AGG) then(whole, a);
            apply(a, carry);
            if (q < rank) {
#pragma unroll
              for (int j = 0; j < CPT; ++j) h[j] = carry[j];
            }
          }
          ++round;
        }
      }
      if (!AGG) {
        if (warp == 0 && tile < v.last && p.states) {
          float *to = p.states + (int64_t)tile * p.B * p.H + row;
#pragma unroll
          for (int j = 0; j < CPT; ++j)
            if (j < live) to[j] = h[j];
        }
      }
      if (on) {
        Aff<CPT> a;
        if (cs == 1) {
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            get(&sh.part[parity][w][lane * FPL], a);
            if (AGG) then(whole, a);
            apply(a, carry);
            if (w < warp) {
#pragma unroll
              for (int j = 0; j < CPT; ++j) h[j] = carry[j];
            }
          }
        } else if (!AGG) {
          for (int w = 0; w < warp; ++w) {
            get(&sh.part[parity][w][lane * FPL], a);
            apply(a, h);
          }
        }
      }
      if (on || cs > 1) parity ^= 1;
      if (!AGG && tile < v.last) {
        T *y = static_cast<T *>(p.y.p) + tw * p.y.st + v.b * p.y.sb + ch;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          float out[CPT];
#pragma unroll
          for (int j = 0; j < CPT; ++j) {
            if (on) h[j] = step(em1[s][j], h[j], in[s][j]);
            out[j] = tw + s < len ? h[j] : 0.f;
          }
          if (tw + s < p.T) store_raw(y, out, live, words >> 3 & 1);
          y += p.y.st;
        }
      }
    }
    if (rank == 0 && warp == 0) {
#pragma unroll
      for (int j = 0; j < CPT; ++j)
        if (j < live) {
          if (AGG) agg[(int64_t)v.seg * p.B * p.H + row + j] = make_float2(whole.p[j], whole.e[j]);
          else if (p.h_n && v.seg == cut.nseg - 1) p.h_n[row + j] = carry[j];
        }
    }
  }
  if (cs > 1) tc::cluster_sync();  // no block leaves while a peer may still write to it
}

// IT: the saved inputs' type, T: the gradients'
template <typename IT, typename T>
__global__ void linrec_bwd_kernel(LinrecBwd p, float *partial, int *err) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= (int64_t)p.B * p.H) return;
  const int b = (int)(id / p.H), h = (int)(id % p.H), nb = ceil_div(p.H, BLOCK8);
  const int len = row_length(p.lengths, b, p.T, err);
  const float k2 = decay_rate2(p.lambda[h], p.c), k = k2 * (1.f / LOG2E);
  float come = p.dh_n ? p.dh_n[id] : 0.f, sum = 0.f;
  float hp[CHUNK];
  for (int c = (p.T - 1) / CHUNK; c >= 0; --c) {
    const int t0 = c * CHUNK, n = min(CHUNK, p.T - t0);
    float s = p.states[(int64_t)c * p.B * p.H + id];
    for (int j = 0; j < n && t0 + j < len; ++j) {
      const int t = t0 + j;
      const int64_t er = t * p.et + b * p.eb;
      float em1, in;
      hp[j] = s;
      gate(value<IT>(p.x, t, b, h, er, nb), value<IT>(p.r, t, b, h, er, nb),
           value<IT>(p.i, t, b, h, er, nb), k2, em1, in);
      s = step(em1, s, in);
    }
    for (int j = n - 1; j >= 0; --j) {
      const int t = t0 + j;
      const int64_t er = t * p.et + b * p.eb;
      Grad d{0.f, 0.f, 0.f, 0.f};
      if (t < len) {
        const float x = value<IT>(p.x, t, b, h, er, nb);
        const Sig v = sigmoids(value<IT>(p.r, t, b, h, er, nb), value<IT>(p.i, t, b, h, er, nb));
        const float em1 = ex2m1(k2 * v.s);
        const float e = come + value<T>(p.dy, t, b, h, 0, 0);
        d = grads(x, v, em1, k, hp[j], e);
        come = step(em1, e, 0.f);
        sum += d.dlog_s;
      }
      if (p.dx.p) static_cast<T *>(p.dx.p)[t * p.dx.st + b * p.dx.sb + h] = from_f<T>(d.dx);
      if (p.dr.p) static_cast<T *>(p.dr.p)[t * p.dr.st + b * p.dr.sb + h] = from_f<T>(d.dr);
      if (p.di.p) static_cast<T *>(p.di.p)[t * p.di.st + b * p.di.sb + h] = from_f<T>(d.di);
    }
  }
  if (p.dh0) p.dh0[id] = come;
  partial[id] = sum;
}

// dlambda[h] = -c sigmoid(lambda) * the sum of the rows' partial sums, in row order
__global__ void linrec_dlambda_kernel(const float *partial, int rows, int H, const float *lambda,
                                      float c, float *dlambda) {
  const int h = blockIdx.x * blockDim.x + threadIdx.x;
  if (h >= H) return;
  float s = 0.f;
  for (int b = 0; b < rows; ++b) s += partial[(int64_t)b * H + h];
  dlambda[h] = -c * s / (1.f + expf(-lambda[h]));
}

template <typename T>
__global__ void linrec_step_kernel(int B, int H, const T *x, int64_t ldx, const T *r, int64_t ldr,
                                   const T *i, int64_t ldi, const float *lambda, float c,
                                   float *state, int slots, const int32_t *slot, T *y,
                                   int64_t ldy, int *err) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= (int64_t)B * H) return;
  const int64_t b = id / H;
  const int h = (int)(id % H);
  int64_t row = slot ? slot[b] : b;
  if (row < -1 || row >= slots) {
    atomicCAS(err, (int)DEV_OK, (int)DEV_SLOTS);
    row = -1;
  }
  float out = 0.f;
  if (row >= 0) {
    float em1, in;
    gate(to_f(x[b * ldx + h]), to_f(r[b * ldr + h]), to_f(i[b * ldi + h]),
         decay_rate2(lambda[h], c), em1, in);
    out = state[row * H + h] = step(em1, state[row * H + h], in);
  }
  y[b * ldy + h] = from_f<T>(out);
}

}  // namespace

namespace {

// A [T, B, H] tensor as a 3-D tensor map (channel, row, step) of boxes of one
// tile; false where TMA cannot address it (16-byte rules) or it is no gain.
bool tile_map(CUtensorMap *map, const SeqIn &v, int bytes, int cw, int T, int B, int H) {
  return tc_map_3d(map, v.p, bytes, H, B, T, v.sb, v.st, cw, 1, CHUNK);
}

bool word_aligned(const void *p, int64_t st, int64_t sb, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 && st * bytes % 4 == 0 && sb * bytes % 4 == 0;
}

struct Plan {
  Cut cut;
  int cs;
};

// How a recurrence over `tiles` tiles of B rows and `groups` groups is cut.
Plan plan_cut(int tiles, int B, int groups, int nsm, int per_sm) {
  Plan pl;
  const int64_t slots = (int64_t)nsm * per_sm, rows = (int64_t)B * groups;
  pl.cut.groups = groups;
  pl.cut.tiles = tiles;
  pl.cs = 1;
  pl.cut.nseg = 1;
  while (pl.cs < MAXCS && rows * pl.cs * 2 <= slots && pl.cs < tiles) pl.cs *= 2;
  pl.cut.tps = ceil_div(tiles, pl.cut.nseg);
  pl.cut.units = (int)(rows * pl.cut.nseg);
  return pl;
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*fn)(KArgs...), int grid, int cs, size_t smem, cudaStream_t s,
                   Args... args) {
  cudaError_t e =
      cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cs;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = cs > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <typename T>
cudaError_t fwd(const LinrecFwd &p, float2 *agg, int *err, int nsm, bool vec, cudaStream_t s,
                int *launches) {
  constexpr int CW = Shape<T>::CW;
  const Plan pl = plan_cut(ceil_div(p.T, CHUNK), p.B, ceil_div(p.H, CW), nsm, 3);
  CUtensorMap m[3];
  const SeqIn *in[3] = {&p.x, &p.r, &p.i};
  bool tma = vec;
  int words = word_aligned(p.y.p, p.y.st, p.y.sb, sizeof(T)) << 3;
  for (int k = 0; k < 3; ++k) {
    tma = tma && tile_map(&m[k], *in[k], sizeof(T), CW, p.T, p.B, p.H);
    words |= word_aligned(in[k]->p, in[k]->st, in[k]->sb, sizeof(T)) << k;
  }
  const size_t smem = sizeof(FwdSmem) + (tma ? FWD_STAGES * 3 * TILE_BYTES : 0);
  const int grid = (int)std::min<int64_t>((int64_t)pl.cut.units * pl.cs, (int64_t)nsm * 3 / pl.cs * pl.cs);
  ++*launches;
  if (tma)
    return launch(linrec_fwd_kernel<T, true, false>, grid, pl.cs, smem, s, m[0], m[1], m[2], p,
                  pl.cut, agg, words, err);
  return launch(linrec_fwd_kernel<T, false, false>, grid, pl.cs, smem, s, m[0], m[1], m[2], p,
                pl.cut, agg, words, err);
}

}  // namespace

size_t linrec_fwd_workspace(const LinrecFwd &, int) { return 0; }

cudaError_t launch_linrec_fwd(const LinrecFwd &p, void *ws, int *err, int nsm, bool vec,
                              cudaStream_t s, int *launches) {
  return p.dtype == RCU_BF16
             ? fwd<bf16>(p, static_cast<float2 *>(ws), err, nsm, vec, s, launches)
             : fwd<float>(p, static_cast<float2 *>(ws), err, nsm, vec, s, launches);
}

size_t linrec_bwd_workspace(const LinrecBwd &p, int) { return (size_t)p.B * p.H * 4; }

cudaError_t launch_linrec_bwd(const LinrecBwd &p, void *ws, int *err, int, bool, cudaStream_t s,
                              int *launches) {
  const unsigned grid = (unsigned)(((int64_t)p.B * p.H + 127) / 128);
  float *partial = static_cast<float *>(ws);
  const bool q8 = p.saved == RCU_I8;
  if (p.dtype == RCU_BF16) {
    if (q8) linrec_bwd_kernel<int8_t, bf16><<<grid, 128, 0, s>>>(p, partial, err);
    else linrec_bwd_kernel<bf16, bf16><<<grid, 128, 0, s>>>(p, partial, err);
  } else {
    if (q8) linrec_bwd_kernel<int8_t, float><<<grid, 128, 0, s>>>(p, partial, err);
    else linrec_bwd_kernel<float, float><<<grid, 128, 0, s>>>(p, partial, err);
  }
  ++*launches;
  if (p.dlambda) {
    linrec_dlambda_kernel<<<ceil_div(p.H, 128), 128, 0, s>>>(partial, p.B, p.H, p.lambda, p.c,
                                                             p.dlambda);
    ++*launches;
  }
  return cudaGetLastError();
}

cudaError_t launch_linrec_step(int dtype, int B, int H, const void *x, int64_t ldx, const void *r,
                               int64_t ldr, const void *i, int64_t ldi, const float *lambda,
                               float c, float *state, int slots, const int32_t *slot, void *y,
                               int64_t ldy, int *err, bool, cudaStream_t s, int *launches) {
  const unsigned grid = (unsigned)(((int64_t)B * H + 127) / 128);
  if (dtype == RCU_BF16)
    linrec_step_kernel<bf16><<<grid, 128, 0, s>>>(B, H, (const bf16 *)x, ldx, (const bf16 *)r, ldr,
                                                  (const bf16 *)i, ldi, lambda, c, state, slots,
                                                  slot, (bf16 *)y, ldy, err);
  else
    linrec_step_kernel<float><<<grid, 128, 0, s>>>(B, H, (const float *)x, ldx, (const float *)r,
                                                   ldr, (const float *)i, ldi, lambda, c, state,
                                                   slots, slot, (float *)y, ldy, err);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace rcu
