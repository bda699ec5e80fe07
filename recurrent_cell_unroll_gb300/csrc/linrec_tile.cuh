// What the gated linear recurrence's forward (linrec_fwd.cu) and backward
// (linrec_bwd.cu) kernels share: how the work is cut into tiles, units and
// clusters, and how a tile's values and the affine maps of its steps move.
//
// A block of NW warps takes a tile of NW * S steps x CW channels of one batch
// row (NW, S: the kernel's own); CW values of the tensors' type are 128 bytes, so
// that a step of a tile is one full line.  Warp w has the steps [w * S, w * S + S),
// lane l the CPT channels from l * CPT.  A step is h -> a h + b, and steps compose to affine
// maps h -> P h + E: each warp reduces its steps to a map, the maps are chained
// in order, and the warp then runs its steps from the state that reaches it.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "linrec_math.cuh"
#include "per_device.h"
#include "rcu.h"
#include "seq.h"
#include "tc.h"
#include "tc_common.cuh"

namespace rcu {
namespace linrec {

using bf16 = __nv_bfloat16;

constexpr int CHUNK = RCU_LINREC_CHUNK;
constexpr int BLOCK8 = RCU_ACT8_BLOCK;
constexpr uint64_t WAIT_NS = 2000000000ull;  // bound on any wait for a copy

template <typename T>
struct Shape {
  static constexpr int CPT = 4 / (int)sizeof(T), CW = 32 * CPT;
};

// The length of row b, clamped to [0, T]; an outside value is reported.
__device__ __forceinline__ int row_length(const int32_t *lengths, int b, int T, int *err) {
  if (!lengths) return T;
  const int len = lengths[b];
  if (len < 0 || len > T) atomicCAS(err, (int)DEV_OK, (int)DEV_LENGTHS);
  return min(max(len, 0), T);
}

// Unit u = (segment of time, batch row, group of CW channels), the groups
// fastest: blocks that run together then read neighbouring channels of the same
// steps.  A cluster takes a unit, its blocks consecutive tiles of it.
//
// Or the blocks have equal shares of the tiles: those of a group's rows, one behind
// another, are cut into pieces of `share`, no fewer than a row has, so that a cut
// row has two blocks.  A block takes its pieces of rows backwards: the row that its
// share ends in first, and last the one that the block before it has begun, whose
// carry is there by then, being the first that block made.
struct Cut {
  int groups, units, tiles, tps, nseg, share;  // tps: tiles of a segment; share: 0 or as above
};
struct Unit {
  int seg, b, c0, first, last;  // tiles [first, last)
};
// The next tile to be copied, and of which unit
struct Next {
  int u, tile, end, len, issued;  // end: of its tiles, forwards
  Unit v;
};
// This block's share [lo, hi) of its group's tiles, counted as they are processed
struct Share {
  int lo, hi;
};
__device__ __forceinline__ Share share_of(const Cut &cut, int B) {
  const int lo = (int)blockIdx.x / cut.groups * cut.share;
  return {lo, min(lo + cut.share, B * cut.tiles)};
}
// How a kernel goes through them: clusters over whole units (or a unit's segments),
// the first launch that reduces the segments to their maps, blocks with shares.
enum Mode { UNITS, MAPS, SHARES };

template <Mode M>
__device__ __forceinline__ int count_units(const Cut &cut, int B) {
  if (M != SHARES) return cut.units;
  const Share s = share_of(cut, B);
  return (s.hi - 1) / cut.tiles - s.lo / cut.tiles + 1;
}
// BACK: the tiles are processed from the last to the first.
template <Mode M, bool BACK>
__device__ __forceinline__ Unit unit_of(const Cut &cut, int B, int u, int cw) {
  Unit v;
  if (M == SHARES) {
    const Share s = share_of(cut, B);
    v.seg = 0;
    v.b = (s.hi - 1) / cut.tiles - u;
    v.c0 = (int)blockIdx.x % cut.groups * cw;
    const int from = max(s.lo - v.b * cut.tiles, 0), to = min(s.hi - v.b * cut.tiles, cut.tiles);
    v.first = BACK ? cut.tiles - to : from;
    v.last = BACK ? cut.tiles - from : to;
    return v;
  }
  if (BACK && M == MAPS) u += B * cut.groups;  // not of the first segment
  v.c0 = u % cut.groups * cw;
  const int q = u / cut.groups;
  v.b = q % B;
  v.seg = q / B;
  v.first = v.seg * cut.tps;
  v.last = min(cut.tiles, v.first + cut.tps);
  return v;
}

// A wait has run out, and results with it.  It is reported in place of a length or slot
// that was out of range, which they would have outlived.
__device__ __forceinline__ void report_timeout(int *err) {
  atomicExch(err, (int)DEV_TIMEOUT);
}
// Whether a wait is to end unfinished: past its limit, or as another one ran out.
__device__ __forceinline__ bool give_up(uint64_t deadline, int *err, volatile int *abort) {
  if (!*abort && ld_volatile_int(err) != (int)DEV_TIMEOUT) {
    if (globaltimer_ns() <= deadline) return false;
    report_timeout(err);
  }
  *abort = 1;
  return true;
}
// Until a tile's copies have landed (whatever has been reported elsewhere: they are this
// block's own).
__device__ __forceinline__ void wait_copy(uint64_t *bar, uint32_t parity, int *err,
                                          volatile int *abort) {
  if (tc::mbar_try_wait(bar, parity)) return;
  const uint64_t deadline = globaltimer_ns() + WAIT_NS;
  uint32_t spins = 0;
  while (!tc::mbar_try_wait(bar, parity)) {
    if ((++spins & 255u) == 0) {
      if (*abort) return;
      if (globaltimer_ns() > deadline) {
        report_timeout(err);
        *abort = 1;
        return;
      }
    }
  }
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// A warp's S steps from shared memory (written by all its lanes, a step 128
// bytes) to the tensor: rows and channels past its ends are left out.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int x, int y,
                                             int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(tc::smem_u32(src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// every committed store of this thread has read its source / has been written
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void store_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- tiles that TMA cannot address (rows not 16-byte aligned)
//
// Each warp copies the rows of its own steps by 16-byte asynchronous copies: the
// aligned words that hold a row's bytes, so that a row keeps its offset (0 to 15)
// in shared memory.  The last word is cut at the row's end; the first one's
// leading bytes are the tensor's or its allocation's, which starts on a word.

template <typename IT, int CPT>
struct Loose {
  static constexpr int BYTES = 32 * CPT * (int)sizeof(IT), PITCH = BYTES + 16;
};

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// `rows` rows of K tensors that lie alike, from `pos` bytes behind each `base` and
// `pitch` bytes apart, `bytes` of each; to `dst`, a tensor `apart` from the one before.
// The loop stays a loop: unrolled, the kernel outgrew the instruction cache.
template <typename IT, int CPT, int K>
__device__ __forceinline__ void copy_rows(uint8_t *dst, int apart, const void *const (&base)[K],
                                          int64_t pos, int64_t pitch, int rows, int bytes) {
  typedef Loose<IT, CPT> L;
  constexpr int WORDS = L::PITCH / 16, TOGETHER = 32 / WORDS;  // of a row; rows at once
  const int lane = threadIdx.x % 32, at = lane % WORDS * 16;
  const int first = lane / WORDS < TOGETHER ? lane / WORDS : rows;
  const uint32_t low = (uint32_t)reinterpret_cast<uintptr_t>(base[0]);
  uint32_t to = tc::smem_u32(dst) + first * L::PITCH + at;
  pos += first * pitch;
#pragma unroll 1
  for (int s = first; s < rows; s += TOGETHER, pos += TOGETHER * pitch, to += TOGETHER * L::PITCH) {
    const int off = (int)((low + (uint32_t)pos) & 15), left = off + bytes - at;
    if (left > 0) {
      const int64_t from = pos + (at - off);
      const int size = min(left, 16);
#pragma unroll
      for (int k = 0; k < K; ++k)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + k * apart),
                     "l"(static_cast<const uint8_t *>(base[k]) + from), "r"(size)
                     : "memory");
    }
  }
}

__device__ __forceinline__ bool alike(const void *a, const void *b) {
  return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

// A lane's CPT values of S rows of K such copies (`apart` bytes from one to the next), whose
// rows start at off[k] of their words and move on by more[k].  Copies that agree in
// both, as tensors of one layout do, share the arithmetic: `same`.
template <typename IT, int CPT, int K, int S>
__device__ __forceinline__ void loose_rows(const uint8_t *tile, int apart, const uint32_t (&off)[K],
                                           const uint32_t (&more)[K], bool same,
                                           uint32_t (&raw)[K][S]) {
  typedef Loose<IT, CPT> L;
  constexpr int N = CPT * (int)sizeof(IT);
  const uint32_t base = tc::smem_u32(tile) + threadIdx.x % 32 * N;
  auto get = [&](int k, int s, uint32_t word, uint32_t shift) {
    const uint32_t at = word + (s * L::PITCH + k * apart);
    uint32_t w0, w1;
    if (sizeof(IT) == 4) {
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(raw[k][s]) : "r"(at) : "memory");
    } else {  // the two words that hold them, shifted together
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w0) : "r"(at) : "memory");
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w1) : "r"(at + 4) : "memory");
      raw[k][s] = __funnelshift_r(w0, w1, shift) & (N == 4 ? ~0u : (1u << (8 * (N & 3))) - 1);
    }
  };
  auto row = [&](int k, int s, uint32_t o, int n) {
    const uint32_t word = (base + o) & ~3u, shift = (base + o) * 8;
#pragma unroll
    for (int m = 0; m < n; ++m) get(k + m, s, word, shift);
  };
  if (same) {
    uint32_t o = off[0];
#pragma unroll
    for (int s = 0; s < S; ++s, o = (o + more[0]) & 15) row(0, s, o, K);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      uint32_t o = off[k];
#pragma unroll
      for (int s = 0; s < S; ++s, o = (o + more[k]) & 15) row(k, s, o, 1);
    }
  }
}

// ---- one lane's values of a step, without a tile

// A lane's values of a step from global memory (`word`: as one access)
template <typename IT, int CPT>
__device__ __forceinline__ uint32_t global_raw(const IT *p, int live, bool word) {
  constexpr int B = CPT * (int)sizeof(IT);
  if (B == 4 && word && live == CPT) return __ldg(reinterpret_cast<const uint32_t *>(p));
  if (B == 2 && word && live == CPT) return __ldg(reinterpret_cast<const unsigned short *>(p));
  uint32_t v = 0;
  if (sizeof(IT) == 4) {
    if (live > 0) v = __ldg(reinterpret_cast<const uint32_t *>(p));
  } else if (sizeof(IT) == 2) {
    const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
    if (live > 0) v = __ldg(q);
    if (CPT > 1 && live > 1) v |= (uint32_t)__ldg(q + 1) << 16;
  } else {
    const unsigned char *q = reinterpret_cast<const unsigned char *>(p);
    if (live > 0) v = __ldg(q);
    if (CPT > 1 && live > 1) v |= (uint32_t)__ldg(q + 1) << 8;
  }
  return v;
}

// ---- one lane's values of a step, as they go out

__device__ __forceinline__ void store_raw(float *p, float v, int live, bool) {
  if (live > 0) *p = v;
}
__device__ __forceinline__ void store_raw(bf16 *p, F2 v, int live, bool word) {
  const __nv_bfloat162 o = __floats2bfloat162_rn(lo(v), hi(v));
  if (live > 1 && word) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = o;
  } else {
    if (live > 0) p[0] = o.x;
    if (live > 1) p[1] = o.y;
  }
}
// channels past the row's end, or a pair that is not one word
__device__ __forceinline__ void store_raw(float *p, float v, int live) {
  if (live > 0) *p = v;
}
__device__ __forceinline__ void store_raw(bf16 *p, F2 v, int live) {
  const __nv_bfloat162 o = __floats2bfloat162_rn(lo(v), hi(v));
  if (live > 0) p[0] = o.x;
  if (live > 1) p[1] = o.y;
}
// a whole word
__device__ __forceinline__ void store_word(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_word(bf16 *p, F2 v) {
  *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(lo(v), hi(v));
}
// a lane's word of a step, for shared memory
__device__ __forceinline__ uint32_t pack(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t pack(F2 v) {
  const __nv_bfloat162 o = __floats2bfloat162_rn(lo(v), hi(v));
  return *reinterpret_cast<const uint32_t *>(&o);
}
__device__ __forceinline__ F2 bf16_pair(uint32_t v) {
  return f2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// ---- a lane's channels: two in a pair (bf16), or one (fp32)

template <typename T>
struct Lane;
template <>
struct Lane<float> {
  typedef float V;
};
template <>
struct Lane<bf16> {
  typedef F2 V;
};
__device__ __forceinline__ float fma_v(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ F2 fma_v(F2 a, F2 b, F2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float add_v(float a, float b) { return a + b; }
__device__ __forceinline__ F2 add_v(F2 a, F2 b) { return add2(a, b); }
__device__ __forceinline__ float mul_v(float a, float b) { return a * b; }
__device__ __forceinline__ F2 mul_v(F2 a, F2 b) { return mul2(a, b); }
__device__ __forceinline__ float neg_v(float a) { return -a; }
__device__ __forceinline__ F2 neg_v(F2 a) { return f2(-lo(a), -hi(a)); }
__device__ __forceinline__ void set(float &v, float c) { v = c; }
__device__ __forceinline__ void set(F2 &v, float c) { v = f2(c); }

// from and to fp32 rows [.., H]
__device__ __forceinline__ void load_v(const float *p, int live, float &v) {
  v = live > 0 ? p[0] : 0.f;
}
__device__ __forceinline__ void load_v(const float *p, int live, F2 &v) {
  v = f2(live > 0 ? p[0] : 0.f, live > 1 ? p[1] : 0.f);
}
__device__ __forceinline__ void store_v(float *p, float v, int live) {
  if (live > 0) p[0] = v;
}
__device__ __forceinline__ void store_v(float *p, F2 v, int live) {
  if (live > 0) p[0] = lo(v);
  if (live > 1) p[1] = hi(v);
}

// the decay rates of the lane's channels (0 for one past the row's end)
__device__ __forceinline__ void rate(const float *lambda, float c, int live, float &k2) {
  k2 = live > 0 ? decay_rate2(lambda[0], c) : 0.f;
}
__device__ __forceinline__ void rate(const float *lambda, float c, int live, F2 &k2) {
  k2 = f2(live > 0 ? decay_rate2(lambda[0], c) : 0.f, live > 1 ? decay_rate2(lambda[1], c) : 0.f);
}

// ---- affine maps h -> P h + E

template <typename V>
struct Aff {
  V p, e;
};
template <typename V>
__device__ __forceinline__ Aff<V> identity() {
  Aff<V> a;
  set(a.p, 1.f);
  set(a.e, 0.f);
  return a;
}
template <typename V>
__device__ __forceinline__ V apply(const Aff<V> &a, V h) {
  return fma_v(a.p, h, a.e);
}
// first a, then b
template <typename V>
__device__ __forceinline__ Aff<V> then(const Aff<V> &a, const Aff<V> &b) {
  return {mul_v(a.p, b.p), fma_v(b.p, a.e, b.e)};
}
// as a lane's 8 or 16 bytes of shared memory
template <typename V>
struct Slot;
template <>
struct Slot<float> {
  typedef float2 type;
};
template <>
struct Slot<F2> {
  typedef float4 type;
};
__device__ __forceinline__ void put(float2 *at, const Aff<float> &a) {
  *at = make_float2(a.p, a.e);
}
__device__ __forceinline__ void put(float4 *at, const Aff<F2> &a) {
  *at = make_float4(lo(a.p), hi(a.p), lo(a.e), hi(a.e));
}
__device__ __forceinline__ Aff<float> get(const float2 *at) {
  const float2 v = *at;
  return {v.x, v.y};
}
__device__ __forceinline__ Aff<F2> get(const float4 *at) {
  const float4 v = *at;
  return {f2(v.x, v.y), f2(v.z, v.w)};
}
// The same into block `rank` of the cluster (its copy of *at), counted there as
// bytes that its barrier `bar` (its copy) expects: the barrier's phase carries
// the data's visibility, so that no fence waits for the outputs' plain stores.
__device__ __forceinline__ void put_peer(float2 *at, uint64_t *bar, int rank, const Aff<float> &a) {
  const uint32_t to = tc::mapa_shared(tc::smem_u32(at), rank);
  const uint32_t b = tc::mapa_shared(tc::smem_u32(bar), rank);
  tc::st_async_f32(to, a.p, b);
  tc::st_async_f32(to + 4, a.e, b);
}
__device__ __forceinline__ void put_peer(float4 *at, uint64_t *bar, int rank, const Aff<F2> &a) {
  tc::st_async_v4(tc::mapa_shared(tc::smem_u32(at), rank), lo(a.p), hi(a.p), lo(a.e), hi(a.e),
                  tc::mapa_shared(tc::smem_u32(bar), rank));
}

// Until the cluster's blocks have sent a round's maps.  An error that is reported
// and stepped over (a length out of range) ends no wait; one that ran out does.
__device__ __forceinline__ void wait_round(uint64_t *bar, uint32_t parity, int *err,
                                           volatile int *abort) {
  if (tc::mbar_try_wait_cluster(bar, parity)) return;
  const uint64_t deadline = globaltimer_ns() + WAIT_NS;
  for (uint32_t spins = 1; !tc::mbar_try_wait_cluster(bar, parity); ++spins)
    if ((spins & 255u) == 0 && give_up(deadline, err, abort)) return;
}

// ---- shares: the carry of a row that this block leaves to the next of its group.
// mem: [blocks] counts of lanes that have, zero before the launch, then [blocks][32]
// carries.  (Lane by lane: a warp's barrier cost the backward registers in its loop.)

constexpr size_t carry_flags(int blocks) { return ((size_t)blocks * 4 + 15) / 16 * 16; }

template <typename V>
__device__ __forceinline__ V *carry_at(void *mem, int block) {
  return reinterpret_cast<V *>(static_cast<uint8_t *>(mem) + carry_flags(gridDim.x)) + block * 32 +
         threadIdx.x % 32;
}
// by one warp
template <typename V>
__device__ __forceinline__ void leave_carry(void *mem, V carry) {
  *carry_at<V>(mem, blockIdx.x) = carry;
  red_release_gpu_add(static_cast<unsigned *>(mem) + blockIdx.x, 1);
}
// by each warp; that block runs (a cooperative launch) and left it before all its other work
template <typename V>
__device__ __forceinline__ V take_carry(void *mem, int from, int *err, volatile int *abort) {
  if (!RCU_DCHECK(from >= 0 && from < (int)blockIdx.x, err)) return V{};
  const unsigned *lanes = static_cast<const unsigned *>(mem) + from;
  if (ld_acquire_gpu(lanes) != 32) {
    const uint64_t deadline = globaltimer_ns() + WAIT_NS;
    while (ld_acquire_gpu(lanes) != 32 && !give_up(deadline, err, abort)) __nanosleep(100);
  }
  return __ldcg(carry_at<V>(mem, from));
}

// ---- segments: the maps that a first launch leaves, [segment][row][group][lane]

template <typename V>
__device__ __forceinline__ typename Slot<V>::type *segment_map(void *maps, const Cut &cut, int B,
                                                               int seg, const Unit &v, int cw) {
  return static_cast<typename Slot<V>::type *>(maps) +
         (((int64_t)seg * B + v.b) * cut.groups + v.c0 / cw) * 32 + threadIdx.x % 32;
}
// The map of segments [from, to) in steps of `by` (forwards or backwards), the
// block's NWARP warps taking a share each: all its threads call this.
template <typename V, int NWARP>
__device__ __forceinline__ Aff<V> chain_segments(void *maps, const Cut &cut, int B, const Unit &v,
                                                 int cw, int from, int to, int by,
                                                 typename Slot<V>::type (*part)[32], int *err) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int n = (to - from) * by, each = ceil_div(n, NWARP);
  Aff<V> a = identity<V>();
#pragma unroll 8
  for (int q = warp * each; q < min(n, (warp + 1) * each); ++q)
    if (RCU_DCHECK(from + q * by >= 0 && from + q * by < cut.nseg && v.b < B, err))
      a = then(a, get(segment_map<V>(maps, cut, B, from + q * by, v, cw)));
  __syncthreads();
  put(&part[warp][lane], a);
  __syncthreads();
  a = identity<V>();
#pragma unroll
  for (int w = 0; w < NWARP; ++w) a = then(a, get(&part[w][lane]));
  __syncthreads();
  return a;
}

// ---- host side

inline bool word_aligned(const void *p, int64_t st, int64_t sb, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 && st * bytes % 4 == 0 && sb * bytes % 4 == 0;
}

struct Plan {
  Cut cut;
  int cs, grid;
};

// How many clusters of each size a kernel can have resident (size 1: blocks), on the
// current device; resident() sets the kernel's limits there too.
struct Resident {
  static constexpr int MAX = 16;
  int clusters[MAX + 1] = {};
};
template <typename... KArgs>
int resident_blocks(void (*fn)(KArgs...), int threads, size_t smem) {
  int dev = 0, nsm = 0, blocks = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, fn, threads, smem);
  return std::max(1, blocks * nsm);
}
template <typename... KArgs>
Resident resident(void (*fn)(KArgs...), int threads, int max_cs, size_t smem0, size_t smem_per_cs) {
  Resident r;
  const size_t most = smem0 + max_cs * smem_per_cs;
  cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (max_cs > 8)
    cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  r.clusters[1] = resident_blocks(fn, threads, smem0 + smem_per_cs);
  for (int cs = 2; cs <= max_cs; ++cs) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at;
    cfg.gridDim = dim3(cs);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem0 + cs * smem_per_cs;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&r.clusters[cs], fn, &cfg) != cudaSuccess)
      r.clusters[cs] = 0;
  }
  cudaGetLastError();  // a size the GPU has no room for is no error of the call
  return r;
}

// Of a pass's kernels: over whole units, the first launch of segments, with shares.
struct Room {
  Resident units, maps;
  int shares;
};

// How the recurrence over `tiles` tiles of B rows x `groups` channel groups is
// cut: the cluster size that needs the fewest turns, a turn being one tile a
// block.  A larger cluster splits a sequence further, which pays where there
// are fewer rows than blocks (or a last, thin wave of them), and costs its
// blocks' exchange and their waiting for one another, some three tenths of a turn
// (backward from 8 bits, T=1000 B=32 H=1024: 145 us in whole rows, 159 in pairs,
// though 32 turns each; 32 rows of 65536 steps forward: 250 us with 12 blocks a
// row, 290 with 8).
//
// With more rows than blocks, but few for each, whole rows leave blocks idle in the
// last wave; equal shares of the tiles cost
// about a turn, the flags' clearing and a cooperative launch.
// bf16 H=1024 T=1000: backward B=24 113 -> 78 us, from 8 bits B=32 144 -> 117,
// forward B=29 65 -> 50.  (A row is never cut in three: the middle would wait for
// the first and the last for both.)
//
// With few rows, clusters leave most of the GPU idle: then the sequence is cut into
// segments that run as rows of their own, after a first launch (costing `map` of
// the second) has reduced each segment to its affine map.  One row of 65536 steps x
// 256 channels, bf16: forward 159 us in a cluster of 12, 57 us in segments;
// backward 389 and 82.
inline Plan plan_cut(int tiles, int B, int groups, const Resident &res, int blocks, double map) {
  Plan pl;
  const int64_t rows = (int64_t)B * groups;
  double best = 0;
  pl.cs = 1;
  for (int cs = 1; cs <= Resident::MAX && cs <= tiles; ++cs) {
    if (res.clusters[cs] < 1) continue;
    const double waves = (double)((rows + res.clusters[cs] - 1) / res.clusters[cs]);
    const double cost = waves * ceil_div(tiles, cs) * (cs > 1 ? 1.3 : 1.0);
    if (cs == 1 || cost < best) best = cost, pl.cs = cs;
  }
  pl.cut.nseg = 1;
  const int nseg = (int)std::min<int64_t>(res.clusters[1] / rows, tiles / 4);
  if (nseg > 1 && (1 + map) * ceil_div(tiles, nseg) + 6 < best)
    best = (1 + map) * ceil_div(tiles, nseg) + 6, pl.cut.nseg = nseg, pl.cs = 1;
  pl.cut.share = 0;
  const int each = blocks / groups;  // blocks of a group
  if (each > 0 && (int64_t)B * tiles < 1 << 30) {
    const int cut = std::max(tiles, ceil_div(B * tiles, each)), whole = ceil_div(B, each) * tiles;
    const int share = cut + 1 < whole ? cut : whole;
    if (share + (share == cut) <= best || share == best) {
      pl.cs = 1;
      pl.cut = Cut{groups, (int)rows, tiles, tiles, 1, share};
      pl.grid = ceil_div(B * tiles, share) * groups;
      return pl;
    }
  }
  pl.cut.groups = groups;
  pl.cut.tiles = tiles;
  pl.cut.tps = ceil_div(tiles, pl.cut.nseg);
  pl.cut.nseg = ceil_div(tiles, pl.cut.tps);
  pl.cut.units = (int)(rows * pl.cut.nseg);
  // a whole number of times the groups, where that many clusters fit: every
  // cluster then stays with its channels, whose constants it keeps
  int64_t clusters = std::min<int64_t>(pl.cut.units, res.clusters[pl.cs]);
  if (clusters < pl.cut.units && clusters >= 4 * groups) clusters -= clusters % groups;
  pl.grid = (int)clusters * pl.cs;
  return pl;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cut(void (*fn)(KArgs...), const Plan &pl, int threads, size_t smem,
                       cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(pl.grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  const bool waits = pl.cut.share && pl.cut.share % pl.cut.tiles;
  if (waits) {  // blocks wait for one another
    at.id = cudaLaunchAttributeCooperative;
    at.val.cooperative = 1;
  } else {
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = pl.cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
  }
  cfg.attrs = &at;
  cfg.numAttrs = pl.cs > 1 || waits ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// The short kernels' warps: `each` a group of channels, which they stay with from row to
// row; no more in all than the GPU has room for, as one block too many takes a wave of
// its own (bf16 T=11 B=188 H=1921, 31 groups: backward 176 us in 465 blocks, 128 in
// 450).  The last block's warps past each * groups have nothing to do.
struct Warps {
  int each, blocks;
};
inline Warps warps_of(int B, int groups, int room, int per_block) {
  const int each = std::max(1, std::min(B, room * per_block / groups));
  return {each, ceil_div(each * groups, per_block)};
}
// Whether they take at most `limit` steps a row of B rows of T steps, counting what warps
// without a row in the last turn could have taken.
inline bool steps_within(int T, int B, const Warps &w, int limit) {
  return (int64_t)T * ceil_div(B, w.each) * w.each <= (int64_t)limit * B;
}
// The forward kernel for short sequences of many rows (linrec_fwd_short.cu), and whether
// it is the faster one; resident_blocks: of the tiled kernel, vec: as of launch_linrec_fwd.
bool short_fwd_pays(const LinrecFwd &p, int resident_blocks, bool vec);
cudaError_t launch_short_fwd(const LinrecFwd &p, int *err, cudaStream_t s, int *launches);

}  // namespace linrec
}  // namespace rcu
