// Gated linear recurrence, one step of many requests: states in a table of
// slots, updated in place.
//
// Bound by latency at serving sizes (a launch and two dependent reads, slot and
// state), by memory above: 16 (bf16) or 24 bytes (fp32) an element.  A channel's
// constants cost more than a step, so a thread keeps VEC channels and takes
// several requests; their reads are in flight together.
// Measured, bf16 B=256 H=1024: 6.5 us with a cold cache, 14.6 us from call to call,
// which is the host's.
#include "linrec_tile.cuh"

namespace rcu {
namespace {

using namespace linrec;

constexpr int NT = 128, ROWS = 4;  // requests a thread reads together

struct StepArgs {
  int B, H, slots, per;  // per: requests of a thread
  const void *x, *r, *i;
  int64_t ldx, ldr, ldi;
  const float *lambda;
  float c;
  float *state;
  const int32_t *slot;
  void *y;
  int64_t ldy;
};

template <int VEC>
struct alignas(VEC * 4) Floats {
  float v[VEC];
};
template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Word {
  T v[VEC];
};

template <typename T, int VEC>
__global__ void __launch_bounds__(NT) linrec_step_kernel(const StepArgs a, int *err) {
  constexpr int PAIRS = (VEC + 1) / 2;
  const int h = (blockIdx.x * NT + threadIdx.x) * VEC;
  if (h >= a.H) return;
  const int64_t b0 = (int64_t)blockIdx.y * a.per, b1 = min(b0 + a.per, (int64_t)a.B);
  float k2[2 * PAIRS], top[2 * PAIRS];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    k2[j] = decay_rate2(a.lambda[h + j], a.c);
    top[j] = limits(k2[j]).top;
  }
  if (VEC == 1) k2[1] = k2[0], top[1] = top[0];
  for (int64_t b = b0; b < b1; b += ROWS) {
    Word<T, VEC> x[ROWS], r[ROWS], i[ROWS];
    Floats<VEC> s[ROWS];
    int64_t row[ROWS];
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      row[q] = -1;
      if (b + q >= b1) continue;
      row[q] = a.slot ? a.slot[b + q] : b + q;
      if (row[q] < -1 || row[q] >= a.slots) {
        atomicCAS(err, (int)DEV_OK, (int)DEV_SLOTS);
        row[q] = -1;
      }
    }
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      if (row[q] < 0) continue;
      x[q] = *reinterpret_cast<const Word<T, VEC> *>(static_cast<const T *>(a.x) + (b + q) * a.ldx + h);
      r[q] = *reinterpret_cast<const Word<T, VEC> *>(static_cast<const T *>(a.r) + (b + q) * a.ldr + h);
      i[q] = *reinterpret_cast<const Word<T, VEC> *>(static_cast<const T *>(a.i) + (b + q) * a.ldi + h);
      s[q] = *reinterpret_cast<const Floats<VEC> *>(a.state + row[q] * a.H + h);
    }
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      if (b + q >= b1) continue;
      Word<T, VEC> y;
      if (row[q] >= 0) {
        F2 vx[PAIRS], vr[PAIRS], vi[PAIRS], k[PAIRS], em1[PAIRS], nb[PAIRS], ns[PAIRS], ng[PAIRS];
        auto at = [&](const Word<T, VEC> &w, int j) { return to_f(w.v[j < VEC ? j : 0]); };
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
          vx[j] = f2(at(x[q], 2 * j), at(x[q], 2 * j + 1));
          vr[j] = exponent_of(
              f2(min_nan(at(r[q], 2 * j), top[2 * j]), min_nan(at(r[q], 2 * j + 1), top[2 * j + 1])));
          vi[j] = exponent_of(f2(at(i[q], 2 * j), at(i[q], 2 * j + 1)));
          const F2 one_x[1] = {vx[j]}, one_r[1] = {vr[j]}, one_i[1] = {vi[j]};
          gates_n<false, false, 1>(one_x, one_r, one_i, f2(k2[2 * j], k2[2 * j + 1]), em1 + j,
                                   nb + j, ns + j, ng + j);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float m = j % 2 ? hi(em1[j / 2]) : lo(em1[j / 2]);
          const float in = j % 2 ? -hi(nb[j / 2]) : -lo(nb[j / 2]);
          s[q].v[j] = step(m, s[q].v[j], in);
          y.v[j] = from_f<T>(s[q].v[j]);
        }
        *reinterpret_cast<Floats<VEC> *>(a.state + row[q] * a.H + h) = s[q];
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) y.v[j] = from_f<T>(0.f);
      }
      *reinterpret_cast<Word<T, VEC> *>(static_cast<T *>(a.y) + (b + q) * a.ldy + h) = y;
    }
  }
}

template <typename T, int VEC>
cudaError_t run(StepArgs a, int nsm, int *err, cudaStream_t s) {
  const int across = ceil_div(ceil_div(a.H, VEC), NT);
  // as many requests a thread as leave eight blocks an SM, 32 at most
  a.per = (int)std::min<int64_t>(std::max<int64_t>((int64_t)a.B * across / (8 * nsm), 1), 32);
  a.per = std::max(a.per, ceil_div(a.B, 65535));
  linrec_step_kernel<T, VEC><<<dim3(across, ceil_div(a.B, a.per)), NT, 0, s>>>(a, err);
  return cudaGetLastError();
}

template <typename T>
cudaError_t step_of(const StepArgs &a, int nsm, int *err, bool vec, cudaStream_t s) {
  auto fits = [](const void *p, int64_t ld, int size) {
    return reinterpret_cast<uintptr_t>(p) % (4 * size) == 0 && ld % 4 == 0;
  };
  const int size = sizeof(T);
  if (vec && a.H % 4 == 0 && fits(a.x, a.ldx, size) && fits(a.r, a.ldr, size) &&
      fits(a.i, a.ldi, size) && fits(a.y, a.ldy, size) && fits(a.state, a.H, 4))
    return run<T, 4>(a, nsm, err, s);
  return run<T, 1>(a, nsm, err, s);
}

}  // namespace

cudaError_t launch_linrec_step(int dtype, int B, int H, const void *x, int64_t ldx, const void *r,
                               int64_t ldr, const void *i, int64_t ldi, const float *lambda,
                               float c, float *state, int slots, const int32_t *slot, void *y,
                               int64_t ldy, int *err, int nsm, bool vec, cudaStream_t s,
                               int *launches) {
  const StepArgs a{B, H, slots, 1, x, r, i, ldx, ldr, ldi, lambda, c, state, slot, y, ldy};
  ++*launches;
  return dtype == RCU_BF16 ? step_of<bf16>(a, nsm, err, vec, s) : step_of<float>(a, nsm, err, vec, s);
}

}  // namespace rcu
