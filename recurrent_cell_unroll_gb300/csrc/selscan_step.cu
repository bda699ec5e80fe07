// Selective scan, one step of many requests: states in a table of slots, updated
// in place.  Bound by memory (8 bytes a state) at serving sizes, by latency below.
//
// A thread keeps 4 states of a channel, neighbouring threads the channel's others,
// and takes several requests one after another, since a channel's rates cost more than
// a step.  Reading four together is faster where the cache takes the states (10 us in
// the place of 21, bf16 B=256 H=2048 N=16), but where memory has to, with tables taken
// in rotation, 39 us in the place of 18 (67 MB): reads and writes then come in bursts
// from all over the table.  From Python a call takes some 17 us.
#include "selscan.cuh"

namespace rcu {
namespace {

using namespace selscan;

constexpr int NT = 128, V = 4;  // states of a thread

template <typename T, int LANES, bool WIDE>
__global__ void __launch_bounds__(NT) scan_step_kernel(const ScanStep a, int per, int *err) {
  const int l = threadIdx.x % LANES;
  const int64_t ch64 = (int64_t)blockIdx.x * (NT / LANES) + threadIdx.x / LANES;
  const bool live = ch64 < a.H;
  const int ch = live ? (int)ch64 : a.H - 1, n0 = l * V;  // lanes beyond join the sums only
  const int64_t b0 = (int64_t)blockIdx.y * per, b1 = min(b0 + per, (int64_t)a.B);
  float A2[V];
#pragma unroll
  for (int k = 0; k < V; ++k)
    A2[k] = n0 + k < a.N ? rate2(a.a_log[(int64_t)ch * a.N + n0 + k]) : 0.f;
  const float bias = a.dt_bias ? a.dt_bias[ch] : 0.f, skip = a.d ? a.d[ch] : 0.f;
  const bool states = n0 < a.N;  // this lane has some
  for (int64_t b = b0; b < b1; ++b) {
    int64_t slot = a.slot ? a.slot[b] : b;
    if (slot < -1 || slot >= a.slots) {
      atomicCAS(err, (int)DEV_OK, (int)DEV_SLOTS);
      slot = -1;
    }
    T *y = static_cast<T *>(a.y) + b * a.ldy + ch;
    if (slot < 0) {  // the same for the warp
      if (live && l == 0) *y = from_f<T>(0.f);
      continue;
    }
    float *state = a.state + (slot * a.H + ch) * a.N + n0;
    const T *bp = static_cast<const T *>(a.b) + b * a.ldb + n0, *cp = static_cast<const T *>(a.c) + b * a.ldc + n0;
    float h[V] = {}, s = 0.f;
    Word<T, V> bw, cw;
    if (WIDE) {
      if (states) {
        const float4 v = *reinterpret_cast<const float4 *>(state);
        h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
        bw = *reinterpret_cast<const Word<T, V> *>(bp);
        cw = *reinterpret_cast<const Word<T, V> *>(cp);
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (n0 + k < a.N) h[k] = state[k], bw.v[k] = bp[k], cw.v[k] = cp[k];
    }
    const float x = to_f(static_cast<const T *>(a.x)[b * a.ldx + ch]);
    const float delta = softplus(to_f(static_cast<const T *>(a.dt)[b * a.lddt + ch]) + bias), u = delta * x;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (WIDE ? states : n0 + k < a.N) {
        h[k] = fmaf(ex2(delta * A2[k]), h[k], u * to_f(bw.v[k]));
        s = fmaf(h[k], to_f(cw.v[k]), s);
      }
    if (live && states) {
      if (WIDE) {
        *reinterpret_cast<float4 *>(state) = make_float4(h[0], h[1], h[2], h[3]);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (n0 + k < a.N) state[k] = h[k];
      }
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (live && l == 0) {
      if (a.d) s = fmaf(skip, x, s);
      if (a.z) {
        const float z = to_f(static_cast<const T *>(a.z)[b * a.ldz + ch]);
        s *= z * sigmoid(z);
      }
      *y = from_f<T>(s);
    }
  }
}

template <typename T, int LANES, bool WIDE>
cudaError_t run(const ScanStep &a, int *err, int nsm, cudaStream_t s) {
  const int64_t across = ((int64_t)a.H * LANES + NT - 1) / NT;
  // as many requests a thread as leave twelve blocks an SM, 32 at most (8 and 24 blocks
  // take 18 and 19 us there, 4 and 48 take 28 and 21)
  int per = (int)std::min<int64_t>(std::max<int64_t>((int64_t)a.B * across / (12 * nsm), 1), 32);
  per = std::max(per, ceil_div(a.B, 65535));
  scan_step_kernel<T, LANES, WIDE><<<dim3((unsigned)across, ceil_div(a.B, per)), NT, 0, s>>>(a, per, err);
  return cudaGetLastError();
}

template <typename T, int LANES>
cudaError_t step_of(const ScanStep &a, int *err, int nsm, bool vec, cudaStream_t s) {
  const int size = sizeof(T);
  return vec && a.N % V == 0 && aligned(a.state, 4, 4, 4) && aligned(a.b, a.ldb, size, V) && aligned(a.c, a.ldc, size, V)
             ? run<T, LANES, true>(a, err, nsm, s)
             : run<T, LANES, false>(a, err, nsm, s);
}

template <typename T>
cudaError_t by_states(const ScanStep &a, int *err, int nsm, bool vec, cudaStream_t s) {
  if (a.N <= 4) return step_of<T, 1>(a, err, nsm, vec, s);
  if (a.N <= 8) return step_of<T, 2>(a, err, nsm, vec, s);
  if (a.N <= 16) return step_of<T, 4>(a, err, nsm, vec, s);
  if (a.N <= 32) return step_of<T, 8>(a, err, nsm, vec, s);
  return step_of<T, 16>(a, err, nsm, vec, s);
}

}  // namespace

cudaError_t launch_scan_step(const ScanStep &p, int *err, int nsm, bool vec, cudaStream_t s,
                             int *launches) {
  ++*launches;
  return p.dtype == RCU_BF16 ? by_states<bf16>(p, err, nsm, vec, s) : by_states<float>(p, err, nsm, vec, s);
}

}  // namespace rcu
