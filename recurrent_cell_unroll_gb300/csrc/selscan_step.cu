// Selective scan, one step of many requests: states in a table of slots, updated
// in place.  Bound by memory (8 bytes a state) at serving sizes, by latency below.
//
// A thread keeps 4 states of a channel, neighbouring threads the channel's others,
// and takes several requests, since a channel's rates cost more than a step; four are
// read together (bf16 B=256 H=2048 N=16, cold: 21 us one by one, 10.3 so).  From Python
// a call takes some 16 us, which bounds it at such sizes.
#include "selscan.cuh"

namespace rcu {
namespace {

using namespace selscan;

constexpr int NT = 128, V = 4, ROWS = 4;  // states of a thread, requests read together

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
  for (int64_t first = b0; first < b1; first += ROWS) {
    // all reads of ROWS requests before the first is worked on
    int64_t slot[ROWS];
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      const int64_t b = first + q;
      slot[q] = -1;
      if (b >= b1) continue;
      slot[q] = a.slot ? a.slot[b] : b;
      if (slot[q] < -1 || slot[q] >= a.slots) {
        atomicCAS(err, (int)DEV_OK, (int)DEV_SLOTS);
        slot[q] = -1;
      }
    }
    T x[ROWS], dt[ROWS], z[ROWS];
    Word<T, V> bw[ROWS], cw[ROWS];
    float4 h[ROWS];
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      if (slot[q] < 0) continue;
      const int64_t b = first + q;
      x[q] = static_cast<const T *>(a.x)[b * a.ldx + ch];
      dt[q] = static_cast<const T *>(a.dt)[b * a.lddt + ch];
      if (a.z) z[q] = static_cast<const T *>(a.z)[b * a.ldz + ch];
      if (!states) continue;
      const float *state = a.state + (slot[q] * a.H + ch) * a.N + n0;
      const T *bp = static_cast<const T *>(a.b) + b * a.ldb + n0, *cp = static_cast<const T *>(a.c) + b * a.ldc + n0;
      if (WIDE) {
        h[q] = *reinterpret_cast<const float4 *>(state);
        bw[q] = *reinterpret_cast<const Word<T, V> *>(bp);
        cw[q] = *reinterpret_cast<const Word<T, V> *>(cp);
      } else {
        float v[V] = {};
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (n0 + k < a.N) v[k] = state[k], bw[q].v[k] = bp[k], cw[q].v[k] = cp[k];
        h[q] = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      const int64_t b = first + q;
      if (b >= b1) break;
      T *y = static_cast<T *>(a.y) + b * a.ldy + ch;
      if (slot[q] < 0) {  // the same for the warp
        if (live && l == 0) *y = from_f<T>(0.f);
        continue;
      }
      const float xv = to_f(x[q]), delta = softplus(to_f(dt[q]) + bias), u = delta * xv;
      float v[V] = {h[q].x, h[q].y, h[q].z, h[q].w}, s = 0.f;
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (WIDE ? states : n0 + k < a.N) {
          v[k] = fmaf(ex2(delta * A2[k]), v[k], u * to_f(bw[q].v[k]));
          s = fmaf(v[k], to_f(cw[q].v[k]), s);
        }
      if (live && states) {
        float *state = a.state + (slot[q] * a.H + ch) * a.N + n0;
        if (WIDE) {
          *reinterpret_cast<float4 *>(state) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k)
            if (n0 + k < a.N) state[k] = v[k];
        }
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (live && l == 0) {
        if (a.d) s = fmaf(skip, xv, s);
        if (a.z) {
          const float zv = to_f(z[q]);
          s *= zv * sigmoid(zv);
        }
        *y = from_f<T>(s);
      }
    }
  }
}

template <typename T, int LANES, bool WIDE>
cudaError_t run(const ScanStep &a, int *err, int nsm, cudaStream_t s) {
  const int64_t across = ((int64_t)a.H * LANES + NT - 1) / NT;
  // as many requests a thread as leave ten blocks an SM, 32 at most
  int per = (int)std::min<int64_t>(std::max<int64_t>((int64_t)a.B * across / (10 * nsm), 1), 32);
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
