// Layer norm, forward, with the residual addition before it.
//
// Bound by memory: a row is read once, as 16-byte words where the rows allow,
// kept in registers as it came (bf16 stays packed) and summed twice, the second
// time about the mean.  A row belongs to W warps of one block, the fewest for
// which a lane has at most 16 values: weight and bias of a lane's columns then
// fit its registers beside them (with 32 values a lane, read again for every row,
// bf16 131072x1024 took 284 us).  Short rows share a block.  Blocks take rows
// until there are none left, and have the next row's loads in flight while they
// work on one.  Measured: bf16 131072x1024 with a residual 170 us, 6.3 TB/s of the
// 1075 MB it must move.
#include "layernorm.cuh"

namespace rcu {
namespace {

using namespace ln;

// Rows of n values, W warps a row, N words of VEC values a lane, R rows a block.
template <typename T, int VEC, int N, int W, int R, bool RES>
__global__ void __launch_bounds__(32 * W * R) ln_fwd_kernel(const LnFwd p) {
  __shared__ float2 part[2][32];
  const int sub = threadIdx.x / (32 * W), lane = threadIdx.x % (32 * W);
  const int64_t step = (int64_t)gridDim.x * R;
  int buf = 0;
  typedef Vals<T, VEC> Word;
  Word next[N], rnext[N];
  auto load = [&](int64_t row) {
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *r = RES ? static_cast<const T *>(p.res) + row * p.ldres : nullptr;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = (k * 32 * W + lane) * VEC;
      next[k].zero();
      if (RES) rnext[k].zero();
      if (row < p.rows && c < p.n) {
        next[k].load(x + c);
        if (RES) rnext[k].load(r + c);
      }
    }
  };
  load((int64_t)blockIdx.x * R + sub);
  float w[N][VEC], b[N][VEC];
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = (k * 32 * W + lane) * VEC + j;
      w[k][j] = p.weight && c < p.n ? __ldg(p.weight + c) : 1.f;
      b[k][j] = p.bias && c < p.n ? __ldg(p.bias + c) : 0.f;
    }
  for (int64_t base = (int64_t)blockIdx.x * R; base < p.rows; base += step) {
    const int64_t row = base + sub;
    Word u[N];
    float s = 0.f, d2 = 0.f, none = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      u[k] = next[k];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (RES) u[k].set(j, u[k][j] + rnext[k][j]);
        s += u[k][j];
      }
    }
    load(row + step);
    if (RES && row < p.rows) {
      T *sum = static_cast<T *>(p.sum) + row * p.ldsum;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int c = (k * 32 * W + lane) * VEC;
        if (c < p.n) u[k].store(sum + c);
      }
    }
    row_sum<W>(s, none, part, buf);
    const float mean = s / p.n;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if ((k * 32 * W + lane) * VEC < p.n) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = u[k][j] - mean;
          d2 = fmaf(d, d, d2);
        }
      }
    }
    row_sum<W>(d2, none, part, buf);
    const float rstd = 1.f / sqrtf(d2 / p.n + p.eps);
    if (row < p.rows) {
      T *y = static_cast<T *>(p.y) + row * p.ldy;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int c = (k * 32 * W + lane) * VEC;
        if (c < p.n) {
          Word o;
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            o.set(j, fmaf((u[k][j] - mean) * rstd, w[k][j], b[k][j]));
          o.store(y + c);
        }
      }
      if (lane == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
      }
    }
  }
}

// Rows too long for registers: one block a row, read once for each sum and once
// for the result (the second and third time from L2).
template <typename T, int VEC>
__global__ void __launch_bounds__(LONG_NT) ln_fwd_long_kernel(const LnFwd p) {
  typedef Vals<T, VEC> Word;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *r = p.res ? static_cast<const T *>(p.res) + row * p.ldres : nullptr;
    T *sum = p.sum ? static_cast<T *>(p.sum) + row * p.ldsum : nullptr;
    T *y = static_cast<T *>(p.y) + row * p.ldy;
    auto get = [&](int c) {
      Word u, v;
      u.load(x + c);
      if (r) {
        v.load(r + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) u.set(j, u[j] + v[j]);
      }
      return u;
    };
    float s = 0.f;
    for (int c = threadIdx.x * VEC; c < p.n; c += LONG_NT * VEC) {
      const Word u = get(c);
      if (sum) u.store(sum + c);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += u[j];
    }
    const float mean = block_sum(s) / p.n;
    s = 0.f;
    for (int c = threadIdx.x * VEC; c < p.n; c += LONG_NT * VEC) {
      const Word u = get(c);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = u[j] - mean;
        s = fmaf(d, d, s);
      }
    }
    const float rstd = 1.f / sqrtf(block_sum(s) / p.n + p.eps);
    for (int c = threadIdx.x * VEC; c < p.n; c += LONG_NT * VEC) {
      const Word u = get(c);
      Word o;
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        o.set(j, fmaf((u[j] - mean) * rstd, p.weight ? p.weight[c + j] : 1.f,
                      p.bias ? p.bias[c + j] : 0.f));
      o.store(y + c);
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
}

template <typename T, int VEC, int N, int W, bool RES>
void run(const LnFwd &p, int nsm, cudaStream_t s) {
  constexpr int R = W >= 4 ? 1 : 4 / W;
  static PerDevice<int> room;
  const int blocks = room.here(
      [&] { return resident_blocks(ln_fwd_kernel<T, VEC, N, W, R, RES>, 32 * W * R, 0, nsm); });
  const int grid = (int)std::min<int64_t>((p.rows + R - 1) / R, blocks);
  ln_fwd_kernel<T, VEC, N, W, R, RES><<<grid, 32 * W * R, 0, s>>>(p);
}

// Values a lane: 8 of a short row, else 16.
template <typename T, int VEC, bool RES>
void shape(const LnFwd &p, int nsm, cudaStream_t s) {
  if (p.n <= 256) run<T, VEC, 8 / VEC, 1, RES>(p, nsm, s);
  else if (p.n <= 512) run<T, VEC, 16 / VEC, 1, RES>(p, nsm, s);
  else if (p.n <= 1024) run<T, VEC, 16 / VEC, 2, RES>(p, nsm, s);
  else if (p.n <= 2048) run<T, VEC, 16 / VEC, 4, RES>(p, nsm, s);
  else if (p.n <= 4096) run<T, VEC, 16 / VEC, 8, RES>(p, nsm, s);
  else if (p.n <= 8192) run<T, VEC, 16 / VEC, 16, RES>(p, nsm, s);
  else ln_fwd_long_kernel<T, VEC><<<(int)std::min<int64_t>(p.rows, 4 * nsm), LONG_NT, 0, s>>>(p);
}

template <typename T, int VEC>
void fwd(const LnFwd &p, int nsm, bool vec, cudaStream_t s) {
  const int size = sizeof(T);
  const bool wide = vec && p.n % VEC == 0 && aligned(p.x, p.ldx, size, 16) &&
                    aligned(p.res, p.ldres, size, 16) && aligned(p.y, p.ldy, size, 16) &&
                    aligned(p.sum, p.ldsum, size, 16);
  if (wide) p.res ? shape<T, VEC, true>(p, nsm, s) : shape<T, VEC, false>(p, nsm, s);
  else p.res ? shape<T, 1, true>(p, nsm, s) : shape<T, 1, false>(p, nsm, s);
}

}  // namespace

cudaError_t launch_ln_fwd(const LnFwd &p, int nsm, bool vec, cudaStream_t s, int *launches) {
  if (p.dtype == RCU_BF16) fwd<bf16, VEC_BF16>(p, nsm, vec, s);
  else fwd<float, VEC_F32>(p, nsm, vec, s);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace rcu
