// Layer norm, backward: du, and the weight's and bias's gradients.
//
// Bound by memory, and shaped as the forward: a row belongs to W warps of one
// block, 16 or 32 values a lane, the next row's loads in flight.  Each lane has the
// same columns of every row its warps take, so the column sums (dweight, dbias)
// build up in its registers; every block writes one row of partial sums at the
// end, and a second kernel adds those in a fixed order.  Measured: bf16
// 131072x1024 with dsum 184 us, 5.9 TB/s; fp32 from 8 bits 12501x1000 29 us (22 and
// 9 for the two kernels with a cold cache), which L2 holds: latency of its waves.
#include "layernorm.cuh"

namespace rcu {
namespace {

using namespace ln;

// As the forward; part_w, part_b: [gridDim.x][n], this block's share of the
// column sums (NULL: not wanted).
template <typename IT, typename T, int VEC, int N, int W, int R>
__global__ void __launch_bounds__(32 * W * R)
    ln_bwd_kernel(const LnBwd p, float *__restrict__ part_w, float *__restrict__ part_b) {
  extern __shared__ float cols[];  // [R][2][N * 32 * W * VEC] at the end, for R > 1
  __shared__ float2 part[2][32];
  const int sub = threadIdx.x / (32 * W), lane = threadIdx.x % (32 * W);
  const int64_t step = (int64_t)gridDim.x * R;
  const int nb = ceil_div(p.n, RCU_ACT8_BLOCK);
  int buf = 0;
  Vals<T, VEC> dy[N], ds[N], dy1[N], ds1[N];  // 1: of the next row
  Vals<IT, VEC> u[N], u1[N];
  float mean1 = 0.f, rstd1 = 0.f;
  auto load = [&](int64_t row) {
    const bool on = row < p.rows;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = (k * 32 * W + lane) * VEC;
      dy1[k].zero();
      u1[k].zero();
      ds1[k].zero();
      if (on && c < p.n) {
        dy1[k].load(static_cast<const T *>(p.dy) + row * p.lddy + c);
        u1[k].load(static_cast<const IT *>(p.u) + row * p.ldu + c);
        u1[k].block(p.ue + row * nb + c / RCU_ACT8_BLOCK);
        if (p.dsum) ds1[k].load(static_cast<const T *>(p.dsum) + row * p.ldds + c);
      }
    }
    mean1 = on ? __ldg(p.mean + row) : 0.f;
    rstd1 = on ? __ldg(p.rstd + row) : 0.f;
  };
  float w[N][VEC], gw[N][VEC], gb[N][VEC];
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = (k * 32 * W + lane) * VEC + j;
      w[k][j] = c < p.n ? (p.weight ? __ldg(p.weight + c) : 1.f) : 0.f;
      gw[k][j] = gb[k][j] = 0.f;
    }
  // 16 warps a row, or a register for every value, leave none for a second row
  constexpr bool AHEAD = W < 16 && VEC > 1;
  if (AHEAD) load((int64_t)blockIdx.x * R + sub);
  for (int64_t base = (int64_t)blockIdx.x * R; base < p.rows; base += step) {
    const int64_t row = base + sub;
    if (!AHEAD) load(row);
    const float mean = mean1, rstd = rstd1;
#pragma unroll
    for (int k = 0; k < N; ++k) dy[k] = dy1[k], u[k] = u1[k], ds[k] = ds1[k];
    if (AHEAD) load(row + step);
    float s1 = 0.f, s2 = 0.f;
    float xh[N][VEC];  // kept to the second pass where making it again costs more (8 bits)
    auto normalise = [&](int k) {
      u[k].decode(xh[k]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) xh[k][j] = (xh[k][j] - mean) * rstd;
    };
#pragma unroll
    for (int k = 0; k < N; ++k) {
      normalise(k);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float g = dy[k][j], q = g * w[k][j];
        s1 += q;
        s2 = fmaf(q, xh[k][j], s2);
        gw[k][j] = fmaf(g, xh[k][j], gw[k][j]);
        gb[k][j] += g;
      }
    }
    row_sum<W>(s1, s2, part, buf);
    s1 /= p.n;
    s2 /= p.n;
    if (row < p.rows) {
      T *du = static_cast<T *>(p.du) + row * p.lddu;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int c = (k * 32 * W + lane) * VEC;
        if (c < p.n) {
          Vals<T, VEC> o;
          if (sizeof(IT) > 1) normalise(k);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float d = fmaf(-xh[k][j], s2, fmaf(dy[k][j], w[k][j], -s1));
            o.set(j, fmaf(rstd, d, p.dsum ? ds[k][j] : 0.f));
          }
          o.store(du + c);
        }
      }
    }
  }
  if (!part_w) return;
  constexpr int COLS = N * 32 * W * VEC;
  if (R > 1) {  // the block's R rows join in order
    float *mine = cols + sub * 2 * COLS;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        mine[(k * VEC + j) * 32 * W + lane] = gw[k][j];
        mine[COLS + (k * VEC + j) * 32 * W + lane] = gb[k][j];
      }
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        for (int q = 1; q < R; ++q) {
          gw[k][j] += cols[q * 2 * COLS + (k * VEC + j) * 32 * W + lane];
          gb[k][j] += cols[q * 2 * COLS + COLS + (k * VEC + j) * 32 * W + lane];
        }
  }
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = (k * 32 * W + lane) * VEC + j;
      if (c < p.n) {
        part_w[(int64_t)blockIdx.x * p.n + c] = gw[k][j];
        part_b[(int64_t)blockIdx.x * p.n + c] = gb[k][j];
      }
    }
}

// out[c] = the sum of `rows` partial rows: a block has 32 columns, its warps
// share the rows, and their sums join in order.
constexpr int SUM_WARPS = 32;
__global__ void __launch_bounds__(32 * SUM_WARPS) ln_columns_kernel(const float *__restrict__ part_w, const float *__restrict__ part_b,
                                  int rows, int n, float *__restrict__ dw, float *__restrict__ db) {
  __shared__ float2 part[SUM_WARPS][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane;
  float a = 0.f, b = 0.f;
  wait_for_previous();
  if (c < n)
#pragma unroll 8
    for (int r = warp; r < rows; r += SUM_WARPS) {
      a += part_w[(int64_t)r * n + c];
      b += part_b[(int64_t)r * n + c];
    }
  part[warp][lane] = make_float2(a, b);
  __syncthreads();
  if (warp == 0 && c < n) {
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < SUM_WARPS; ++w) a += part[w][lane].x, b += part[w][lane].y;
    if (dw) dw[c] = a;
    if (db) db[c] = b;
  }
}

// Rows too long for registers: du as in the forward's long form, and the column
// sums by blocks of 32 columns over a share of the rows each.
template <typename IT>
__device__ __forceinline__ float saved(const LnBwd &p, int64_t row, int c) {
  return to_f(static_cast<const IT *>(p.u)[row * p.ldu + c]);
}
template <>
__device__ __forceinline__ float saved<int8_t>(const LnBwd &p, int64_t row, int c) {
  return act8_value(static_cast<const int8_t *>(p.u)[row * p.ldu + c],
                    p.ue[row * ceil_div(p.n, RCU_ACT8_BLOCK) + c / RCU_ACT8_BLOCK]);
}
template <typename IT, typename T>
__global__ void __launch_bounds__(LONG_NT) ln_bwd_long_kernel(const LnBwd p) {
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T *dy = static_cast<const T *>(p.dy) + row * p.lddy;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < p.n; c += LONG_NT) {
      const float q = to_f(dy[c]) * (p.weight ? p.weight[c] : 1.f);
      s1 += q;
      s2 = fmaf(q, (saved<IT>(p, row, c) - mean) * rstd, s2);
    }
    s1 = block_sum(s1) / p.n;
    s2 = block_sum(s2) / p.n;
    for (int c = threadIdx.x; c < p.n; c += LONG_NT) {
      const float xh = (saved<IT>(p, row, c) - mean) * rstd;
      const float d = fmaf(-xh, s2, fmaf(to_f(dy[c]), p.weight ? p.weight[c] : 1.f, -s1));
      const float more = p.dsum ? to_f(static_cast<const T *>(p.dsum)[row * p.ldds + c]) : 0.f;
      static_cast<T *>(p.du)[row * p.lddu + c] = from_f<T>(fmaf(rstd, d, more));
    }
  }
}
template <typename IT, typename T>
__global__ void __launch_bounds__(32 * SUM_WARPS)
    ln_bwd_long_columns_kernel(const LnBwd p, float *__restrict__ part_w,
                               float *__restrict__ part_b) {
  __shared__ float2 part[SUM_WARPS][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane;
  float a = 0.f, b = 0.f;
  if (c < p.n)
    for (int64_t row = blockIdx.y * SUM_WARPS + warp; row < p.rows;
         row += (int64_t)gridDim.y * SUM_WARPS) {
      const float g = to_f(static_cast<const T *>(p.dy)[row * p.lddy + c]);
      a = fmaf(g, (saved<IT>(p, row, c) - p.mean[row]) * p.rstd[row], a);
      b += g;
    }
  part[warp][lane] = make_float2(a, b);
  __syncthreads();
  if (warp == 0 && c < p.n) {
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < SUM_WARPS; ++w) a += part[w][lane].x, b += part[w][lane].y;
    part_w[(int64_t)blockIdx.y * p.n + c] = a;
    part_b[(int64_t)blockIdx.y * p.n + c] = b;
  }
}

template <typename IT, typename T, int VEC, int N, int W>
cudaError_t run(const LnBwd &p, DevMem &ws, int nsm, cudaStream_t s, int *launches) {
  constexpr int R = W >= 4 ? 1 : 4 / W, NT = 32 * W * R;
  constexpr size_t SMEM = R > 1 ? (size_t)R * 2 * N * 32 * W * VEC * 4 : 0;
  static_assert(SMEM <= 40 << 10, "within the default limit, with what the kernel has besides");
  static PerDevice<int> room;
  const int blocks = room.here(
      [&] { return resident_blocks(ln_bwd_kernel<IT, T, VEC, N, W, R>, NT, SMEM, nsm); });
  const int grid = (int)std::min<int64_t>((p.rows + R - 1) / R, blocks);
  float *part = nullptr;
  const bool columns = p.dweight || p.dbias;
  if (columns) {
    const cudaError_t e = ws.get((size_t)grid * p.n * 8, &part);
    if (e != cudaSuccess) return e;
  }
  float *part_b = columns ? part + (int64_t)grid * p.n : nullptr;
  ln_bwd_kernel<IT, T, VEC, N, W, R><<<grid, NT, SMEM, s>>>(p, part, part_b);
  ++*launches;
  if (columns) {
    const cudaError_t e = launch_after(ln_columns_kernel, dim3(ceil_div(p.n, 32)), 32 * SUM_WARPS, s,
                                       part, part_b, grid, p.n, p.dweight, p.dbias);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaGetLastError();
}

template <typename IT, typename T>
cudaError_t run_long(const LnBwd &p, DevMem &ws, int nsm, cudaStream_t s, int *launches) {
  ln_bwd_long_kernel<IT, T><<<(int)std::min<int64_t>(p.rows, 4 * nsm), LONG_NT, 0, s>>>(p);
  ++*launches;
  if (!p.dweight && !p.dbias) return cudaGetLastError();
  const int shares = (int)std::min<int64_t>((p.rows + SUM_WARPS - 1) / SUM_WARPS, 16);
  float *part = nullptr;
  const cudaError_t e = ws.get((size_t)shares * p.n * 8, &part);
  if (e != cudaSuccess) return e;
  float *part_b = part + (int64_t)shares * p.n;
  ln_bwd_long_columns_kernel<IT, T>
      <<<dim3(ceil_div(p.n, 32), shares), 32 * SUM_WARPS, 0, s>>>(p, part, part_b);
  *launches += 2;
  return launch_after(ln_columns_kernel, dim3(ceil_div(p.n, 32)), 32 * SUM_WARPS, s, part, part_b,
                      shares, p.n, p.dweight, p.dbias);
}

// Values a lane (PER): 32 where they lie packed (bf16 by 16-byte words), so that a
// row of 1024 needs no barrier (182 us at 131072 rows, 191 with 16 values in two
// warps); else 16 (fp32 from 8 bits 12501x1000: 29 us, 38 with 32).
template <typename IT, typename T, int VEC>
cudaError_t shape(const LnBwd &p, DevMem &ws, int nsm, cudaStream_t s, int *launches) {
  constexpr bool PACKED = sizeof(IT) == 2 && VEC == VEC_BF16;
  constexpr int PER = PACKED ? 32 : 16, MORE = PER / 16;
  if (p.n <= 256) return run<IT, T, VEC, 8 / VEC, 1>(p, ws, nsm, s, launches);
  if (p.n <= 512) return run<IT, T, VEC, 16 / VEC, 1>(p, ws, nsm, s, launches);
  if (p.n <= 1024) return run<IT, T, VEC, PER / VEC, 2 / MORE>(p, ws, nsm, s, launches);
  if (p.n <= 2048) return run<IT, T, VEC, PER / VEC, 4 / MORE>(p, ws, nsm, s, launches);
  if (p.n <= 4096) return run<IT, T, VEC, PER / VEC, 8 / MORE>(p, ws, nsm, s, launches);
  if (p.n <= 8192) return run<IT, T, VEC, PER / VEC, 16 / MORE>(p, ws, nsm, s, launches);
  return run_long<IT, T>(p, ws, nsm, s, launches);
}

template <typename IT, typename T, int VEC>
cudaError_t bwd(const LnBwd &p, DevMem &ws, int nsm, bool vec, cudaStream_t s, int *launches) {
  const int size = sizeof(T), in = sizeof(IT);
  const bool wide = vec && p.n % VEC == 0 && aligned(p.dy, p.lddy, size, 16) &&
                    aligned(p.u, p.ldu, in, VEC * in) && aligned(p.dsum, p.ldds, size, 16) &&
                    aligned(p.du, p.lddu, size, 16);
  return wide ? shape<IT, T, VEC>(p, ws, nsm, s, launches)
              : shape<IT, T, 1>(p, ws, nsm, s, launches);
}

}  // namespace

cudaError_t launch_ln_bwd(const LnBwd &p, DevMem &ws, int nsm, bool vec, cudaStream_t s,
                          int *launches) {
  const bool q8 = p.saved == RCU_I8;
  if (p.dtype == RCU_BF16)
    return q8 ? bwd<int8_t, bf16, VEC_BF16>(p, ws, nsm, vec, s, launches)
              : bwd<bf16, bf16, VEC_BF16>(p, ws, nsm, vec, s, launches);
  return q8 ? bwd<int8_t, float, VEC_F32>(p, ws, nsm, vec, s, launches)
            : bwd<float, float, VEC_F32>(p, ws, nsm, vec, s, launches);
}

}  // namespace rcu
