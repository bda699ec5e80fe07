// Sums over the rows of a [rows, cols] fp32 matrix of partial sums, in a fixed
// order: a block takes 32 columns, its 8 warps every eighth row each, and adds
// the warps' sums in their order.  Reads each partial sum once.
#include "ssm_common.cuh"

namespace rcu {
namespace {

constexpr int WARPS = 8;

__global__ void __launch_bounds__(32 * WARPS) column_sum_kernel(const ColumnSum a) {
  __shared__ float sums[WARPS][32];
  wait_for_previous();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float v[4] = {};
  if (col < a.cols) {
    int64_t r = warp;
    for (; r + 3 * WARPS < a.rows; r += 4 * WARPS)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += a.part[(r + k * WARPS) * a.cols + col];
    for (; r < a.rows; r += WARPS) v[0] += a.part[r * a.cols + col];
  }
  sums[warp][lane] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  if (warp || col >= a.cols) return;
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < WARPS; ++k) s += sums[k][lane];
  if (col < a.n0) {
    if (a.out0) a.out0[col] = s;
  } else if (col < a.n0 + a.n1) {
    if (a.out1) a.out1[col - a.n0] = s;
  } else if (a.out2) {
    a.out2[col - a.n0 - a.n1] = s;
  }
}

}  // namespace

cudaError_t launch_column_sum(const ColumnSum &p, cudaStream_t s, int *launches) {
  ++*launches;
  return launch_after(column_sum_kernel, dim3((unsigned)((p.cols + 31) / 32)), 32 * WARPS, s, p);
}

}  // namespace rcu
