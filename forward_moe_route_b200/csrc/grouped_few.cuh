// moe_grouped_mm for a handful of rows (generated tokens): every SM streams
// weights, with no tiles to fill, no clusters and no pipeline to start.
//
// A warp takes two weight rows at a time, its lanes 8 elements of the contraction
// each, four such pieces of either row in flight, and multiplies them with one or
// two of the group's rows in fp32 on the CUDA cores.  Bound by the weights' bytes
// and, at these sizes, by latency.  Back to back in a graph, the weights in L2, and
// (in brackets) k_grouped_mm: a row in 4096 x 4096 6.8 us (15.4), one row of 64
// groups 2048 x 2816 4.3 us (10.5); single calls with the weights out of L2 18.4 us
// (20.5) and 10.2 us (16.4).
#pragma once

#include "common.cuh"
#include "grouped.cuh"
#include "norm.cuh"

namespace moe {
namespace grouped {

constexpr int FEW_MAX = 16;            // most rows of a call
constexpr int FEW_BLOCK = 2;           // rows that share one pass over the weights
constexpr int FEW_THREADS = 256;
constexpr int FEW_FEATURES = 2;        // weight rows of a warp at a time
constexpr int FEW_PIECES = 4;          // pieces of each in flight

// The groups that have rows, in the order of their rows: first row, rows, number.
struct FewRuns {
  int first[FEW_MAX], rows[FEW_MAX], group[FEW_MAX], of_row[FEW_MAX];
  int n;
};
__device__ __forceinline__ void few_runs(FewRuns& s, const int* offsets, int n, int n_rows) {
  if (threadIdx.x < FEW_MAX) s.of_row[threadIdx.x] = -1;
  __syncthreads();
  for (int g = threadIdx.x; g < n; g += blockDim.x) {
    const int r0 = offsets[g], r1 = offsets[g + 1];
    if (!group_ok(r0, r1, n_rows)) {
      if (blockIdx.x == 0) set_status(MOE_ERR_DEVICE_CHECK);
      continue;
    }
    for (int r = r0; r < r1; ++r) s.of_row[r] = g;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int runs = 0;
    for (int r = 0; r < n_rows; ++r) {
      const int g = s.of_row[r];
      if (g < 0) continue;
      if (runs && s.group[runs - 1] == g && s.first[runs - 1] + s.rows[runs - 1] == r) {
        ++s.rows[runs - 1];
        continue;
      }
      s.first[runs] = r;
      s.rows[runs] = 1;
      s.group[runs++] = g;
    }
    s.n = runs;
  }
  __syncthreads();
}

using Piece = norm::Raw<__nv_bfloat16, 8>;

// `feats` features (FEW_FEATURES at most) of ROWS rows.
template <int ROWS>
__device__ __forceinline__ void few_mm_item(const Args& a, const __nv_bfloat16* w,
                                            const __nv_bfloat16* x, __nv_bfloat16* y, int feats) {
  const int lane = lane_id();
  float acc[FEW_FEATURES][ROWS];
#pragma unroll
  for (int f = 0; f < FEW_FEATURES; ++f)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) acc[f][r] = 0.f;
  for (int k0 = lane * 8; k0 < a.contract; k0 += 256 * FEW_PIECES) {
    Piece pw[FEW_PIECES][FEW_FEATURES];
#pragma unroll
    for (int p = 0; p < FEW_PIECES; ++p)
#pragma unroll
      for (int f = 0; f < FEW_FEATURES; ++f) {
        const int k = k0 + 256 * p;
        if (k < a.contract) pw[p][f].load(w + (size_t)(f < feats ? f : 0) * a.contract + k);
        else pw[p][f].zero();
      }
#pragma unroll
    for (int p = 0; p < FEW_PIECES; ++p) {
      const int k = k0 + 256 * p;
      if (k >= a.contract) break;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        Piece px;
        px.load(x + (size_t)r * a.contract + k);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int f = 0; f < FEW_FEATURES; ++f)
            acc[f][r] = fmaf(pw[p][f].get(j), px.get(j), acc[f][r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int f = 0; f < FEW_FEATURES; ++f) {
      const float v = warp_sum(acc[f][r]);
      if (lane == f && f < feats) y[(size_t)r * a.feats + f] = __float2bfloat16_rn(v);
    }
}

// The features of all runs are strided over the grid's warps.
__global__ void __launch_bounds__(FEW_THREADS, 4) k_few_mm(const Args a, const __nv_bfloat16* x,
                                                        const __nv_bfloat16* w) {
  grid_dep_sync();
  __shared__ FewRuns runs;
  few_runs(runs, a.offsets, a.n, a.n_rows);
  const int items = (a.feats + FEW_FEATURES - 1) / FEW_FEATURES;
  const int warps = (int)gridDim.x * (FEW_THREADS / 32);
  for (int i = (int)blockIdx.x * (FEW_THREADS / 32) + warp_id(); i < runs.n * items; i += warps) {
    const int run = i / items, f = (i - run * items) * FEW_FEATURES;
    const int feats = min(FEW_FEATURES, a.feats - f);
    const __nv_bfloat16* wf = w + ((size_t)runs.group[run] * a.feats + f) * a.contract;
    for (int r = 0; r < runs.rows[run]; r += FEW_BLOCK) {
      const __nv_bfloat16* xr = x + (size_t)(runs.first[run] + r) * a.contract;
      __nv_bfloat16* yr = a.y + (size_t)(runs.first[run] + r) * a.feats + f;
      if (runs.rows[run] - r == 1) few_mm_item<1>(a, wf, xr, yr, feats);
      else few_mm_item<2>(a, wf, xr, yr, feats);
    }
  }
}

}  // namespace grouped
}  // namespace moe
