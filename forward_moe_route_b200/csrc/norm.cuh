// Norms before and after a block, and their backward passes.
//
//   before the layer   x = u r(u) w,            r(v) = (mean(v^2) + eps)^-1/2
//   behind the layer   y = sum of the token's expert rows,
//                      h = res u + gate * (y r(y) w),   x_next = h r(h) w_next
//
// in one pass over the row: the row stays in registers between its sums and
// its outputs, so each input is read and each output written once.  All
// arithmetic is fp32; every output is rounded once, from the fp32 value (x_next
// from the unrounded h, its norm from the unrounded sum).
//
// Backward of n = v r(v) for c = dL/dn: with q = mean(v^2) + eps and r = q^-1/2,
//   dv = r c - v r^3 mean(v c),
// so both sums of a row (v^2 and v c) are taken in the same reduction and no
// statistic is kept from the forward.  c = upstream * w (* gate); the weight's
// gradient is sum_t upstream * gate * n, the gate's sum over its tokens of
// upstream * w * n.
//
// These kernels are bound by memory: at most 30 operations per element read.
// A row is held by one warp (up to 4 vectors of 16 bytes a lane) or by one
// block.  Row sums are warp shuffles, then one shared-memory exchange.
#pragma once

#include "common.cuh"

namespace moe {
namespace norm {

constexpr int MAX_THREADS = 1024;

template <typename E>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int VEC = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

// V elements at p, as fp32: one 16-byte access when V fills it, else single elements.
template <typename E, int V>
__device__ __forceinline__ void load_vec(const E* p, float (&v)[V]) {
  if constexpr (V == Elem<E>::VEC) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p);
    const E* e = reinterpret_cast<const E*>(&raw);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = Elem<E>::get(e[i]);
  } else {
    static_assert(V == 1, "");
    v[0] = Elem<E>::get(*p);
  }
}
template <typename E, int V>
__device__ __forceinline__ void store_vec(E* p, const float (&v)[V]) {
  if constexpr (V == Elem<E>::VEC) {
    uint4 raw;
    E* e = reinterpret_cast<E*>(&raw);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = Elem<E>::put(v[i]);
    *reinterpret_cast<uint4*>(p) = raw;
  } else {
    *p = Elem<E>::put(v[0]);
  }
}

// The threads that share a row: one warp of the block (tpr = 32), or the block.
// Sums over them; `red` is double-buffered, so one barrier per sum suffices:
// a buffer is written again only behind the next sum's barrier.
struct RowGroup {
  int tpr, tid;          // threads of the row, this thread's place among them
  float2 (*red)[32];     // [2][32] shared
  int buf;
  __device__ __forceinline__ float2 sum2(float a, float b) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (tpr == 32) return make_float2(a, b);
    const int nw = tpr >> 5;
    if (lane_id() == 0) red[buf][warp_id()] = make_float2(a, b);
    __syncthreads();
    const float2 v = lane_id() < nw ? red[buf][lane_id()] : make_float2(0.f, 0.f);
    buf ^= 1;
    return make_float2(warp_sum(v.x), warp_sum(v.y));
  }
  __device__ __forceinline__ float sum(float a) { return sum2(a, 0.f).x; }
};

__device__ __forceinline__ float inv_rms(float sumsq, int d, float eps) {
  return 1.0f / sqrtf(sumsq / (float)d + eps);
}

struct FwdArgs {
  const void* u;         // [T, d]: the input of k_norm; the residual of k_combine_norm
  const void* slots;     // [T, S, d]
  const void* w;         // [d]
  const void* gate;      // [n_gate, d] or null
  const void* w_next;    // [d] or null
  void* h;               // [T, d]: x of k_norm
  void* y;               // [T, d] or null
  void* x_next;          // [T, d] with w_next
  int T, d, S, gate_group;
  int tpr;               // threads of a row
  float eps, res;
};

// COMBINE = false: h = u r(u) w.  Rows are strided over the grid's row groups.
template <typename E, int V, int VPT, bool COMBINE>
__global__ void __launch_bounds__(MAX_THREADS) k_norm_fwd(const FwdArgs a) {
  grid_dep_sync();
  __shared__ float2 red[2][32];
  const int rows_here = blockDim.x / a.tpr;
  RowGroup g{a.tpr, (int)threadIdx.x % a.tpr, red, 0};
  const int d = a.d;
  const E* w = static_cast<const E*>(a.w);
  for (long long t = (long long)blockIdx.x * rows_here + threadIdx.x / a.tpr; t < a.T;
       t += (long long)gridDim.x * rows_here) {
    float v[VPT][V];
    float ss = 0.f;
    const E* in = COMBINE ? static_cast<const E*>(a.slots) + t * a.S * d
                          : static_cast<const E*>(a.u) + t * d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (g.tid + i * a.tpr) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = 0.f;
      if (c < d) {
        if (COMBINE) {
#pragma unroll 4
          for (int s = 0; s < a.S; ++s) {
            float x[V];
            load_vec<E, V>(in + (long long)s * d + c, x);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] += x[j];
          }
        } else {
          load_vec<E, V>(in + c, v[i]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(v[i][j], v[i][j], ss);
      }
    }
    const float r = inv_rms(g.sum(ss), d, a.eps);
    if (!COMBINE) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (g.tid + i * a.tpr) * V;
        if (c < d) {
          float x[V];
          load_vec<E, V>(w + c, x);
#pragma unroll
          for (int j = 0; j < V; ++j) x[j] = v[i][j] * r * x[j];
          store_vec<E, V>(static_cast<E*>(a.h) + t * d + c, x);
        }
      }
      continue;
    }
    const E* gate = a.gate ? static_cast<const E*>(a.gate) + (t / a.gate_group) * d : nullptr;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (g.tid + i * a.tpr) * V;
      if (c < d) {
        if (a.y) store_vec<E, V>(static_cast<E*>(a.y) + t * d + c, v[i]);
        float x[V], u[V];
        load_vec<E, V>(w + c, x);
        load_vec<E, V>(static_cast<const E*>(a.u) + t * d + c, u);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = v[i][j] * r * x[j];
        if (gate) {
          load_vec<E, V>(gate + c, x);
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] *= x[j];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[i][j] = fmaf(a.res, u[j], v[i][j]);
          ss = fmaf(v[i][j], v[i][j], ss);
        }
        store_vec<E, V>(static_cast<E*>(a.h) + t * d + c, v[i]);
      }
    }
    if (a.w_next) {
      const float rn = inv_rms(g.sum(ss), d, a.eps);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (g.tid + i * a.tpr) * V;
        if (c < d) {
          float x[V];
          load_vec<E, V>(static_cast<const E*>(a.w_next) + c, x);
#pragma unroll
          for (int j = 0; j < V; ++j) x[j] = v[i][j] * rn * x[j];
          store_vec<E, V>(static_cast<E*>(a.x_next) + t * d + c, x);
        }
      }
    }
  }
}

struct BwdArgs {
  const void* v;         // [T, d]: the normalised rows' input (u before the layer, y behind it)
  const void* w;         // [d]
  const void* gate;      // [n_gate, d] or null
  const void* up;        // [T, d]: upstream gradient of the norm's output (or of h)
  const void* add;       // [T, d] or null: res * add joins the row's gradient
  void* dv;              // [T, d]
  void* dgate;           // [n_gate, d] with gate
  float* part_w;         // [gridDim.x, d]
  float* part_g;         // [units, d] when a gate row's tokens are split over units
  int T, d;
  int group;             // tokens of a gate row (T without gate)
  int split;             // units a gate row's tokens are split into
  int rows;              // tokens of a unit
  int units;
  int tpr;
  float eps, res;
};

// A unit is a run of tokens of one gate row; units are strided over the
// blocks.  Every thread keeps the sums of its columns over the unit's tokens
// (the gate's gradient) and over all of the block's (the weight's); both are
// joined in a fixed order, so two runs agree bit for bit.  With one warp per
// row a block's row groups share the unit's tokens and join their sums in
// shared memory at the unit's end.
template <typename E, int V, int VPT, bool GATE>
__global__ void __launch_bounds__(VPT* V > 8 ? 512 : MAX_THREADS) k_norm_bwd(const BwdArgs a) {
  grid_dep_sync();
  extern __shared__ float joined[];   // one warp per row: [row groups][d]
  __shared__ float2 red[2][32];
  const int rows_here = blockDim.x / a.tpr, mine = threadIdx.x / a.tpr;
  RowGroup g{a.tpr, (int)threadIdx.x % a.tpr, red, 0};
  const int d = a.d;
  const E* w = static_cast<const E*>(a.w);
  float aw[VPT][V];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) aw[i][j] = 0.f;

  // the row groups' sums of the block, complete in row group 0's threads
  auto join = [&](float (&s)[VPT][V]) {
    if (rows_here == 1) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (g.tid + i * a.tpr) * V;
      if (c < d)
#pragma unroll
        for (int j = 0; j < V; ++j) joined[mine * d + c + j] = s[i][j];
    }
    __syncthreads();
    if (mine == 0)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (g.tid + i * a.tpr) * V;
        if (c < d)
          for (int q = 1; q < rows_here; ++q)
#pragma unroll
            for (int j = 0; j < V; ++j) s[i][j] += joined[q * d + c + j];
      }
  };

  for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const int k = unit / a.split;
    const long long t0 = (long long)k * a.group + (long long)(unit - k * a.split) * a.rows;
    const long long t1 = min(min(t0 + a.rows, (long long)(k + 1) * a.group), (long long)a.T);
    float ag[VPT][V];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) ag[i][j] = 0.f;
    for (long long t = t0 + mine; t < t1; t += rows_here) {
      float v[VPT][V], up[VPT][V];
      float ss = 0.f, sc = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (g.tid + i * a.tpr) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = up[i][j] = 0.f;
        if (c < d) {
          load_vec<E, V>(static_cast<const E*>(a.v) + t * d + c, v[i]);
          load_vec<E, V>(static_cast<const E*>(a.up) + t * d + c, up[i]);
          float x[V], gt[V];
          load_vec<E, V>(w + c, x);
          if (GATE) load_vec<E, V>(static_cast<const E*>(a.gate) + (long long)k * d + c, gt);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            ss = fmaf(v[i][j], v[i][j], ss);
            sc = fmaf(v[i][j], up[i][j] * x[j] * (GATE ? gt[j] : 1.f), sc);
          }
        }
      }
      const float2 s = g.sum2(ss, sc);
      const float r = inv_rms(s.x, d, a.eps);
      const float m = r * r * (s.y / (float)d);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (g.tid + i * a.tpr) * V;
        if (c < d) {
          float x[V], gt[V], o[V];
          load_vec<E, V>(w + c, x);
          if (GATE) load_vec<E, V>(static_cast<const E*>(a.gate) + (long long)k * d + c, gt);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float un = up[i][j] * (v[i][j] * r);    // upstream * n
            aw[i][j] = fmaf(un, GATE ? gt[j] : 1.f, aw[i][j]);
            if (GATE) ag[i][j] += un;
            o[j] = r * (up[i][j] * x[j] * (GATE ? gt[j] : 1.f) - v[i][j] * m);
          }
          if (a.add) {
            float y[V];
            load_vec<E, V>(static_cast<const E*>(a.add) + t * d + c, y);
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = fmaf(a.res, y[j], o[j]);
          }
          store_vec<E, V>(static_cast<E*>(a.dv) + t * d + c, o);
        }
      }
    }
    if (GATE) {
      join(ag);
      if (mine == 0)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = (g.tid + i * a.tpr) * V;
          if (c < d) {
            if (a.split == 1) {
              float x[V];
              load_vec<E, V>(w + c, x);
#pragma unroll
              for (int j = 0; j < V; ++j) x[j] *= ag[i][j];
              store_vec<E, V>(static_cast<E*>(a.dgate) + (long long)k * d + c, x);
            } else {
#pragma unroll
              for (int j = 0; j < V; ++j) a.part_g[(long long)unit * d + c + j] = ag[i][j];
            }
          }
        }
    }
  }
  join(aw);
  if (mine == 0)
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (g.tid + i * a.tpr) * V;
      if (c < d)
#pragma unroll
        for (int j = 0; j < V; ++j) a.part_w[(long long)blockIdx.x * d + c + j] = aw[i][j];
    }
}

// Rows too long for the registers of a block (see norm_shape): the same sums
// and outputs in loops over the columns, one block per row, the row read again
// (from L2) for each pass.
template <typename E, int V, bool COMBINE>
__global__ void __launch_bounds__(MAX_THREADS) k_norm_fwd_wide(const FwdArgs a) {
  grid_dep_sync();
  __shared__ float2 red[2][32];
  RowGroup g{(int)blockDim.x, (int)threadIdx.x, red, 0};
  const int d = a.d, step = (int)blockDim.x * V;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E* in = COMBINE ? static_cast<const E*>(a.slots) + t * a.S * d
                          : static_cast<const E*>(a.u) + t * d;
    auto input = [&](int c, float (&v)[V]) {
      load_vec<E, V>(in + c, v);
      for (int s = 1; COMBINE && s < a.S; ++s) {
        float x[V];
        load_vec<E, V>(in + (long long)s * d + c, x);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += x[j];
      }
    };
    const E* gate = COMBINE && a.gate
                        ? static_cast<const E*>(a.gate) + (t / a.gate_group) * d
                        : nullptr;
    // the unrounded h (k_norm: x) of V columns
    auto output = [&](int c, float r, float (&v)[V]) {
      float x[V];
      input(c, v);
      load_vec<E, V>(static_cast<const E*>(a.w) + c, x);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = v[j] * r * x[j];
      if (!COMBINE) return;
      if (gate) {
        load_vec<E, V>(gate + c, x);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= x[j];
      }
      load_vec<E, V>(static_cast<const E*>(a.u) + t * d + c, x);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = fmaf(a.res, x[j], v[j]);
    };
    float v[V];
    float ss = 0.f;
    for (int c = threadIdx.x * V; c < d; c += step) {
      input(c, v);
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(v[j], v[j], ss);
      if (COMBINE && a.y) store_vec<E, V>(static_cast<E*>(a.y) + t * d + c, v);
    }
    const float r = inv_rms(g.sum(ss), d, a.eps);
    ss = 0.f;
    for (int c = threadIdx.x * V; c < d; c += step) {
      output(c, r, v);
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(v[j], v[j], ss);
      store_vec<E, V>(static_cast<E*>(a.h) + t * d + c, v);
    }
    if (!COMBINE || !a.w_next) continue;
    const float rn = inv_rms(g.sum(ss), d, a.eps);
    for (int c = threadIdx.x * V; c < d; c += step) {
      float x[V];
      output(c, r, v);
      load_vec<E, V>(static_cast<const E*>(a.w_next) + c, x);
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = v[j] * rn * x[j];
      store_vec<E, V>(static_cast<E*>(a.x_next) + t * d + c, x);
    }
  }
}

// The column sums are kept in the block's own partial rows (a thread always
// meets the same columns), part_g of a gate row that is not split in row
// blockIdx.x.
template <typename E, int V, bool GATE>
__global__ void __launch_bounds__(MAX_THREADS) k_norm_bwd_wide(const BwdArgs a) {
  grid_dep_sync();
  __shared__ float2 red[2][32];
  RowGroup g{(int)blockDim.x, (int)threadIdx.x, red, 0};
  const int d = a.d, step = (int)blockDim.x * V;
  float* pw = a.part_w + (long long)blockIdx.x * d;
  for (int c = threadIdx.x * V; c < d; c += step)
#pragma unroll
    for (int j = 0; j < V; ++j) pw[c + j] = 0.f;
  for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const int k = unit / a.split;
    const long long t0 = (long long)k * a.group + (long long)(unit - k * a.split) * a.rows;
    const long long t1 = min(min(t0 + a.rows, (long long)(k + 1) * a.group), (long long)a.T);
    float* pg = a.part_g + (long long)(a.split == 1 ? blockIdx.x : unit) * d;
    if (GATE)
      for (int c = threadIdx.x * V; c < d; c += step)
#pragma unroll
        for (int j = 0; j < V; ++j) pg[c + j] = 0.f;
    for (long long t = t0; t < t1; ++t) {
      // v and c = upstream * w * gate of V columns, and the upstream times the gate
      auto input = [&](int c, float (&v)[V], float (&up)[V], float (&cc)[V], float (&gt)[V]) {
        float x[V];
        load_vec<E, V>(static_cast<const E*>(a.v) + t * d + c, v);
        load_vec<E, V>(static_cast<const E*>(a.up) + t * d + c, up);
        load_vec<E, V>(static_cast<const E*>(a.w) + c, x);
        if (GATE) load_vec<E, V>(static_cast<const E*>(a.gate) + (long long)k * d + c, gt);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (!GATE) gt[j] = 1.f;
          cc[j] = up[j] * x[j] * gt[j];
        }
      };
      float v[V], up[V], cc[V], gt[V];
      float ss = 0.f, sc = 0.f;
      for (int c = threadIdx.x * V; c < d; c += step) {
        input(c, v, up, cc, gt);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          ss = fmaf(v[j], v[j], ss);
          sc = fmaf(v[j], cc[j], sc);
        }
      }
      const float2 s = g.sum2(ss, sc);
      const float r = inv_rms(s.x, d, a.eps);
      const float m = r * r * (s.y / (float)d);
      for (int c = threadIdx.x * V; c < d; c += step) {
        input(c, v, up, cc, gt);
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float un = up[j] * (v[j] * r);
          pw[c + j] = fmaf(un, gt[j], pw[c + j]);
          if (GATE) pg[c + j] += un;
          o[j] = r * (cc[j] - v[j] * m);
        }
        if (a.add) {
          float x[V];
          load_vec<E, V>(static_cast<const E*>(a.add) + t * d + c, x);
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] = fmaf(a.res, x[j], o[j]);
        }
        store_vec<E, V>(static_cast<E*>(a.dv) + t * d + c, o);
      }
    }
    if (GATE && a.split == 1)
      for (int c = threadIdx.x * V; c < d; c += step) {
        float x[V];
        load_vec<E, V>(static_cast<const E*>(a.w) + c, x);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] *= pg[c + j];
        store_vec<E, V>(static_cast<E*>(a.dgate) + (long long)k * d + c, x);
      }
  }
}

// Column sums of the partial rows: dw from n_part rows (blockIdx.y = 0), and
// for a split gate the rows of gate row k = blockIdx.y - 1, times w.  A block
// sums 32 columns with 32 slices of the rows, joined in order.
template <typename E>
__global__ void __launch_bounds__(1024) k_norm_join(const float* part_w, int n_part, float* dw,
                                                    const float* part_g, int split, const E* w,
                                                    E* dgate, int d) {
  grid_dep_sync();
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  const int k = (int)blockIdx.y - 1;
  const float* p = k < 0 ? part_w : part_g + (long long)k * split * d;
  const int n = k < 0 ? n_part : split;
  float v = 0.f;
  if (c < d)
    for (int i = threadIdx.y; i < n; i += 32) v += p[(long long)i * d + c];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int co = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && co < d) {
    if (k < 0) dw[co] = v;
    else dgate[(long long)k * d + co] = Elem<E>::put(v * Elem<E>::get(w[co]));
  }
}

}  // namespace norm
}  // namespace moe
