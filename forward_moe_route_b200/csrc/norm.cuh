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
// With at most 30 operations per element read, memory is the floor.  The end of a
// block and the backward before the layer come within 15 to 30% of it in batches.
// Farther off are the norm before the layer, which asks for nothing ahead of the row
// at hand (16384 x 7168 bf16 137 us, floor 72), and the backward with gate rows
// (below).
//   k_norm_fwd     a row held by one warp (up to 4 vectors of 16 bytes a lane) or
//                  by one block, its sums warp shuffles and one exchange in shared
//                  memory
//   k_norm_stream  many tokens: rows through a ring in shared memory, loads in
//                  flight while a token's sums are taken (16384 tokens x 9 rows of
//                  7168 bf16 531 us, 5.7 TB/s; k_norm_fwd 554 us)
//   k_norm_bwd     the same ring for several rows a block (8192 x 5120 bf16 with
//                  the residual 64 us, 5.2 TB/s; with the loads of a row behind the
//                  row before it 119 us.  Gate rows of 1024 tokens are farther off:
//                  8191 x 2048 bf16 30 us, floor 15, its warps at their row sums and
//                  the blocks' sums to be joined; 8192 columns with whole gate rows
//                  leave the ring one stage: 8192 rows 106 us, floor 63)
//   *_wide         rows beyond a block's registers, in loops over the columns
#pragma once

#include "bulk.cuh"
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

// V elements as they are stored: half the registers of their fp32 values in bf16.
template <typename E, int V>
struct Raw {
  static constexpr int WORDS = V == 1 ? 1 : 4;
  uint32_t word[WORDS];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) word[i] = 0u;
  }
  __device__ __forceinline__ void load(const E* p) {
    if constexpr (V == 1) {
      if constexpr (sizeof(E) == 4) word[0] = *reinterpret_cast<const uint32_t*>(p);
      else word[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      word[0] = x.x;
      word[1] = x.y;
      word[2] = x.z;
      word[3] = x.w;
    }
  }
  // the V elements from column c of a row of d in shared memory, zeros behind its
  // end.  Single elements are read without a branch (at the row's last one, which
  // a select then drops): eight branches a row took most of the instructions.
  __device__ __forceinline__ void load_column(const E* row, int c, int d) {
    if constexpr (V == 1) {
      load(row + min(c, d - 1));
      word[0] = c < d ? word[0] : 0u;
    } else {
      if (c < d) load(row + c);
      else zero();
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(E) == 4) return __uint_as_float(word[j]);
    else return __uint_as_float((j & 1) ? word[j >> 1] & 0xffff0000u : word[j >> 1] << 16);
  }
};

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

// Rows of d elements in shared memory, by bulk copies, which go by 16 bytes.  Rows of
// whole vectors (V > 1) are copied as they are.  Others (V = 1) start and end inside
// a 16-byte piece: the pieces that cover the row are copied, its elements then stand
// `shift` bytes from the copy's start; a piece that reaches behind the array (of
// `total` elements) is not, its elements are written one by one.
template <typename E, int V>
struct SharedRow {
  static constexpr uint32_t SZ = sizeof(E);
  __host__ __device__ static constexpr uint32_t room(int d) {
    return V > 1 ? d * SZ : (d * SZ + 15) / 16 * 16 + 16;
  }
  static __device__ __forceinline__ uint32_t shift(long long at) {
    return V > 1 ? 0u : (uint32_t)(at * SZ) & 15u;
  }
  // bytes of the copy of the row that begins with element `at`
  static __device__ __forceinline__ uint32_t bytes(long long at, int d, long long total) {
    if (V > 1) return d * SZ;
    const long long lo = at * SZ & ~15ll;
    const long long hi = min(((at + d) * SZ + 15) & ~15ll, total * SZ & ~15ll);
    return hi > lo ? (uint32_t)(hi - lo) : 0u;
  }
  // before the arrival that makes the row complete
  static __device__ __forceinline__ void last_elements(uint8_t* to, const E* array, long long at,
                                                       int d, long long total) {
    if (V > 1) return;
    const long long lo = at * SZ & ~15ll, end = (lo + bytes(at, d, total)) / SZ;
    for (long long e = end > at ? end : at; e < at + d; ++e)
      *reinterpret_cast<E*>(to + (e * SZ - lo)) = array[e];
  }
  static __device__ __forceinline__ void copy(uint8_t* to, const E* array, long long at, int d,
                                              long long total, uint64_t* bar) {
    const uint32_t n = bytes(at, d, total);
    const long long lo = V > 1 ? at * SZ : at * SZ & ~15ll;
    if (n) bulk_load_1d(to, reinterpret_cast<const uint8_t*>(array) + lo, n, bar);
  }
};

struct FwdArgs {
  const void* u;         // [T, d]: the input of moe_norm; the residual of moe_combine_norm
  const void* slots;     // [T, S, d]
  const void* w;         // [d]
  const void* gate;      // [n_gate, d] or null
  const void* w_next;    // [d] or null
  void* h;               // [T, d]: the result of moe_norm
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
    const E* gate =
        COMBINE && a.gate ? static_cast<const E*>(a.gate) + (t / a.gate_group) * d : nullptr;
    // what follows the first sum is asked for before it, where registers allow
    constexpr bool EARLY = V > 1 && VPT == 1;
    Raw<E, V> early[EARLY ? 4 : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (g.tid + i * a.tpr) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = 0.f;
      if (c < d) {
        if constexpr (EARLY) {
          early[0].load(w + c);
          if (COMBINE) {
            early[1].load(static_cast<const E*>(a.u) + t * d + c);
            if (gate) early[2].load(gate + c);
            if (a.w_next) early[3].load(static_cast<const E*>(a.w_next) + c);
          }
        }
        if (COMBINE) {
#pragma unroll (VPT == 1 ? 8 : 4)
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
    // V values of operand `which`, whose column c is at p + c
    auto operand = [&](int which, const E* p, int c, float (&x)[V]) {
      if constexpr (EARLY) {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = early[which].get(j);
      } else {
        load_vec<E, V>(p + c, x);
      }
    };
    const float r = inv_rms(g.sum(ss), d, a.eps);
    if (!COMBINE) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (g.tid + i * a.tpr) * V;
        if (c < d) {
          float x[V];
          operand(0, w, c, x);
#pragma unroll
          for (int j = 0; j < V; ++j) x[j] = v[i][j] * r * x[j];
          store_vec<E, V>(static_cast<E*>(a.h) + t * d + c, x);
        }
      }
      continue;
    }
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (g.tid + i * a.tpr) * V;
      if (c < d) {
        if (a.y) store_vec<E, V>(static_cast<E*>(a.y) + t * d + c, v[i]);
        float x[V], u[V];
        operand(0, w, c, x);
        operand(1, static_cast<const E*>(a.u) + t * d, c, u);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = v[i][j] * r * x[j];
        if (gate) {
          operand(2, gate, c, x);
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
          operand(3, static_cast<const E*>(a.w_next), c, x);
#pragma unroll
          for (int j = 0; j < V; ++j) x[j] = v[i][j] * rn * x[j];
          store_vec<E, V>(static_cast<E*>(a.x_next) + t * d + c, x);
        }
      }
    }
  }
}

// moe_combine_norm of many tokens (and moe_norm of rows that are not whole vectors).
// The S expert rows and the residual's row of token after token stream through a
// ring in shared memory, one row a stage: a warp of its own issues the copies, so
// loads go on while the other warps are at a token's sums and outputs.  Arithmetic
// as in k_norm_fwd; w and w_next stay in registers.
constexpr int STREAM_STAGES = 16;      // at most
template <typename E, int V, int VPT, bool COMBINE>
__global__ void __launch_bounds__(V > 1 && VPT == 4 ? 544 : MAX_THREADS)
    k_norm_stream(const FwdArgs a, int stages) {
  using Row = SharedRow<E, V>;
  grid_dep_sync();
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ float red[2][32];
  __shared__ uint64_t full[STREAM_STAGES], empty[STREAM_STAGES];
  __shared__ int abort_word;
  const int tid = (int)threadIdx.x, d = a.d, S = COMBINE ? a.S : 0;
  const int nw = a.tpr >> 5;                       // warps at the rows; one more copies
  const uint32_t row_bytes = Row::room(d);
  const long long rows = a.T;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], nw);
    }
    abort_word = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  int stage = 0;
  uint32_t phase = 0;
  auto advance = [&]() {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  };
  if (tid >= a.tpr) {
    if (elect_one()) {
      bool ok = true;
      for (long long t = blockIdx.x; t < a.T && ok; t += gridDim.x)
        for (int s = 0; s <= S && ok; ++s) {
          ok = mbar_wait(&empty[stage], phase ^ 1u, &abort_word);
          if (!ok) break;
          const E* array = static_cast<const E*>(s < S ? a.slots : a.u);
          const long long at = (s < S ? t * S + s : t) * d, total = rows * d * (s < S ? S : 1);
          uint8_t* to = dyn + (size_t)stage * row_bytes;
          Row::last_elements(to, array, at, d, total);
          mbar_arrive_expect_tx(&full[stage], Row::bytes(at, d, total));
          Row::copy(to, array, at, d, total, &full[stage]);
          advance();
        }
      bulk_drain(full, stage, phase, stages);   // of use when the readers gave up
    }
    return;
  }
  int buf = 0;
  auto sum = [&](float x) {
    x = warp_sum(x);
    if (lane_id() == 0) red[buf][warp_id()] = x;
    asm volatile("bar.sync 1, %0;" ::"r"(a.tpr) : "memory");
    x = lane_id() < nw ? red[buf][lane_id()] : 0.f;
    buf ^= 1;
    return warp_sum(x);
  };
  Raw<E, V> w[VPT], w_next[VPT], gate[VPT], x[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (tid + i * a.tpr) * V;
    if (c < d) {
      w[i].load(static_cast<const E*>(a.w) + c);
      if (COMBINE && a.w_next) w_next[i].load(static_cast<const E*>(a.w_next) + c);
    }
  }
  // the next row of the ring into x (a wait that ran out is reported, the results
  // are void, and the copying warp is left to give up too)
  auto take = [&](long long element) {
    const bool there = mbar_wait(&full[stage], phase, &abort_word);
    const E* row =
        reinterpret_cast<const E*>(dyn + (size_t)stage * row_bytes + Row::shift(element));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      x[i].load_column(row, (tid + i * a.tpr) * V, d);
    }
    __syncwarp();
    if (lane_id() == 0 && there) mbar_arrive(&empty[stage]);
    advance();
  };
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (COMBINE && a.gate) {
      const E* g = static_cast<const E*>(a.gate) + (long long)((int)t / a.gate_group) * d;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * a.tpr) * V;
        if (c < d) gate[i].load(g + c);
      }
    }
    float v[VPT][V];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = 0.f;
    for (int s = 0; s < S; ++s) {
      take((t * S + s) * d);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] += x[i].get(j);
    }
    if (!COMBINE) {
      take(t * d);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = x[i].get(j);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (tid + i * a.tpr) * V;
      if (COMBINE && a.y && c < d) store_vec<E, V>(static_cast<E*>(a.y) + t * d + c, v[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    const float r = inv_rms(sum(ss), d, a.eps);
    if (!COMBINE) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * a.tpr) * V;
        if (c < d) {
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] = v[i][j] * r * w[i].get(j);
          store_vec<E, V>(static_cast<E*>(a.h) + t * d + c, v[i]);
        }
      }
      continue;
    }
    take(t * d);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (tid + i * a.tpr) * V;
      if (c < d) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[i][j] = v[i][j] * r * w[i].get(j);
          if (a.gate) v[i][j] *= gate[i].get(j);
          v[i][j] = fmaf(a.res, x[i].get(j), v[i][j]);
          ss = fmaf(v[i][j], v[i][j], ss);
        }
        store_vec<E, V>(static_cast<E*>(a.h) + t * d + c, v[i]);
      }
    }
    if (a.w_next) {
      const float rn = inv_rms(sum(ss), d, a.eps);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * a.tpr) * V;
        if (c < d) {
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] = v[i][j] * rn * w_next[i].get(j);
          store_vec<E, V>(static_cast<E*>(a.x_next) + t * d + c, v[i]);
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
  int alone;             // 1: a unit is one row group's, 0: the block's row groups share it
  int stages;            // rows of the ring of each row group
  float eps, res;
};

// A unit is a run of tokens of one gate row; units are strided over the blocks,
// which share each among their row groups (or, when gate rows have few tokens,
// over the row groups).  Every thread sums upstream * n of its columns over the
// unit, s.  The unit's share of the gate's gradient is w s and of the weight's
// gate s, so one sum serves both: a unit that is a whole gate row writes its
// gate gradient and adds gate s to the thread's sum for dw, the units of a split
// gate row leave s to the join.  All sums are joined in a fixed order: two runs
// agree bit for bit.
//
// Rows reach the threads through shared memory: each row group
// keeps `stages` rows of its operands in flight with bulk copies, across units,
// and refills a stage as soon as its threads have the row in registers (behind
// the barrier of the row's sums).
//
// What a row costs beside its elements (the barrier, the sums, the waits) is
// about 80 instructions a thread, so a thread takes up to 4 vectors of a row,
// which it holds as they are stored, and a block of up to 512 threads several
// rows at a time.  One block on each SM.
//
// A gate row for every token needs no units: it comes through the ring as a third
// operand, its gradient leaves with the row, and s collects gate * upstream * n.
constexpr int BWD_THREADS = 512;
enum GateKind { GATE_NONE = 0, GATE_ROWS = 1, GATE_EACH = 2 };
template <typename E, int V, int VPT, int GATE_KIND>
__global__ void __launch_bounds__(BWD_THREADS, 1) k_norm_bwd(const BwdArgs a) {
  using Row = SharedRow<E, V>;
  constexpr bool GATE = GATE_KIND == GATE_ROWS, EACH = GATE_KIND == GATE_EACH;
  grid_dep_sync();
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ float red[2][2][32];
  __shared__ uint64_t full[16][8];
  __shared__ int abort_word;
  const int rows_here = blockDim.x / a.tpr, mine = threadIdx.x / a.tpr;
  const int tid = (int)threadIdx.x % a.tpr;
  const int d = a.d;
  const E* w = static_cast<const E*>(a.w);
  const uint32_t row_bytes = Row::room(d);
  constexpr bool ADD = GATE_KIND == GATE_NONE;   // the residual's gradient joins moe_norm's only
  const bool add = ADD && a.add != nullptr;
  const int parts = add || EACH ? 3 : 2;
  const uint32_t stage_bytes = parts * row_bytes;
  uint8_t* ring = dyn + (size_t)mine * a.stages * stage_bytes;
  // the row groups' sums [rows_here][d], in the ring's place when it has run dry
  // and behind it with gates; with whole gate rows shared by the block the sum
  // for dw [d] follows
  float* joined = reinterpret_cast<float*>(
      dyn + (GATE ? (size_t)rows_here * a.stages * stage_bytes : 0));
  const bool keep = GATE && a.split == 1;   // dw collected over the units
  float* acc = a.alone ? joined + mine * d : joined + rows_here * d;
  if (tid == 0)
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[mine][s], 1);
  if (threadIdx.x == 0) abort_word = 0;
  fence_barrier_init();
  fence_proxy_async_smem();
  __syncthreads();

  // the rows of this row group, unit after unit
  struct Place {
    int unit;
    long long t, t1;
  };
  const int unit_step = a.alone ? (int)gridDim.x * rows_here : (int)gridDim.x;
  const int first = a.alone ? 0 : mine, step = a.alone ? 1 : rows_here;
  auto enter = [&](Place& p) {
    const int k = p.unit / a.split;
    const long long t0 = (long long)k * a.group + (long long)(p.unit - k * a.split) * a.rows;
    p.t = t0 + first;
    p.t1 = min(min(t0 + a.rows, (long long)(k + 1) * a.group), (long long)a.T);
  };
  Place here;
  here.unit = a.alone ? (int)blockIdx.x * rows_here + mine : (int)blockIdx.x;
  here.t = here.t1 = 0;
  if (here.unit < a.units) enter(here);
  // thread 0 of the row group fetches rows ahead
  Place ahead = here;
  int into = 0;          // below 0 (see the rows' loop) once a wait has run out
  auto fetch = [&]() {
    while (ahead.unit < a.units && ahead.t >= ahead.t1) {
      ahead.unit += unit_step;
      if (ahead.unit < a.units) enter(ahead);
    }
    if (ahead.unit >= a.units) return;
    uint64_t* bar = &full[mine][into];
    uint8_t* to = ring + (size_t)into * stage_bytes;
    if (++into == a.stages) into = 0;
    const long long at = ahead.t * d, total = (long long)a.T * d;
    const E* part[3] = {static_cast<const E*>(a.v), static_cast<const E*>(a.up),
                        static_cast<const E*>(EACH ? a.gate : a.add)};
    for (int i = 0; i < parts; ++i) Row::last_elements(to + i * row_bytes, part[i], at, d, total);
    mbar_arrive_expect_tx(bar, parts * Row::bytes(at, d, total));
    for (int i = 0; i < parts; ++i) Row::copy(to + i * row_bytes, part[i], at, d, total, bar);
    ahead.t += step;
  };
  if (tid == 0)
    for (int s = 0; s < a.stages; ++s) fetch();

  const int lane = lane_id(), nw = a.tpr >> 5, w0 = mine * nw;
  int buf = 0, stage = 0;
  uint32_t phase = 0;
  // both sums over the row group; the lower half of a warp reduces x, the upper y
  auto sum2 = [&](float x, float y) {
    const bool up_half = lane >= 16;
    float z = (up_half ? y : x) + __shfl_xor_sync(0xffffffffu, up_half ? x : y, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (a.tpr == 32) {
      __syncwarp();
      return make_float2(__shfl_sync(0xffffffffu, z, 0), __shfl_sync(0xffffffffu, z, 16));
    }
    if ((lane & 15) == 0) red[buf][lane >> 4][warp_id()] = z;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + mine), "r"(a.tpr) : "memory");
    x = y = 0.f;
    for (int i = 0; i < nw; ++i) {
      x += red[buf][0][w0 + i];
      y += red[buf][1][w0 + i];
    }
    buf ^= 1;
    return make_float2(x, y);
  };
  // V / Q accesses of Q floats cover a vector
  constexpr int Q = V == 1 ? 1 : 4;
  float s[VPT][V];
  // put(c, x) with the sums over the row groups of Q columns from c on, by every
  // thread of the block for its share of the columns; `mine_in`: the row groups'
  // sums are in `joined` already
  auto join = [&](bool mine_in, auto put) {
    __syncthreads();
    if (!mine_in) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * a.tpr) * V;
        if (c < d)
#pragma unroll
          for (int q = 0; q < V; q += Q)
            store_vec<float, Q>(joined + mine * d + c + q,
                                *reinterpret_cast<const float(*)[Q]>(&s[i][q]));
      }
      __syncthreads();
    }
    for (int c = threadIdx.x * Q; c < d; c += blockDim.x * Q) {
      float x[Q];
      load_vec<float, Q>(joined + c, x);
      for (int g = 1; g < rows_here; ++g) {
        float y[Q];
        load_vec<float, Q>(joined + g * d + c, y);
#pragma unroll
        for (int j = 0; j < Q; ++j) x[j] += y[j];
      }
      put(c, x);
    }
  };
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) s[i][j] = 0.f;
  if (keep && a.alone)
    for (int c = tid; c < d; c += a.tpr) acc[c] = 0.f;
  else if (keep)
    for (int c = threadIdx.x; c < d; c += blockDim.x) acc[c] = 0.f;
  if (keep) __syncthreads();

  for (; here.unit < a.units; here.unit += unit_step) {
    enter(here);
    const int k = here.unit / a.split;
    const E* gate = GATE ? static_cast<const E*>(a.gate) + (long long)k * d : nullptr;
    // w (as stored), or w * gate
    Raw<E, V> wr[GATE ? 1 : VPT];
    float wg[GATE ? VPT : 1][V];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (tid + i * a.tpr) * V;
      if (GATE)
#pragma unroll
        for (int j = 0; j < V; ++j) s[i][j] = 0.f;
      if (c < d) {
        if constexpr (GATE) {
          Raw<E, V> x, g;
          x.load(w + c);
          g.load(gate + c);
#pragma unroll
          for (int j = 0; j < V; ++j) wg[i][j] = x.get(j) * g.get(j);
        } else {
          wr[i].load(w + c);
        }
      }
    }
    auto weight = [&](int i, int j) {
      if constexpr (GATE) return wg[i][j];
      else return wr[i].get(j);
    };
    for (; here.t < here.t1; here.t += step) {
      const uint8_t* at = ring + (size_t)stage * stage_bytes + Row::shift(here.t * d);
      // a wait that ran out is reported, the results from this row on are void, and
      // no more rows are fetched
      if (!mbar_wait(&full[mine][stage], phase, &abort_word) && into >= 0)
        into = -1 - 2 * into - (int)ring_parity(into, stage, phase);
      if (++stage == a.stages) {
        stage = 0;
        phase ^= 1u;
      }
      const E* v_row = reinterpret_cast<const E*>(at);
      const E* up_row = reinterpret_cast<const E*>(at + row_bytes);
      const E* more_row = reinterpret_cast<const E*>(at + 2 * row_bytes);
      // `more`: the residual's gradient, or the token's gate
      Raw<E, V> v[VPT], up[VPT], more[ADD || EACH ? VPT : 1];
      float ss = 0.f, sc = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * a.tpr) * V;
        if (c < d) {
          v[i].load(v_row + c);
          up[i].load(up_row + c);
          if constexpr (EACH) more[i].load(more_row + c);
          if constexpr (ADD) {
            if (add) more[i].load(more_row + c);
            else more[i].zero();
          }
#pragma unroll
          for (int j = 0; j < V; ++j) {
            ss = fmaf(v[i].get(j), v[i].get(j), ss);
            sc = fmaf(v[i].get(j), up[i].get(j) * weight(i, j) * (EACH ? more[i].get(j) : 1.f), sc);
          }
        }
      }
      const float2 q = sum2(ss, sc);
      if (tid == 0 && into >= 0) fetch();      // the stage is in registers
      const float r = inv_rms(q.x, d, a.eps);
      const float m = r * r * (q.y / (float)d);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * a.tpr) * V;
        if (c < d) {
          float o[V], dg[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float un = up[i].get(j) * (v[i].get(j) * r);    // upstream * n
            const float g = EACH ? more[i].get(j) : 1.f;
            s[i][j] = fmaf(un, g, s[i][j]);
            if constexpr (EACH) dg[j] = un * weight(i, j);
            o[j] = r * (up[i].get(j) * weight(i, j) * g - v[i].get(j) * m);
            if constexpr (ADD) o[j] = fmaf(a.res, more[i].get(j), o[j]);
          }
          if constexpr (EACH)
            store_vec<E, V>(static_cast<E*>(a.dgate) + here.t * d + c, dg);
          store_vec<E, V>(static_cast<E*>(a.dv) + here.t * d + c, o);
        }
      }
    }
    if (!GATE) continue;
    // acc += gate * x, the gate's gradient w * x, of Q columns
    auto finish = [&](int c, const float (&x)[Q]) {
      float o[Q];
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        acc[c + j] = fmaf(Elem<E>::get(gate[c + j]), x[j], acc[c + j]);
        o[j] = Elem<E>::get(w[c + j]) * x[j];
      }
      E* to = static_cast<E*>(a.dgate) + (long long)k * d + c;
#pragma unroll
      for (int j = 0; j < Q; ++j) to[j] = Elem<E>::put(o[j]);
    };
    if (!a.alone) {
      join(false, [&](int c, const float (&x)[Q]) {
        if (keep) finish(c, x);
        else store_vec<float, Q>(a.part_g + (long long)here.unit * d + c, x);
      });
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * a.tpr) * V;
        if (c < d)
#pragma unroll
          for (int q = 0; q < V; q += Q)
            finish(c + q, *reinterpret_cast<const float(*)[Q]>(&s[i][q]));
      }
    }
  }
  if (tid == 0 && into < 0) bulk_drain(full[mine], (-1 - into) >> 1, (-1 - into) & 1, a.stages);
  if (GATE && !keep) return;
  auto write = [&](int c, const float (&x)[Q]) {
    store_vec<float, Q>(a.part_w + (long long)blockIdx.x * d + c, x);
  };
  if (GATE && !a.alone) {
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += blockDim.x)
      a.part_w[(long long)blockIdx.x * d + c] = acc[c];
  } else {
    join(GATE, write);
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
    // the unrounded h (moe_norm: its result) of V columns
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

// Column sums of the partial rows.  blockIdx.y = 0: dw, from n_part rows; when
// those are the units of split gate rows, each times its gate (`gate` given).
// blockIdx.y = k + 1: the gradient of split gate row k, from its units, times w.
// A block sums 32 columns with 32 slices of the rows, joined in order.
constexpr int JOIN_SLICES = 32;
template <typename E>
__global__ void __launch_bounds__(32 * JOIN_SLICES)
    k_norm_join(const float* part_w, int n_part, float* dw, const float* part_g, int split,
                const E* w, const E* gate, E* dgate, int d) {
  grid_dep_sync();
  __shared__ float s[JOIN_SLICES][32];
  const int c = blockIdx.x * 32 + threadIdx.x;
  const int k = (int)blockIdx.y - 1;
  const float* p = k < 0 ? part_w : part_g + (long long)k * split * d;
  const int n = k < 0 ? n_part : split;
  float v = 0.f;
  if (c < d) {
    if (k < 0 && gate) {
#pragma unroll 5
      for (int i = threadIdx.y; i < n; i += JOIN_SLICES)
        v = fmaf(p[(long long)i * d + c], Elem<E>::get(gate[(long long)(i / split) * d + c]), v);
    } else {
#pragma unroll 5
      for (int i = threadIdx.y; i < n; i += JOIN_SLICES) v += p[(long long)i * d + c];
    }
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= d) return;
#pragma unroll
  for (int i = 1; i < JOIN_SLICES; ++i) v += s[i][threadIdx.x];
  if (k < 0) dw[c] = v;
  else dgate[(long long)k * d + c] = Elem<E>::put(v * Elem<E>::get(w[c]));
}

}  // namespace norm
}  // namespace moe
