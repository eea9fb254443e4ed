// Products grouped by expert over a ragged row list, with their gradients, on
// tcgen05 / TMEM, fed by TMA, on CTA pairs (tcgen05.mma.cta_group::2).
//
//   rows of group g: offsets[g] .. offsets[g+1] - 1, anywhere in the row list
//   y_r  = W_g x_r              k_grouped_mm<false>   (contracts over d_in)
//   dx_r = W_g^T dy_r           k_grouped_mm<true>    (contracts over d_out)
//   dW_g = sum_r dy_r x_r^T     k_grouped_dw          (contracts over the rows)
//
// All operands bf16, accumulation fp32: in TMEM over segments of the contraction, the
// segments added in registers (see MM_SEGMENT).
//
// k_grouped_mm computes D = (weights) x (rows)^T: 256 features on the UMMA M
// side, up to 256 rows of one group on the N side, so a group of few rows
// costs few columns and streams its weights once.  The weights are addressed
// through a three-dimensional tensor map [G, d_out, d_in], so a tile's edge is
// filled with zeros instead of the next expert's weights; for dx they are read
// MN-major (gemm_bwd.cuh), not transposed in memory.  Rows of the next group
// that a row tile brings along only reach accumulator columns nobody stores.
//
// k_grouped_dw has the ragged rows on the contraction side, where the next
// group's rows must not enter the sum, and zeros in one operand would not
// cancel a NaN in the other.  Rows are taken 64 a stage and 16 per UMMA; of a
// group's last stage only the 16-row steps that hold rows are issued, and in
// the last step the shared-memory lines behind the group's end are overwritten
// with zeros in both operands: that stage's copies complete on a barrier of
// their own in each CTA (one per stage), warp 3 clears the lines (fewer than 16)
// and the leader's, when the peer's has reported too, arrives for the stage in
// the producer's place.  (Having the peer's producer or tail warp arrive on the
// leader's barrier for every stage cost a remote arrival a stage: 631 us instead
// of 337 us at 16 groups of 1024 rows, 2048 x 7168.)  No row is copied or padded
// in global memory.
//
// Measured (24570 rows in 64 uneven groups, 2048 x 2816, 283 GFLOP): 230 us alone,
// 312 us in a loop under the power cap; uniform groups run within 5% of cuBLAS's
// batched product of the same sizes, both bound by the tensor cores' power.  The
// weight gradients of 24571 rows 2048 x 1408 in bf16 take 173 to 207 us: stores
// that share the SM's way to L2 with the operand loads cost a quarter of it (113 us
// without them, 150 us with them on equal groups), ragged group ends a tenth.
//
// Every CTA reads the offsets itself (no preparing launch); a group whose offsets
// decrease or leave [0, n_rows] is reported and treated as empty.
//
// Warp roles (384 threads): warp 0 TMA
// producer, warp 1 MMA issuer (leader CTA), warp 2 TMEM allocator, warp 3 tail
// rows (k_grouped_dw), the rest epilogue.  Two accumulators of 256 columns, taken by
// one segment after the other.
// Barriers and bounded waits as in gemm_t.cuh.
#pragma once

#include "bulk.cuh"
#include "common.cuh"
#include "gemm.cuh"
#include "gemm_bwd.cuh"
#include "gemm_t.cuh"

namespace moe {
namespace grouped {

constexpr int MAX_GROUPS = 1024;
constexpr int STAGES = 6;
constexpr uint32_t STAGE_BYTES = 32768;        // 16 KB of either operand per CTA
constexpr uint32_t HALF_STAGE = STAGE_BYTES / 2;
constexpr int ACC_COLS = 256;
constexpr int TMEM_COLS = 512;
constexpr uint32_t BAR_BYTES = (4 * STAGES + 6) * 8 + 16;
constexpr uint32_t TAB_BYTES = (3 * MAX_GROUPS + 1) * 4 + 12;

// The tensor cores add to the accumulator in TMEM by cutting sums off, not rounding
// them: every step of 16 loses up to a unit of 2^-23 of the running sum, always
// towards zero, so the error grows with the length (one group of 32768 rows: 3.8e-5 of
// a random weight gradient, 1.8e-4 of one whose products have one sign).  So TMEM
// accumulates segments of a contraction only, and the epilogue warps add these up in
// fp32 registers, rounded to nearest: the same gradients are then 4.9e-7 and 9.0e-7
// off at any length.  The next segment's products run meanwhile.
// Stages (of 64) of a segment.  dW, which may be fp32: 512 rows, as 1024 leave twice
// the error; 256 rows take the epilogue longer to add than the tensor cores to make
// (32768 rows 4096 x 4096 767 us, 1024 rows 756, 256 rows 903).  Outputs in bf16: 1024,
// 1e-6, far below their rounding; with 512 a tile's stores do not fit beside the next
// one's two segments (batch 250 us and 261 us, 64 groups of 384 rows 247 and 258).
constexpr int MM_SEGMENT = 16;
constexpr int DW_SEGMENT = 8;

// The first warpgroup gives registers to the two epilogue warpgroups, which hold 128
// sums a thread: 128 x 72 + 256 x 216 = 384 x 168, what a block of 384 threads with
// an SM to itself is launched with (the host checks).
constexpr int LAUNCH_REGS = 168;
constexpr int CTRL_REGS = 72;
constexpr int EPI_REGS = 216;
static_assert(128 * CTRL_REGS + 256 * EPI_REGS == 384 * LAUNCH_REGS, "register split");

// ---- rows on the N side -------------------------------------------------------------
constexpr int MM_THREADS = 384;
constexpr int MM_EPI_WARPS = 8;
constexpr uint32_t MM_XPOSE = 16 * 32 * 2;     // a warp's 16 rows x 32 features, bf16
// Row tiles of up to 256 rows, or of up to FEW_ROWS where groups are so small that
// the weights set the pace: a stage then keeps less for the rows, and ten of them
// instead of six hold more of the weight stream in flight.
constexpr int TILE_ROWS = 256;
constexpr int FEW_ROWS = 64;
__host__ __device__ constexpr int mm_stages(int tile_rows) { return tile_rows == FEW_ROWS ? 10 : STAGES; }
__host__ __device__ constexpr uint32_t mm_stage_bytes(int tile_rows) {
  return HALF_STAGE + tile_rows / 2 * 128;
}
constexpr uint32_t mm_smem(int tile_rows) {
  return 1024 + mm_stages(tile_rows) * mm_stage_bytes(tile_rows) + MM_EPI_WARPS * MM_XPOSE +
         (2 * mm_stages(tile_rows) + 6) * 8 + 16 + TAB_BYTES;
}

// ---- weight gradients -----------------------------------------------------------------
constexpr int DW_THREADS = 384;
constexpr int DW_EPI_WARPS = 8;
// a warp's staging: one block of 32 rows of 128 bytes.  (Two of them and five
// stages instead of six: the same on groups of 384 rows, 5% slower on 1024.)
constexpr uint32_t DW_STAGING = 4096;
constexpr uint32_t DW_STORE = DW_EPI_WARPS * DW_STAGING;
constexpr uint32_t DW_SMEM = 1024 + STAGES * STAGE_BYTES + DW_STORE + BAR_BYTES;
static_assert(mm_smem(TILE_ROWS) <= 232448 && mm_smem(FEW_ROWS) <= 232448 && DW_SMEM <= 232448,
              "shared memory of one block");

struct Args {
  const int* offsets;   // [n + 1]
  int n, n_rows;
  int feats, contract;  // k_grouped_mm: output features, contraction length
  int d_out, d_in;      // k_grouped_dw
  int accumulate;
  __nv_bfloat16* y;     // k_grouped_mm: [n_rows, feats]
};

__device__ __forceinline__ void tma_load_3d_pair(const CUtensorMap* map, uint32_t bar_cluster,
                                                 void* smem_dst, int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"((uint64_t)map), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, const void* smem_src, int32_t x,
                                           int32_t y, int32_t z) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
      " [%0, {%2, %3, %4}], [%1];" ::"l"((uint64_t)map),
      "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// rows r0 .. r1 - 1 of a group lie within the row list
__device__ __forceinline__ bool group_ok(int r0, int r1, int n_rows) {
  return r0 >= 0 && r1 >= r0 && r1 <= n_rows;
}

// k_grouped_mm cuts a group of r rows into ceil(r / ROWS) row tiles of equal
// height, rounded up to the 32 rows that the UMMA N goes by (r = 257: 160 + 97,
// not 256 + 1): 5 to 8% faster than full tiles and a rest on uneven groups, as
// a low tile costs the loads of its weights all the same.
template <int ROWS>
__device__ __forceinline__ int row_tiles(int rows) {
  return (rows + ROWS - 1) / ROWS;
}
template <int ROWS>
__device__ __forceinline__ int tile_height(int rows) {
  const int n = row_tiles<ROWS>(rows);
  return n ? ((rows + n - 1) / n + 31) & ~31 : 0;
}

// The group list in shared memory: first row and rows of each group, and the
// prefix of its row tiles.  One warp builds it.
template <int ROWS>
struct Groups {
  int *row0, *rows, *prefix;   // [n], [n], [n + 1]
  int n;
  __device__ __forceinline__ Groups(int* base, int count)
      : row0(base), rows(base + MAX_GROUPS), prefix(base + 2 * MAX_GROUPS), n(count) {}
  __device__ __forceinline__ void build(const int* offsets, int n_rows) {
    const int lane = lane_id();
    int carry = 0;
    for (int base = 0; base < n; base += 32) {
      const int g = base + lane;
      int r = 0;
      if (g < n) {
        const int r0 = offsets[g], r1 = offsets[g + 1];
        if (group_ok(r0, r1, n_rows)) r = r1 - r0;
        else if (blockIdx.x == 0) set_status(MOE_ERR_DEVICE_CHECK);
        row0[g] = r0;
        rows[g] = r;
      }
      const int v = row_tiles<ROWS>(r);
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (g < n) prefix[g] = carry + incl - v;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) prefix[n] = carry;
  }
};

template <bool W_MN, int ROWS>
__global__ void __launch_bounds__(MM_THREADS, 1)
    k_grouped_mm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                 const __grid_constant__ CUtensorMap tmX64,
                 const __grid_constant__ CUtensorMap tmX32, const Args a) {
  using namespace gemmt;   // cluster helpers of the pair kernels
  constexpr int TF = 256;             // features of a pair's tile
  constexpr int S = mm_stages(ROWS);
  constexpr uint32_t SB = mm_stage_bytes(ROWS);
  grid_dep_sync();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* xpose = smem + S * SB;
  uint64_t* full = reinterpret_cast<uint64_t*>(xpose + MM_EPI_WARPS * MM_XPOSE);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Groups<ROWS> gr(reinterpret_cast<int*>(tmem_slot + 4), a.n);

  const int warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  if (warp == 0) gr.build(a.offsets, a.n_rows);
  if (threadIdx.x == 32) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(&tfull[j], 1);
      mbar_init(&tempty[j], 2 * MM_EPI_WARPS * 32);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmX64);
    tma_prefetch_desc(&tmX32);
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();      // barrier initialisation is visible to the peer from here on
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int n_ft = (a.feats + TF - 1) / TF;
  const int num_kb = (a.contract + 63) / 64;
  const int total = gr.prefix[a.n] * n_ft;
  const int tile0 = (int)(blockIdx.x >> 1), tstep = (int)(gridDim.x >> 1);

  // feature tiles run fastest, so the pairs of one wave share a group's rows in L2
  struct Tile {
    int g, ft, row, rows, cols;   // group, feature tile, first row, its rows, UMMA N
  };
  auto locate = [&](int tile) {
    Tile t;
    const int rt = tile / n_ft;
    t.ft = tile - rt * n_ft;
    const int p = gemm::find_group(gr.prefix, a.n, rt);
    const int height = tile_height<ROWS>(gr.rows[p]), at = (rt - gr.prefix[p]) * height;
    t.g = p;
    t.row = gr.row0[p] + at;
    t.rows = min(height, gr.rows[p] - at);
    t.cols = (t.rows + 31) & ~31;
    return t;
  };

  if (warp < 4) {
    if constexpr (ROWS == TILE_ROWS)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTRL_REGS));
    if (warp == 0) {
      // ------------------------------------------------------------------ TMA producer (both CTAs)
      if (elect_one()) {
        int it = 0;
        bool ok = true;
        for (int tile = tile0; tile < total && ok; tile += tstep) {
          const Tile t = locate(tile);
          // the CTA's rows in boxes of 128, 64 and 32, no more than they need: a
          // tile of few rows is bound by its loads
          const int half = t.cols / 2, load = (half + 31) & ~31;
          const uint32_t bytes = HALF_STAGE + (uint32_t)load * 128u;
          const int xrow = t.row + (int)rank * half;
          const int f = t.ft * TF + (int)rank * 128;
          for (int kb = 0; kb < num_kb; ++kb, ++it) {
            const int s = it % S;
            const uint32_t ph = (uint32_t)(it / S) & 1u;
            if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag)) { ok = false; break; }
            uint8_t* sw = smem + (size_t)s * SB;
            const uint32_t fl = mapa(smem_u32(&full[s]), 0);
            if (leader) mbar_arrive_expect_tx(&full[s], 2 * bytes);
            const int k = kb * 64;
            if (W_MN) {
              tma_load_3d_pair(&tmW, fl, sw, f, k, t.g);
              tma_load_3d_pair(&tmW, fl, sw + gbwd::MN_BOX_BYTES, f + 64, k, t.g);
            } else {
              tma_load_3d_pair(&tmW, fl, sw, k, f, t.g);
            }
            uint8_t* sx = sw + HALF_STAGE;
            if (ROWS == TILE_ROWS && load == 128) {
              tma_load_2d_pair(&tmX, fl, sx, k, xrow);
            } else {
              if (ROWS == TILE_ROWS && (load & 64)) tma_load_2d_pair(&tmX64, fl, sx, k, xrow);
              if (load & 32)
                tma_load_2d_pair(&tmX32, fl, sx + (load & 64) * 128, k, xrow + (load & 64));
            }
          }
        }
        // the copies this CTA issued land before the block may leave (bounded)
        volatile int no_abort = 0;
        for (int j = (it - S > 0 ? it - S : 0); j < it; ++j)
          mbar_wait(&empty[j % S], (uint32_t)(j / S) & 1u, &no_abort);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------------ MMA issuer (leader)
      if (leader && elect_one()) {
        int it = 0, scount = 0;
        bool ok = true;
        for (int tile = tile0; tile < total && ok; tile += tstep) {
          const Tile t = locate(tile);
          const uint32_t idesc = umma_idesc(1, TF, t.cols) | (W_MN ? (1u << 15) : 0u);
          uint32_t d_tmem = 0;
          int acc = 0;
          for (int kb = 0; kb < num_kb; ++kb, ++it) {
            const bool begins = kb % MM_SEGMENT == 0;
            if (begins) {
              acc = scount & 1;
              const uint32_t use = (uint32_t)(scount >> 1);
              ++scount;
              if (!mbar_wait(&tempty[acc], (use & 1u) ^ 1u, abort_flag)) { ok = false; break; }
              tc_fence_after();
              d_tmem = tmem_base + (uint32_t)(acc * ACC_COLS);
            }
            const int s = it % S;
            const uint32_t ph = (uint32_t)(it / S) & 1u;
            if (!mbar_wait(&full[s], ph, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sw = smem_u32(smem + (size_t)s * SB);
            const uint64_t wd = W_MN ? gbwd::umma_desc_sw128_mn(sw) : umma_desc_sw128(sw);
            const uint64_t xd = umma_desc_sw128(sw + HALF_STAGE);
            constexpr uint64_t w_step = W_MN ? (2048 >> 4) : (32 >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_pair<0>(d_tmem, wd + w_step * k, xd + (uint64_t)(2 * k), idesc,
                           !begins || k != 0 ? 1u : 0u);
            const uint32_t e_local = smem_u32(&empty[s]);
            umma_commit_pair(mapa(e_local, 0));
            umma_commit_pair(mapa(e_local, 1));
            if (kb % MM_SEGMENT == MM_SEGMENT - 1 || kb == num_kb - 1) {
              const uint32_t t_local = smem_u32(&tfull[acc]);
              umma_commit_pair(mapa(t_local, 0));
              umma_commit_pair(mapa(t_local, 1));
            }
          }
        }
        umma_commit_pair(mapa(smem_u32(drain), 0));
        volatile int no_abort = 0;
        mbar_wait(drain, 0, &no_abort);
      }
      __syncwarp();
    }
  } else {
    if constexpr (ROWS == TILE_ROWS)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    // ------------------------------------------------------------------ epilogue (both CTAs)
    // Warp w reads TMEM lanes 32 (w % 4) .. +31 (32 features) and every other
    // chunk of 16 rows; a chunk is transposed in shared memory and stored as
    // 64 bytes per row.  Several segments are added up in registers first (the
    // chunks' loops unrolled); one goes out chunk by chunk as it is read, in a
    // loop (512 long, 64 groups of 384 rows: 114 us, through the registers 130).
    constexpr int CHUNKS = ROWS / 32;              // of a warp
    const int ew = warp - 4, q = warp & 3, par = ew >> 2;
    uint8_t* xb = xpose + (size_t)ew * MM_XPOSE;
    const uint32_t tempty_leader0 = mapa(smem_u32(&tempty[0]), 0);
    const uint32_t tempty_leader1 = mapa(smem_u32(&tempty[1]), 0);
    const int segments = (num_kb + MM_SEGMENT - 1) / MM_SEGMENT;
    int scount = 0;
    uint32_t tb = 0;          // the warp's lanes of the segment's accumulator
    auto take = [&]() {
      const int acc = scount & 1;
      const uint32_t use = (uint32_t)(scount >> 1);
      const bool there = mbar_wait_warp(&tfull[acc], use & 1u, abort_flag);
      tc_fence_after();
      tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * ACC_COLS);
      return there;
    };
    auto release = [&]() {
      const int acc = scount & 1;
      tc_fence_before();
      if (leader) mbar_arrive(&tempty[acc]);
      else mbar_arrive_cluster(acc ? tempty_leader1 : tempty_leader0);
      ++scount;
    };
    bool ok = true;
    for (int tile = tile0; tile < total && ok; tile += tstep) {
      const Tile t = locate(tile);
      // rows 8 m + lane / 4 of a chunk, 8 features
      const int f = t.ft * TF + (int)rank * 128 + q * 32 + (lane & 3) * 8;
      int left = f < a.feats ? t.rows - 16 * par - (lane >> 2) : 0;
      __nv_bfloat16* to = a.y + (size_t)(t.row + 16 * par + (lane >> 2)) * a.feats + f;
      auto store = [&](const float (&v)[16]) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          reinterpret_cast<__nv_bfloat16*>(xb)[j * 32 + lane] = __float2bfloat16_rn(v[j]);
        __syncwarp();
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint4 val = *reinterpret_cast<const uint4*>(xb + (lane + 32 * m) * 16);
          if (left > 8 * m) *reinterpret_cast<uint4*>(to + (size_t)(8 * m) * a.feats) = val;
        }
        __syncwarp();
        left -= 32;
        to += (size_t)32 * a.feats;
      };
      if (segments == 1) {
        if (!(ok = take())) break;
#pragma unroll 1
        for (int c = par; c * 16 < t.rows; c += 2) {
          float v[16];
          tmem_ld16(tb + (uint32_t)(16 * c), v);
          store(v);
        }
        release();
        continue;
      }
      float sum[CHUNKS][16];
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[i][j] = 0.f;
      for (int seg = 0; seg < segments; ++seg) {
        if (!(ok = take())) break;
#pragma unroll
        for (int i = 0; i < CHUNKS; i += 2) {      // two loads in flight
          const int c = par + 2 * i;
          if (c * 16 < t.rows) {
            uint32_t v[2][16];
            tmem_ld16_nowait(tb + (uint32_t)(16 * c), v[0]);
            tmem_ld16_nowait(tb + (uint32_t)(16 * c + 32), v[1]);
            tmem_wait_ld2(v[0], v[1]);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              sum[i][j] += __uint_as_float(v[0][j]);
              sum[i + 1][j] += __uint_as_float(v[1][j]);
            }
          }
        }
        release();
      }
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i)
        if (par * 16 + i * 32 < t.rows) store(sum[i]);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();      // the peer no longer touches this CTA's barriers or TMEM
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(TMEM_COLS)
                 : "memory");
  }
}

// dW tile of 256 output features (d_out, the UMMA M side) x 256 input features
// (d_in); both operands MN-major.  tmC: [G, d_out, d_in], boxes of 32 rows x
// 128 bytes.
template <bool OUT_BF16>
__global__ void __launch_bounds__(DW_THREADS, 1)
    k_grouped_dw(const __grid_constant__ CUtensorMap tmDy, const __grid_constant__ CUtensorMap tmX,
                 const __grid_constant__ CUtensorMap tmC, const Args a) {
  using namespace gemmt;
  constexpr int TO = 256, TI = 256;
  constexpr int S = STAGES;
  constexpr uint32_t BOX = gbwd::MN_BOX_BYTES;    // 64 rows x 64 features
  static_assert(4 * BOX == STAGE_BYTES, "two boxes of either operand per CTA");
  grid_dep_sync();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* store_buf = smem + S * STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(store_buf + DW_STORE);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* tail = drain + 1;
  uint64_t* peer_tail = tail + S;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(peer_tail + S);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  // by ordinary loads, here and below: the kernel that writes the offsets may still
  // run when this one is launched, and grid_dep_sync makes its writes visible to those
  auto rows_of = [&](int g) {
    const int r0 = a.offsets[g], r1 = a.offsets[g + 1];
    return group_ok(r0, r1, a.n_rows) ? r1 - r0 : 0;
  };
  if (threadIdx.x == 32) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
      mbar_init(&peer_tail[s], 1);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(&tfull[j], 1);
      mbar_init(&tempty[j], 2 * DW_EPI_WARPS * 32);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tmDy);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int n_it = (a.d_in + TI - 1) / TI, n_ot = (a.d_out + TO - 1) / TO;
  const int per_group = n_it * n_ot;
  const int total = a.n * per_group;
  const int tile0 = (int)(blockIdx.x >> 1), tstep = (int)(gridDim.x >> 1);

  struct Tile {
    int g, ot, it, row, rows, nkb, cols;
  };
  auto locate = [&](int tile) {
    Tile t;
    t.g = tile / per_group;
    const int l = tile - t.g * per_group;
    t.ot = l / n_it;
    t.it = l - t.ot * n_it;
    t.row = a.offsets[t.g];
    t.rows = rows_of(t.g);
    t.nkb = (t.rows + 63) / 64;
    t.cols = (min(TI, a.d_in - t.it * TI) + 31) & ~31;
    return t;
  };
  // nothing to add: every role leaves the tile out
  auto idle = [&](const Tile& t) { return a.accumulate && t.rows == 0; };
  // the group's last stage when its rows end inside a 16-row step
  auto is_tail = [&](const Tile& t, int kb) { return kb == t.nkb - 1 && (t.rows & 15) != 0; };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTRL_REGS));
    if (warp == 0) {
      // ------------------------------------------------------------------ TMA producer (both CTAs)
      if (elect_one()) {
        int it = 0;
        bool ok = true;
        for (int tile = tile0; tile < total && ok; tile += tstep) {
          const Tile t = locate(tile);
          if (idle(t)) continue;
          const int o = t.ot * TO + (int)rank * 128;
          const int i = t.it * TI + (int)rank * (t.cols / 2);
          for (int kb = 0; kb < t.nkb; ++kb, ++it) {
            const int s = it % S;
            const uint32_t ph = (uint32_t)(it / S) & 1u;
            if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag)) { ok = false; break; }
            uint8_t* sa = smem + (size_t)s * STAGE_BYTES;
            const int r = t.row + kb * 64;
            if (is_tail(t, kb)) {
              mbar_arrive_expect_tx(&tail[s], STAGE_BYTES);
              tma_load_2d(&tmDy, &tail[s], sa, o, r);
              tma_load_2d(&tmDy, &tail[s], sa + BOX, o + 64, r);
              tma_load_2d(&tmX, &tail[s], sa + 2 * BOX, i, r);
              tma_load_2d(&tmX, &tail[s], sa + 3 * BOX, i + 64, r);
            } else {
              const uint32_t fl = mapa(smem_u32(&full[s]), 0);
              if (leader) mbar_arrive_expect_tx(&full[s], 2 * STAGE_BYTES);
              tma_load_2d_pair(&tmDy, fl, sa, o, r);
              tma_load_2d_pair(&tmDy, fl, sa + BOX, o + 64, r);
              tma_load_2d_pair(&tmX, fl, sa + 2 * BOX, i, r);
              tma_load_2d_pair(&tmX, fl, sa + 3 * BOX, i + 64, r);
            }
          }
        }
        volatile int no_abort = 0;
        for (int j = (it - S > 0 ? it - S : 0); j < it; ++j)
          mbar_wait(&empty[j % S], (uint32_t)(j / S) & 1u, &no_abort);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------------------------------------------------ tail rows (both CTAs)
      if (blockIdx.x == 0)
        for (int g = lane; g < a.n; g += 32)
          if (!group_ok(a.offsets[g], a.offsets[g + 1], a.n_rows)) set_status(MOE_ERR_DEVICE_CHECK);
      int it = 0;
      uint32_t uses = 0;       // parity of the uses of each stage's tail barrier
      for (int tile = tile0; tile < total; tile += tstep) {
        const Tile t = locate(tile);
        if (idle(t)) continue;
        it += t.nkb;
        if (t.nkb == 0 || !is_tail(t, t.nkb - 1)) continue;
        const int s = (it - 1) % S;
        const uint32_t ph = (uses >> s) & 1u;
        uses ^= 1u << s;
        if (!mbar_wait_warp(&tail[s], ph, abort_flag)) break;
        const int first = t.rows - (t.nkb - 1) * 64, end = (first + 15) & ~15;
        uint8_t* sa = smem + (size_t)s * STAGE_BYTES;
        // a row is one 128-byte line of each of the four boxes; the swizzle
        // moves 16-byte pieces within a line only
        for (int j = lane; j < (end - first) * 32; j += 32) {
          const int row = first + (j >> 5), box = (j >> 3) & 3, piece = j & 7;
          *reinterpret_cast<uint4*>(sa + box * BOX + row * 128 + piece * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (!leader) {
          if (lane == 0) mbar_arrive_cluster(mapa(smem_u32(&peer_tail[s]), 0));
          continue;
        }
        if (!mbar_wait_warp(&peer_tail[s], ph, abort_flag)) break;
        asm volatile("fence.acq_rel.cluster;" ::: "memory");   // the peer's cleared lines
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------ MMA issuer (leader)
      if (leader && elect_one()) {
        int it = 0, scount = 0;
        bool ok = true;
        for (int tile = tile0; tile < total && ok; tile += tstep) {
          const Tile t = locate(tile);
          const uint32_t idesc = umma_idesc(1, TO, t.cols) | (1u << 15) | (1u << 16);
          uint32_t d_tmem = 0;
          int acc = 0;
          for (int kb = 0; kb < t.nkb; ++kb, ++it) {
            const bool begins = kb % DW_SEGMENT == 0;
            if (begins) {
              acc = scount & 1;
              const uint32_t use = (uint32_t)(scount >> 1);
              ++scount;
              if (!mbar_wait(&tempty[acc], (use & 1u) ^ 1u, abort_flag)) { ok = false; break; }
              tc_fence_after();
              d_tmem = tmem_base + (uint32_t)(acc * ACC_COLS);
            }
            const int s = it % S;
            const uint32_t ph = (uint32_t)(it / S) & 1u;
            if (!mbar_wait(&full[s], ph, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + (size_t)s * STAGE_BYTES);
            const uint64_t ad = gbwd::umma_desc_sw128_mn(sa);
            const uint64_t bd = gbwd::umma_desc_sw128_mn(sa + 2 * BOX);
            const int steps = min(4, (t.rows - kb * 64 + 15) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < steps)
                umma_pair<0>(d_tmem, ad + (uint64_t)(128 * k), bd + (uint64_t)(128 * k), idesc,
                             !begins || k != 0 ? 1u : 0u);
            const uint32_t e_local = smem_u32(&empty[s]);
            umma_commit_pair(mapa(e_local, 0));
            umma_commit_pair(mapa(e_local, 1));
            if (kb % DW_SEGMENT == DW_SEGMENT - 1 || kb == t.nkb - 1) {
              const uint32_t t_local = smem_u32(&tfull[acc]);
              umma_commit_pair(mapa(t_local, 0));
              umma_commit_pair(mapa(t_local, 1));
            }
          }
        }
        umma_commit_pair(mapa(smem_u32(drain), 0));
        volatile int no_abort = 0;
        mbar_wait(drain, 0, &no_abort);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    // ------------------------------------------------------------------ epilogue (both CTAs)
    // Blocks of 32 rows x 128 bytes through shared memory to TMA stores (or,
    // accumulating, TMA additions: each element of dW is added to once), which
    // clip the edges.
    // Warp w reads TMEM lanes 32 (w % 4) .. +31 and every other block.
    const int ew = warp - 4, q = warp & 3, par = ew >> 2;
    const uint32_t tempty_leader0 = mapa(smem_u32(&tempty[0]), 0);
    const uint32_t tempty_leader1 = mapa(smem_u32(&tempty[1]), 0);
    constexpr int W = OUT_BF16 ? 64 : 32;                   // columns of a block
    constexpr int BLOCKS = TI / W / 2;                      // of a warp
    int scount = 0;
    bool ok = true;
    for (int tile = tile0; tile < total && ok; tile += tstep) {
      const Tile t = locate(tile);
      if (idle(t)) continue;
      const int o = t.ot * TO + (int)rank * 128 + q * 32;   // the warp's first output feature
      const int chunks = o < a.d_out ? (t.cols + W - 1) / W : 0;
      float sum[BLOCKS][W];                                 // of row `lane`
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (int j = 0; j < W; ++j) sum[b][j] = 0.f;
      for (int k0 = 0; k0 < t.nkb; k0 += DW_SEGMENT, ++scount) {
        const int acc = scount & 1;
        const uint32_t use = (uint32_t)(scount >> 1);
        if (!mbar_wait_warp(&tfull[acc], use & 1u, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * ACC_COLS);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          const int c = par + 2 * b;
          if (c < chunks) {
#pragma unroll
            for (int h = 0; h < W; h += 32) {
              uint32_t v[2][16];
              tmem_ld16_nowait(tb + (uint32_t)(W * c + h), v[0]);
              tmem_ld16_nowait(tb + (uint32_t)(W * c + h + 16), v[1]);
              tmem_wait_ld2(v[0], v[1]);
#pragma unroll
              for (int j = 0; j < 32; ++j) sum[b][h + j] += __uint_as_float(v[j >> 4][j & 15]);
            }
          }
        }
        tc_fence_before();
        if (leader) mbar_arrive(&tempty[acc]);
        else mbar_arrive_cluster(acc ? tempty_leader1 : tempty_leader0);
      }
      if (!ok) break;
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) {
        const int c = par + 2 * b;
        if (c < chunks) {
          uint8_t* buf = store_buf + (size_t)ew * DW_STAGING;
          // the last store has read the block
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
          // row `lane`, 16-byte piece j at j ^ (row % 8) (128-byte swizzle)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t w4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w4[i] = OUT_BF16 ? gemm::pack_bf16x2(sum[b][(8 * j + 2 * i) % W],
                                                   sum[b][(8 * j + 2 * i + 1) % W])
                               : __float_as_uint(sum[b][(4 * j + i) % W]);
            *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(w4[0], w4[1], w4[2], w4[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (a.accumulate) tma_add_3d(&tmC, buf, t.it * TI + W * c, o, t.g);
            else gbwd::tma_store_3d(&tmC, buf, t.it * TI + W * c, o, t.g);
            bulk_commit_group();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(TMEM_COLS)
                 : "memory");
  }
}

}  // namespace grouped
}  // namespace moe
