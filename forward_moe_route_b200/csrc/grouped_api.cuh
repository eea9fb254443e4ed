// Entry points of the grouped products.  Included by api.cu, whose helpers it
// uses.
#pragma once

#include "grouped.cuh"
#include "grouped_few.cuh"

namespace {

// Tensor map of rank 2 or 3 over a contiguous array, 128-byte swizzle; dims
// innermost first.
moe_status grouped_map(CUtensorMap* m, const void* base, bool f32, int rank, const uint64_t* dims,
                       const uint32_t* box) {
  const uint64_t esz = f32 ? 4 : 2;
  cuuint64_t n[3], strides[2];
  cuuint32_t b[3], one[3] = {1, 1, 1};
  uint64_t bytes = esz;
  for (int i = 0; i < rank; ++i) {
    n[i] = dims[i] > 0 ? dims[i] : 1;
    b[i] = box[i];
    bytes *= n[i];
    if (i + 1 < rank) strides[i] = bytes;
  }
  const CUresult r = g_encode(
      m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
      (cuuint32_t)rank, const_cast<void*>(base), n, strides, b, one,
      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    snprintf(t_errmsg, sizeof(t_errmsg), "cuTensorMapEncodeTiled (grouped): CUresult %d (inner "
             "%llu, rows %llu)", (int)r, (unsigned long long)n[0], (unsigned long long)n[1]);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

moe_status grouped_dims(int32_t n_groups, int32_t n_rows, int32_t d_in, int32_t d_out) {
  if (n_groups < 1 || n_groups > grouped::MAX_GROUPS || n_rows < 0 || d_in < 8 || d_out < 8 ||
      d_in > 65536 || d_out > 65536 || d_in % 8 || d_out % 8)
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Products of at most FEW_MAX rows, two a group on average, stream their weights by
// k_few_mm while these are 64 MiB at most, counted with a group for each row.  Measured,
// k_few_mm and k_grouped_mm, 2048 x 2816, back to back in a graph and (in brackets) one
// call with the weights out of L2: one row in each of 4 groups 9.5 and 11.9 us (21.6
// and 20.5), of 5, 55 MiB, 10.5 and 11.6 (22.7 and 22.5), of 6, 66 MiB, 11.1 and 11.9
// (26.6 and 24.6), of 8 15.2 and 17.2 (32.8 and 32.8), of 12 34 and 27 (45 and 39).  So
// just above 64 MiB streaming can still win by 7% from L2 and loses as much from memory;
// well above it loses.  Each group's rows go by two, so rows that share a group read
// its weights again: 8 rows of one group 4096 x 4096 35 and 16 us, which the size and
// the average keep out; all 16 rows in one of 64 groups 512 x 512, 12 and 6 us, they
// cannot, as the offsets are on the device.
constexpr int64_t kFewBytes = 64 << 20;
bool grouped_few(const grouped::Args& a) {
  return a.n_rows <= grouped::FEW_MAX && a.n_rows <= 2 * a.n &&
         2ll * a.n_rows * a.feats * a.contract <= kFewBytes;
}
moe_status launch_grouped_few(const grouped::Args& a, const void* x, const void* w, int sms,
                              cudaStream_t st) {
  // as many items as there can be, each row with a group of its own
  const int64_t items = (int64_t)(a.n < a.n_rows ? a.n : a.n_rows) *
                        ((a.feats + grouped::FEW_FEATURES - 1) / grouped::FEW_FEATURES);
  const int64_t blocks = (items + grouped::FEW_THREADS / 32 - 1) / (grouped::FEW_THREADS / 32);
  return launch_chain("k_few_mm", grouped::k_few_mm,
                      dim3((unsigned)(blocks < 16 * sms ? blocks : 16 * sms)),
                      dim3(grouped::FEW_THREADS), 0, st, a,
                      static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(w));
}

// y = rows x W^T (dx: rows x W); the weights [G, d_out, d_in]
moe_status launch_grouped_mm(bool dx, int32_t G, int32_t R, int32_t d_in, int32_t d_out,
                             const void* rows, const void* w, const int32_t* offsets, void* y,
                             int sms, cudaStream_t st) {
  const uint64_t contract = dx ? d_out : d_in, feats = dx ? d_in : d_out;
  grouped::Args a;
  memset(&a, 0, sizeof(a));
  a.offsets = offsets;
  a.n = G;
  a.n_rows = R;
  a.feats = (int)feats;
  a.contract = (int)contract;
  a.y = static_cast<__nv_bfloat16*>(y);
  if (!dx && grouped_few(a)) return launch_grouped_few(a, rows, w, sms, st);
  const uint64_t wdims[3] = {(uint64_t)d_in, (uint64_t)d_out, (uint64_t)G};
  const uint32_t wbox[3] = {64, dx ? 64u : 128u, 1};
  const uint64_t xdims[2] = {contract, (uint64_t)R};
  const uint32_t xbox[3][2] = {{64, 128}, {64, 64}, {64, 32}};
  CUtensorMap tw, tx[3];
  moe_status rc = grouped_map(&tw, w, false, 3, wdims, wbox);
  for (int i = 0; i < 3 && rc == MOE_OK; ++i)
    rc = grouped_map(&tx[i], rows, false, 2, xdims, xbox[i]);
  if (rc != MOE_OK) return rc;
  // Groups of 32 rows on average or fewer take the lower row tiles (64 groups 2048 x
  // 2816 of 8 rows: 122 and 127 us, of 32 rows 125 and 129 us, of 64 rows no
  // difference).  The row gradients, whose weights come in whole lines either way,
  // were slower with them (116 and 110 us).
  const bool few = !dx && R <= (int64_t)G * 32;
  // at most this many row tiles: every group may add a partly filled one
  const int64_t row_tiles = R / (few ? grouped::FEW_ROWS : grouped::TILE_ROWS) + (G < R ? G : R);
  const int64_t tiles = row_tiles * (int64_t)((feats + 255) / 256);
  auto* k = dx    ? grouped::k_grouped_mm<true, grouped::TILE_ROWS>
            : few ? grouped::k_grouped_mm<false, grouped::FEW_ROWS>
                  : grouped::k_grouped_mm<false, grouped::TILE_ROWS>;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  rc = pair_config(dx ? 5 : few ? 8 : 4, k, grouped::MM_THREADS,
                   few ? grouped::mm_smem(grouped::FEW_ROWS) : grouped::mm_smem(grouped::TILE_ROWS),
                   tiles, st, &cfg, attr);
  if (rc != MOE_OK) return rc;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, tw, tx[0], tx[1], tx[2], a);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "k_grouped_mm");
}

}  // namespace

extern "C" {

moe_status moe_grouped_mm(int32_t n_groups, int32_t n_rows, int32_t d_in, int32_t d_out,
                          const void* x, const void* w, const int32_t* offsets, void* y,
                          cudaStream_t stream) {
  moe_status rc = grouped_dims(n_groups, n_rows, d_in, d_out);
  if (rc != MOE_OK) return rc;
  if (n_rows == 0) return MOE_OK;
  if (!given(x) || !given(w) || !given(offsets) || !given(y) || y == x || y == w)
    return MOE_ERR_INVALID_ARG;
  int sms;
  if ((rc = device_setup(&sms)) != MOE_OK) return rc;
  return launch_grouped_mm(false, n_groups, n_rows, d_in, d_out, x, w, offsets, y, sms, stream);
}

moe_status moe_grouped_mm_dx(int32_t n_groups, int32_t n_rows, int32_t d_in, int32_t d_out,
                             const void* dy, const void* w, const int32_t* offsets, void* dx,
                             cudaStream_t stream) {
  moe_status rc = grouped_dims(n_groups, n_rows, d_in, d_out);
  if (rc != MOE_OK) return rc;
  if (n_rows == 0) return MOE_OK;
  if (!given(dy) || !given(w) || !given(offsets) || !given(dx) || dx == dy || dx == w)
    return MOE_ERR_INVALID_ARG;
  int sms;
  if ((rc = device_setup(&sms)) != MOE_OK) return rc;
  return launch_grouped_mm(true, n_groups, n_rows, d_in, d_out, dy, w, offsets, dx, sms, stream);
}

moe_status moe_grouped_mm_dw(int32_t n_groups, int32_t n_rows, int32_t d_in, int32_t d_out,
                             const void* dy, const void* x, const int32_t* offsets, void* dw,
                             int32_t bf16_grads, int32_t accumulate, cudaStream_t stream) {
  moe_status rc = grouped_dims(n_groups, n_rows, d_in, d_out);
  if (rc != MOE_OK) return rc;
  if ((bf16_grads != 0 && bf16_grads != 1) || (accumulate != 0 && accumulate != 1) ||
      (bf16_grads && accumulate))
    return MOE_ERR_INVALID_ARG;
  if (!given(offsets) || !given(dw) || (n_rows > 0 && (!given(dy) || !given(x))) || dw == dy ||
      dw == x)
    return MOE_ERR_INVALID_ARG;
  if (n_rows == 0 && accumulate) return MOE_OK;
  int sms;
  if ((rc = device_setup(&sms)) != MOE_OK) return rc;
  // without rows no group loads any: the maps only need some valid address
  if (n_rows == 0) dy = x = dw;
  const uint64_t ydims[2] = {(uint64_t)d_out, (uint64_t)n_rows};
  const uint64_t xdims[2] = {(uint64_t)d_in, (uint64_t)n_rows};
  const uint64_t cdims[3] = {(uint64_t)d_in, (uint64_t)d_out, (uint64_t)n_groups};
  const uint32_t box[2] = {64, 64}, cbox[3] = {bf16_grads ? 64u : 32u, 32, 1};
  CUtensorMap ty, tx, tc;
  rc = grouped_map(&ty, dy, false, 2, ydims, box);
  if (rc == MOE_OK) rc = grouped_map(&tx, x, false, 2, xdims, box);
  if (rc == MOE_OK) rc = grouped_map(&tc, dw, !bf16_grads, 3, cdims, cbox);
  if (rc != MOE_OK) return rc;
  grouped::Args a;
  memset(&a, 0, sizeof(a));
  a.offsets = offsets;
  a.n = n_groups;
  a.n_rows = n_rows;
  a.d_in = d_in;
  a.d_out = d_out;
  a.accumulate = accumulate;
  const int64_t tiles = (int64_t)n_groups * ((d_in + 255) / 256) * ((d_out + 255) / 256);
  auto* k = bf16_grads ? grouped::k_grouped_dw<true> : grouped::k_grouped_dw<false>;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  rc = pair_config(bf16_grads ? 7 : 6, k, grouped::DW_THREADS, grouped::DW_SMEM, tiles, stream,
                   &cfg, attr);
  if (rc != MOE_OK) return rc;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, ty, tx, tc, a);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "k_grouped_dw");
}

}  // extern "C"
