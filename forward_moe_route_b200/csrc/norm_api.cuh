// Entry points of the block norms: argument checks, the shape rule and the
// launches.  Included by api.cu, whose helpers it uses.
#pragma once

#include "norm.cuh"

namespace {

struct NormDims {
  int64_t T, d;
  bool bf16;
  int vec;          // elements of a 16-byte vector
  int64_t n_gate;   // gate rows (0 without gate)
};

moe_status norm_dims(const moe_norm_desc* s, NormDims* D) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->T < 0 || s->d < 1 || s->d > 65536 || s->n_slots < 1 ||
      s->n_slots > route::MAXK + kMaxShared || s->gate_group < 0 ||
      (s->act_dtype != MOE_DT_F32 && s->act_dtype != MOE_DT_BF16))
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(s->eps) || !(s->eps > 0.f) || !std::isfinite(s->res_scale))
    return MOE_ERR_INVALID_ARG;
  D->T = s->T;
  D->d = s->d;
  D->bf16 = s->act_dtype == MOE_DT_BF16;
  D->vec = D->bf16 ? 8 : 4;
  D->n_gate = s->gate_group ? (D->T + s->gate_group - 1) / s->gate_group : 0;
  return MOE_OK;
}

// How a row is held.  Rows of whole 16-byte vectors are read in vectors
// (V = 8 bf16 or 4 fp32), others in single elements; rows that do not fit take
// the looping kernels (vpt = 0).
// Forward: a row of up to 128 vectors or 256 single elements belongs to one warp,
// a longer one to a block, with one vector a thread when there are fewer rows than
// SMs and latency counts, else with two or four.
// Backward: up to 4 vectors (16 single elements) a thread and as many rows a
// block as it holds.
constexpr int64_t NORM_SMS = 148;
struct NormShape {
  int v, vpt, tpr, threads;
  int rows_here() const { return threads / tpr; }
};

NormShape norm_shape(const NormDims& D, bool backward) {
  NormShape s;
  const bool whole = D.d % D.vec == 0;
  s.v = whole ? D.vec : 1;
  const int64_t n = D.d / s.v;
  if (backward) {
    s.vpt = !whole ? 16 : n <= 32 ? 1 : n <= 64 ? 2 : 4;
    s.tpr = (int)((n + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    if (s.tpr > norm::BWD_THREADS) {
      s.vpt = 0;
      s.tpr = s.threads = norm::MAX_THREADS;
      return s;
    }
    s.threads = norm::BWD_THREADS / s.tpr * s.tpr;
    return s;
  }
  if (n <= (whole ? 128 : 256)) {
    s.vpt = !whole ? 8 : n <= 32 ? 1 : n <= 64 ? 2 : 4;
    s.tpr = 32;
    s.threads = 256;
    return s;
  }
  const int widest = whole ? 4 : 8;
  s.vpt = !whole ? 8 : D.T < NORM_SMS && n <= norm::MAX_THREADS ? 1 : 2;
  if (n > (int64_t)s.vpt * norm::MAX_THREADS) s.vpt = widest;
  if (n > (int64_t)s.vpt * norm::MAX_THREADS) {
    s.vpt = 0;
    s.tpr = s.threads = norm::MAX_THREADS;
    return s;
  }
  s.tpr = (int)((n + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  s.threads = s.tpr;
  return s;
}

// How the backward cuts the tokens: units, none across two gate rows, one for
// each block that runs at a time (one on each of 148 SMs, four of the looping
// kernel).  A gate row of more tokens
// is split; gate rows of fewer tokens than keep a block's row groups busy are
// single row groups' units (`alone`).
struct NormCut {
  int64_t group, rows, split, units, blocks;
  bool alone;
};
NormCut norm_cut(const NormDims& D, int64_t gate_group, const NormShape& s) {
  NormCut c;
  c.group = gate_group && gate_group < D.T ? gate_group : D.T;
  if (c.group == 0) return NormCut{0, 0, 1, 0, 0, false};
  const int64_t most = NORM_SMS * (s.vpt ? 1 : 4);
  const int64_t here = s.rows_here();
  c.alone = gate_group && here > 1 && c.group < 4 * here;
  if (c.alone) {
    c.rows = c.group;
    c.split = 1;
    c.units = (D.T + c.group - 1) / c.group;
    const int64_t blocks = (c.units + here - 1) / here;
    c.blocks = blocks < most ? blocks : most;
    return c;
  }
  // units in one to four full waves of blocks, whichever leaves the last block
  // the fewest rows (a unit costs about as much as four more)
  const int64_t gates = (D.T + c.group - 1) / c.group;
  int64_t best = 0;
  for (int64_t wave = 1; wave <= 4; ++wave) {
    int64_t split = wave * most / gates;
    if (split * here > c.group) split = c.group / here;
    if (split < 1) split = 1;
    const int64_t rows = (c.group + split - 1) / split;
    split = (c.group + rows - 1) / rows;
    const int64_t cost =
        (gates * split + most - 1) / most * ((rows + here - 1) / here + 4);
    if (best && cost >= best) continue;
    best = cost;
    c.rows = rows;
    c.split = split;
  }
  c.units = (D.T + c.group - 1) / c.group * c.split;
  c.blocks = c.units < most ? c.units : most;
  return c;
}

constexpr int64_t kNormSmem = 208 * 1024;   // of a block that has an SM to itself
// Rows in flight for each row group, in the shared memory beside the row groups'
// sums.
constexpr int64_t kNormRing = 8;
// sums of the row groups, and the weight's when blocks share whole gate rows
int64_t norm_joined(const NormDims& D, const NormShape& s, const NormCut& c, bool gate) {
  const int64_t keep = gate && c.split == 1 && !c.alone ? 1 : 0;
  return (s.rows_here() + keep) * D.d * 4;
}
int64_t norm_room(const NormDims& D, const NormShape& s) {
  if (s.v > 1) return D.d * (D.bf16 ? 2 : 4);
  return D.bf16 ? norm::SharedRow<__nv_bfloat16, 1>::room((int)D.d)
                : norm::SharedRow<float, 1>::room((int)D.d);
}
int norm_stages(const NormDims& D, const NormShape& s, int parts, int64_t joined) {
  const int64_t n = (kNormSmem - joined) / (s.rows_here() * parts * norm_room(D, s));
  return (int)(n < kNormRing ? n : kNormRing);
}

struct NormLayout {
  size_t part_w, part_g, total;
};
NormLayout norm_layout(const NormDims& D, const NormCut& c, bool wide) {
  NormLayout L;
  const size_t row = (size_t)D.d * 4;
  L.part_w = 0;
  L.part_g = align_up((size_t)c.blocks * row, kAlign);
  const size_t g = !D.n_gate ? 0 : c.split > 1 ? (size_t)c.units : wide ? (size_t)c.blocks : 0;
  L.total = align_up(L.part_g + g * row, kAlign);
  if (!L.total) L.total = kAlign;
  return L;
}

// Streams many tokens' rows through shared memory: up to 4 vectors a thread (8 single
// elements), as many blocks on an SM as 1024 threads hold, the shared memory divided
// among them.  Short rows stay with k_norm_fwd's warps, and so does moe_norm with
// rows of whole vectors (16384 x 7168 bf16 137 us, floor 72), for which the ring is
// not built.
// Measured, stream and warps or blocks: 4000 tokens x 7 rows of 7168 bf16 110 and
// 148 us, 16000 x 7 x 1024 fp32 115 and 132 us, 16000 x 7 x 512 bf16 (rows of 1 KB)
// 53 and 42 us, 700 x 7 x 2048 fp32 14.6 and 11.2 us.
constexpr int64_t kStreamRow = 2048;      // bytes of a row
constexpr int64_t kStreamTokens = 1184;   // eight for each of 148 SMs
bool norm_streams(const NormDims& D, bool combine) {
  const bool whole = D.d % D.vec == 0;
  return D.T >= kStreamTokens && (whole ? combine && D.d * (D.bf16 ? 2 : 4) >= kStreamRow &&
                                              D.d / D.vec <= 2048
                                        : D.d > 256 && D.d <= 8 * 992);
}
template <typename E, bool COMBINE>
moe_status launch_norm_stream(norm::FwdArgs a, int sms, cudaStream_t st) {
  constexpr int VEC = norm::Elem<E>::VEC;
  const bool whole = a.d % VEC == 0;
  const int n = whole ? a.d / VEC : a.d;
  const int vpt = !whole ? 8 : n <= 512 ? 1 : n <= 1024 ? 2 : 4;
  a.tpr = ((n + vpt - 1) / vpt + 31) / 32 * 32;
  const int threads = a.tpr + 32;
  const int per_sm = 1024 / threads < 1 ? 1 : 1024 / threads > 8 ? 8 : 1024 / threads;
  const int64_t row = whole ? (int64_t)a.d * sizeof(E) : norm::SharedRow<E, 1>::room(a.d);
  int stages = (int)(kNormSmem / per_sm / row);
  if (stages > norm::STREAM_STAGES) stages = norm::STREAM_STAGES;
  auto* k = norm::k_norm_stream<E, 1, 8, COMBINE>;
  if constexpr (COMBINE) {
    if (whole)
      k = vpt == 1   ? norm::k_norm_stream<E, VEC, 1, true>
          : vpt == 2 ? norm::k_norm_stream<E, VEC, 2, true>
                     : norm::k_norm_stream<E, VEC, 4, true>;
  }
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kNormSmem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute (k_norm_stream)");
  const int64_t blocks = a.T < (int64_t)sms * per_sm ? a.T : (int64_t)sms * per_sm;
  return launch_chain("k_norm_stream", k, dim3((unsigned)blocks), dim3(threads),
                      (size_t)stages * row, st, a, stages);
}

template <typename E, bool COMBINE>
moe_status launch_norm_fwd(const NormShape& s, norm::FwdArgs a, int sms, cudaStream_t st) {
  constexpr int VEC = norm::Elem<E>::VEC;
  auto* k = s.v == 1 ? (s.vpt ? norm::k_norm_fwd<E, 1, 8, COMBINE>
                              : norm::k_norm_fwd_wide<E, 1, COMBINE>)
            : s.vpt == 1 ? norm::k_norm_fwd<E, VEC, 1, COMBINE>
            : s.vpt == 2 ? norm::k_norm_fwd<E, VEC, 2, COMBINE>
            : s.vpt == 4 ? norm::k_norm_fwd<E, VEC, 4, COMBINE>
                         : norm::k_norm_fwd_wide<E, VEC, COMBINE>;
  a.tpr = s.tpr;
  const int64_t blocks = (a.T + s.rows_here() - 1) / s.rows_here();
  // Resident blocks stride over many rows (16384 rows of 7168: 554 us, one block
  // a row 703 us); with few waves one block a row spares the half-empty last one
  // (4097 rows of 1001: 7.5 us, strided 9.0 us).
  const int64_t resident = (int64_t)sms * (2048 / s.threads);
  const int64_t most = blocks < 4 * resident ? blocks : resident;
  return launch_chain(COMBINE ? "k_norm_fwd (combine)" : "k_norm_fwd", k,
                      dim3((unsigned)(blocks < most ? blocks : most)), dim3(s.threads), 0, st, a);
}

template <typename E, int GATE_KIND>
moe_status launch_norm_bwd(const NormDims& D, const NormShape& s, const NormCut& c,
                           norm::BwdArgs a, float* dw, cudaStream_t st) {
  constexpr int VEC = norm::Elem<E>::VEC;
  constexpr bool GATE = GATE_KIND == norm::GATE_ROWS;
  const bool wide = s.vpt == 0;
  if (a.T > 0) {
    auto* k = s.v == 1 ? (wide ? norm::k_norm_bwd_wide<E, 1, GATE>
                               : norm::k_norm_bwd<E, 1, 16, GATE_KIND>)
              : wide       ? norm::k_norm_bwd_wide<E, VEC, GATE>
              : s.vpt == 1 ? norm::k_norm_bwd<E, VEC, 1, GATE_KIND>
              : s.vpt == 2 ? norm::k_norm_bwd<E, VEC, 2, GATE_KIND>
                           : norm::k_norm_bwd<E, VEC, 4, GATE_KIND>;
    a.tpr = s.tpr;
    size_t smem = 0;
    if (!wide) {
      const int parts = a.add || GATE_KIND == norm::GATE_EACH ? 3 : 2;
      const size_t joined = (size_t)norm_joined(D, s, c, GATE);
      a.stages = norm_stages(D, s, parts, GATE ? (int64_t)joined : 0);
      smem = (size_t)s.rows_here() * a.stages * parts * norm_room(D, s);
      smem = GATE ? smem + joined : smem > joined ? smem : joined;
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)kNormSmem);
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute (k_norm_bwd)");
    }
    const moe_status rc = launch_chain("k_norm_bwd", k, dim3((unsigned)c.blocks),
                                       dim3(s.threads), smem, st, a);
    if (rc != MOE_OK) return rc;
  }
  const int64_t gates = GATE && c.split > 1 ? c.units / c.split : 0;
  // split gate rows leave one set of sums for both gradients (the looping kernel
  // keeps the weight's by themselves)
  const bool shared = gates && !wide;
  return launch_chain("k_norm_join", norm::k_norm_join<E>,
                      dim3((unsigned)((a.d + 31) / 32), (unsigned)(1 + gates)),
                      dim3(32, norm::JOIN_SLICES), 0,
                      st, static_cast<const float*>(shared ? a.part_g : a.part_w),
                      (int)(shared ? c.units : c.blocks), dw,
                      static_cast<const float*>(a.part_g), (int)c.split,
                      static_cast<const E*>(a.w),
                      static_cast<const E*>(shared ? a.gate : nullptr),
                      static_cast<E*>(a.dgate), a.d);
}

// Shape, cut and workspace of a backward pass.  A gate row for every token is cut
// like none (the looping kernel has only whole gate rows as units).
struct NormPlan {
  NormShape s;
  NormCut c;
  NormLayout L;
  int gate;
};
NormPlan norm_plan(const NormDims& D, int64_t gate_group) {
  NormPlan p;
  p.s = norm_shape(D, true);
  p.gate = !gate_group ? norm::GATE_NONE
           : gate_group == 1 && p.s.vpt ? norm::GATE_EACH : norm::GATE_ROWS;
  NormDims rows = D;
  if (p.gate != norm::GATE_ROWS) rows.n_gate = 0;
  p.c = norm_cut(D, p.gate == norm::GATE_ROWS ? gate_group : 0, p.s);
  p.L = norm_layout(rows, p.c, p.s.vpt == 0);
  return p;
}

moe_status norm_backward(const moe_norm_desc& desc, const NormDims& D, bool with_gate,
                         norm::BwdArgs a, float* dw, void* ws, size_t ws_bytes,
                         cudaStream_t st) {
  const NormPlan p = norm_plan(D, with_gate ? desc.gate_group : 0);
  const NormShape& s = p.s;
  const NormCut& c = p.c;
  const NormLayout& L = p.L;
  if (!ws || ws_bytes < L.total || !aligned16(ws)) return MOE_ERR_WORKSPACE;
  int sms;
  const moe_status rc = device_setup(&sms);
  if (rc != MOE_OK) return rc;
  a.part_w = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + L.part_w);
  a.part_g = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + L.part_g);
  a.T = (int)D.T;
  a.d = (int)D.d;
  a.group = (int)c.group;
  a.rows = (int)c.rows;
  a.split = (int)c.split;
  a.units = (int)c.units;
  a.alone = c.alone ? 1 : 0;
  a.eps = desc.eps;
  a.res = desc.res_scale;
  using norm::GATE_EACH, norm::GATE_NONE, norm::GATE_ROWS;
  if (D.bf16)
    return p.gate == GATE_NONE ? launch_norm_bwd<__nv_bfloat16, GATE_NONE>(D, s, c, a, dw, st)
           : p.gate == GATE_EACH
               ? launch_norm_bwd<__nv_bfloat16, GATE_EACH>(D, s, c, a, dw, st)
               : launch_norm_bwd<__nv_bfloat16, GATE_ROWS>(D, s, c, a, dw, st);
  return p.gate == GATE_NONE   ? launch_norm_bwd<float, GATE_NONE>(D, s, c, a, dw, st)
         : p.gate == GATE_EACH ? launch_norm_bwd<float, GATE_EACH>(D, s, c, a, dw, st)
                               : launch_norm_bwd<float, GATE_ROWS>(D, s, c, a, dw, st);
}

// a required pointer: present and 16-byte aligned
inline bool given(const void* p) { return p && aligned16(p); }
inline bool given_or_null(const void* p) { return aligned16(p); }

}  // namespace

extern "C" {

moe_status moe_norm(const moe_norm_desc* desc, const void* x, const void* w, void* out,
                    cudaStream_t stream) {
  NormDims D;
  moe_status rc = norm_dims(desc, &D);
  if (rc != MOE_OK) return rc;
  if (D.T == 0) return MOE_OK;
  if (!given(x) || !given(w) || !given(out) || out == x || out == w) return MOE_ERR_INVALID_ARG;
  int sms;
  if ((rc = device_setup(&sms)) != MOE_OK) return rc;
  norm::FwdArgs a;
  memset(&a, 0, sizeof(a));
  a.u = x; a.w = w; a.h = out;
  a.T = (int)D.T; a.d = (int)D.d; a.S = 1; a.eps = desc->eps;
  if (norm_streams(D, false))
    return D.bf16 ? launch_norm_stream<__nv_bfloat16, false>(a, sms, stream)
                  : launch_norm_stream<float, false>(a, sms, stream);
  const NormShape s = norm_shape(D, false);
  return D.bf16 ? launch_norm_fwd<__nv_bfloat16, false>(s, a, sms, stream)
                : launch_norm_fwd<float, false>(s, a, sms, stream);
}

moe_status moe_combine_norm(const moe_norm_desc* desc, const void* x_residual,
                            const void* y_slots, const void* w, const void* gate,
                            const void* w_next, void* h, void* y, void* x_next,
                            cudaStream_t stream) {
  NormDims D;
  moe_status rc = norm_dims(desc, &D);
  if (rc != MOE_OK) return rc;
  // without tokens x_next and the gate have no rows, so their addresses may be null
  if (D.T == 0)
    return (x_next && !w_next) || (gate && !desc->gate_group) ? MOE_ERR_INVALID_ARG : MOE_OK;
  if (!w_next != !x_next || !gate != !desc->gate_group) return MOE_ERR_INVALID_ARG;
  if (!given(x_residual) || !given(y_slots) || !given(w) || !given(h) || !given_or_null(gate) ||
      !given_or_null(w_next) || !given_or_null(y) || !given_or_null(x_next))
    return MOE_ERR_INVALID_ARG;
  // outputs apart from the inputs and from one another
  const void* out[3] = {h, y, x_next};
  const void* in[5] = {x_residual, y_slots, w, gate, w_next};
  for (int i = 0; i < 3; ++i) {
    if (!out[i]) continue;
    for (const void* p : in)
      if (p == out[i]) return MOE_ERR_INVALID_ARG;
    for (int j = i + 1; j < 3; ++j)
      if (out[j] == out[i]) return MOE_ERR_INVALID_ARG;
  }
  int sms;
  if ((rc = device_setup(&sms)) != MOE_OK) return rc;
  norm::FwdArgs a;
  memset(&a, 0, sizeof(a));
  a.u = x_residual; a.slots = y_slots; a.w = w; a.gate = gate; a.w_next = w_next;
  a.h = h; a.y = y; a.x_next = x_next;
  a.T = (int)D.T; a.d = (int)D.d; a.S = desc->n_slots; a.gate_group = desc->gate_group;
  a.eps = desc->eps; a.res = desc->res_scale;
  if (norm_streams(D, true))
    return D.bf16 ? launch_norm_stream<__nv_bfloat16, true>(a, sms, stream)
                  : launch_norm_stream<float, true>(a, sms, stream);
  const NormShape s = norm_shape(D, false);
  return D.bf16 ? launch_norm_fwd<__nv_bfloat16, true>(s, a, sms, stream)
                : launch_norm_fwd<float, true>(s, a, sms, stream);
}

size_t moe_norm_backward_workspace_size(const moe_norm_desc* desc) {
  NormDims D;
  if (norm_dims(desc, &D) != MOE_OK) return 0;
  const size_t without = norm_plan(D, 0).L.total;
  const size_t with = norm_plan(D, desc->gate_group).L.total;
  return with > without ? with : without;
}

moe_status moe_norm_backward(const moe_norm_desc* desc, const void* x, const void* w,
                             const void* dout, const void* dh, void* dx, float* dw, void* ws,
                             size_t ws_bytes, cudaStream_t stream) {
  NormDims D;
  moe_status rc = norm_dims(desc, &D);
  if (rc != MOE_OK) return rc;
  if (!given(dw)) return MOE_ERR_INVALID_ARG;
  if (D.T > 0 && (!given(x) || !given(w) || !given(dout) || !given_or_null(dh) || !given(dx) ||
                  dx == x || dx == w || dx == dout || dx == dh))
    return MOE_ERR_INVALID_ARG;
  norm::BwdArgs a;
  memset(&a, 0, sizeof(a));
  a.v = x; a.w = w; a.up = dout; a.add = dh; a.dv = dx;
  return norm_backward(*desc, D, false, a, dw, ws, ws_bytes, stream);
}

moe_status moe_combine_norm_backward(const moe_norm_desc* desc, const void* y, const void* w,
                                     const void* gate, const void* dh, void* dy, float* dw,
                                     void* dgate, void* ws, size_t ws_bytes,
                                     cudaStream_t stream) {
  NormDims D;
  moe_status rc = norm_dims(desc, &D);
  if (rc != MOE_OK) return rc;
  // without tokens the gate and its gradient have no rows, so their addresses may be null
  if (!given(dw) || ((gate || dgate) && !desc->gate_group)) return MOE_ERR_INVALID_ARG;
  if (D.T > 0 && (!gate != !desc->gate_group || !gate != !dgate)) return MOE_ERR_INVALID_ARG;
  if (D.T > 0 && (!given(y) || !given(w) || !given_or_null(gate) || !given(dh) || !given(dy) ||
                  !given_or_null(dgate) || dy == y || dy == w || dy == gate || dy == dh ||
                  dy == dgate || (gate && dgate == gate)))
    return MOE_ERR_INVALID_ARG;
  norm::BwdArgs a;
  memset(&a, 0, sizeof(a));
  a.v = y; a.w = w; a.gate = gate; a.up = dh; a.dv = dy; a.dgate = dgate;
  return norm_backward(*desc, D, gate != nullptr, a, dw, ws, ws_bytes, stream);
}

}  // extern "C"
