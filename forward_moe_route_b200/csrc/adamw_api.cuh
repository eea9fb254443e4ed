// Entry points of the AdamW step: the table of a tensor list, and the launch.
// Included by api.cu, whose helpers it uses.
#pragma once

#include <float.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "adamw.cuh"

namespace {

constexpr int kMaxTensors = 1 << 24;    // the random counter has 24 bits for the tensor
constexpr int64_t kMaxChunks = 0x7fffffff;

// Spans of a chunk: with 8-bit states a block asks for spans while it works on the
// ones before, so chunks are as long as four blocks of them on each of 148 SMs
// still come in four waves, 16 at most.  fp32 states are bound by memory with one.
int adamw_spans(int64_t elements, bool small) {
  const int64_t n = small ? elements / ((int64_t)adamw::SPAN * 148 * 16) : 1;
  return n < 1 ? 1 : n > 16 ? 16 : (int)n;
}
int64_t adamw_chunks(int64_t n, int spans) {
  const int64_t size = (int64_t)spans * adamw::SPAN;
  return n / size + (n % size != 0);
}

// chunks of one span of the list, -1 when a length or the count is not accepted
int64_t adamw_list_chunks(const moe_adamw_tensor* tensors, int32_t n) {
  if (n < 0 || n > kMaxTensors || (n > 0 && !tensors)) return -1;
  int64_t chunks = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (tensors[i].n < 0) return -1;
    const int64_t c = adamw_chunks(tensors[i].n, 1);
    if (c > kMaxChunks - chunks) return -1;
    chunks += c;
  }
  return chunks;
}

size_t adamw_map_at(int32_t n) { return align_up((size_t)n * sizeof(adamw::Entry), kAlign); }

struct AdamwSpan {
  uintptr_t at, end;
  bool written;
  bool operator<(const AdamwSpan& o) const { return at < o.at; }
};

}  // namespace

extern "C" {

size_t moe_adamw_table_size(const moe_adamw_tensor* tensors, int32_t n_tensors) {
  const int64_t chunks = adamw_list_chunks(tensors, n_tensors);
  if (chunks < 0) return 0;
  const size_t bytes = align_up(adamw_map_at(n_tensors) + (size_t)chunks * 4, kAlign);
  return bytes ? bytes : kAlign;
}

moe_status moe_adamw_table(const moe_adamw_tensor* tensors, int32_t n_tensors, int32_t state_bits,
                           void* table, size_t table_bytes, int64_t* n_chunks) {
  const int64_t chunks = adamw_list_chunks(tensors, n_tensors);
  if (chunks < 0 || (state_bits != 8 && state_bits != 32) || !table || !n_chunks)
    return MOE_ERR_INVALID_ARG;
  if (table_bytes < moe_adamw_table_size(tensors, n_tensors)) return MOE_ERR_WORKSPACE;
  const bool small = state_bits == 8;
  std::vector<AdamwSpan> spans;
  try {
    spans.reserve((size_t)n_tensors * 7);
  } catch (...) {
    snprintf(t_errmsg, sizeof(t_errmsg), "moe_adamw_table: no host memory");
    return MOE_ERR_CUDA;
  }
  uint8_t* image = static_cast<uint8_t*>(table);
  memset(image, 0, table_bytes);
  int32_t* map = reinterpret_cast<int32_t*>(image + adamw_map_at(n_tensors));
  int64_t chunk = 0;
  const int per_chunk = adamw_spans(chunks * adamw::SPAN, small);
  for (int32_t i = 0; i < n_tensors; ++i) {
    const moe_adamw_tensor& s = tensors[i];
    if (s.n == 0) continue;
    if (!s.p || !s.grad || !s.m || !s.v || (small && (!s.m_scale || !s.v_scale)) ||
        (s.grad_bf16 != 0 && s.grad_bf16 != 1) || !std::isfinite(s.weight_decay))
      return MOE_ERR_INVALID_ARG;
    const uintptr_t n = (uintptr_t)s.n, state = small ? 1 : 4, gsz = s.grad_bf16 ? 2 : 4;
    const uintptr_t scales = ((n + adamw::BLOCK - 1) / adamw::BLOCK) * 4;
    const struct {
      const void* at;
      uintptr_t bytes, element, vector;
      bool written;
    } parts[7] = {{s.p, n * 4, 4, 32, true},
                  {s.grad, n * gsz, gsz, gsz * 8, false},
                  {s.m, n * state, state, small ? 16u : 32u, true},
                  {s.v, n * state, state, small ? 16u : 32u, true},
                  {small ? s.m_scale : nullptr, scales, 4, 4, true},
                  {small ? s.v_scale : nullptr, scales, 4, 4, true},
                  {s.p_bf16, n * 2, 2, 16, true}};
    adamw::Entry e;
    memset(&e, 0, sizeof(e));
    e.flags = (s.grad_bf16 ? adamw::GRAD_BF16 : 0) | adamw::ALIGNED | (small ? adamw::STATE8 : 0);
    for (const auto& part : parts) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(part.at);
      if (!at) continue;
      if (at % part.element || at + part.bytes < at) return MOE_ERR_INVALID_ARG;
      if (at % part.vector) e.flags &= ~adamw::ALIGNED;
      spans.push_back(AdamwSpan{at, at + part.bytes, part.written});
    }
    e.p = s.p;
    e.g = s.grad;
    e.m = s.m;
    e.v = s.v;
    e.m_scale = s.m_scale;
    e.v_scale = s.v_scale;
    e.pb = static_cast<__nv_bfloat16*>(s.p_bf16);
    e.n = s.n;
    e.first = (int)chunk;
    e.decay = s.weight_decay;
    e.spans = per_chunk;
    memcpy(image + (size_t)i * sizeof(e), &e, sizeof(e));
    for (int64_t c = adamw_chunks(s.n, per_chunk); c > 0; --c) map[chunk++] = i;
  }
  // nothing that is written may be any other tensor's, or another part of the same
  std::sort(spans.begin(), spans.end());
  uintptr_t read_end = 0, written_end = 0;
  for (const AdamwSpan& s : spans) {
    if (s.at < written_end || (s.written && s.at < read_end)) return MOE_ERR_INVALID_ARG;
    uintptr_t& end = s.written ? written_end : read_end;
    if (s.end > end) end = s.end;
  }
  *n_chunks = chunk;
  return MOE_OK;
}

moe_status moe_adamw(const moe_adamw_desc* desc, const void* table, int32_t n_tensors,
                     int64_t n_chunks, int32_t step, const int32_t* step_dev, const float* lr_dev,
                     cudaStream_t stream) {
  if (!desc || (desc->state_bits != 8 && desc->state_bits != 32) || !std::isfinite(desc->lr) ||
      !(desc->beta1 >= 0.0 && desc->beta1 < 1.0) || !(desc->beta2 >= 0.0 && desc->beta2 < 1.0) ||
      !std::isfinite((float)desc->eps) || !((float)desc->eps >= FLT_MIN))
    return MOE_ERR_INVALID_ARG;
  if (n_tensors < 0 || n_tensors > kMaxTensors || n_chunks < 0 || n_chunks > kMaxChunks ||
      (!step_dev && step < 1) || ((uintptr_t)step_dev & 3) || ((uintptr_t)lr_dev & 3))
    return MOE_ERR_INVALID_ARG;
  if (n_chunks == 0) return MOE_OK;
  if (!given(table) || n_tensors == 0) return MOE_ERR_INVALID_ARG;
  int sms;
  const moe_status rc = device_setup(&sms);
  if (rc != MOE_OK) return rc;
  adamw::Args a;
  memset(&a, 0, sizeof(a));
  a.entries = static_cast<const adamw::Entry*>(table);
  a.tensor_of = reinterpret_cast<const int*>(static_cast<const uint8_t*>(table) +
                                             adamw_map_at(n_tensors));
  a.step_dev = step_dev;
  a.lr_dev = lr_dev;
  a.lr = desc->lr;
  a.beta1 = desc->beta1;
  a.beta2 = desc->beta2;
  a.b1 = (float)desc->beta1;
  a.b2 = (float)desc->beta2;
  a.c1 = (float)(1.0 - desc->beta1);
  a.c2 = (float)(1.0 - desc->beta2);
  a.eps = (float)desc->eps;
  a.seed = (uint32_t)(desc->seed ^ (desc->seed >> 32));
  a.host_step = step_dev ? 0 : step;
  const bool dev = step_dev || lr_dev;
  if (!dev) a.coef = adamw::coef_of(a.lr, a.beta1, a.beta2, a.seed, (uint32_t)step);
  auto* k = desc->state_bits == 8
                ? (dev ? adamw::k_adamw<true, true> : adamw::k_adamw<true, false>)
                : (dev ? adamw::k_adamw<false, true> : adamw::k_adamw<false, false>);
  const size_t smem = desc->state_bits == 8 ? adamw::RING_BYTES : 0;
  if (smem) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute (k_adamw)");
  }
  return launch_chain("k_adamw", k, dim3((unsigned)n_chunks), dim3(adamw::THREADS), smem, stream, a);
}

}  // extern "C"
