// One AdamW step over a list of tensors in one launch.
//
//   m' = b1 m + (1 - b1) g,        v' = b2 v + (1 - b2) g^2
//   p' = (1 - lr wd) p - lr / (1 - b1^t) m' / (sqrt(v' / (1 - b2^t)) + eps)
//
// in fp32 for every element of every tensor; p' is also rounded to bf16, and
// m', v' are kept in fp32 or in 8 bits.
//
// 8-bit states.  128 elements in a row share a scale, max |x| / 448, and hold
// x / scale as E4M3 codes; the second moment is held as its root, which halves
// the range of exponents it has to cover.  Codes are rounded up with the
// probability of the distance to the code below (the moments are averages over
// many steps: increments below half a code step would be lost for good by
// rounding to nearest).  A positive root never becomes code 0, so no element
// whose gradient was ever seen divides by eps alone.  The random bits are a
// counter-based generator's (Philox-2x32 with 7 rounds; Salmon et al.,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011) keyed by seed and
// step and counted by the element's place, so a step gives the same result
// however it is split.
//
// Bytes an element, with bf16 gradients and the bf16 copy: 28 with fp32 states, 16.1
// with 8-bit ones.  fp32 states are bound by memory (360M elements 1460 us, 6.9
// TB/s); with 8-bit ones the arithmetic of decoding, rounding and the generator
// comes near it (1050 to 1110 us, 5.5 to 5.2 TB/s, 75 instructions an element, the
// schedulers issuing in 73% of their active cycles).  Step and rate read from device
// memory cost every block the coefficients before its first load: 1463 instead of
// 1458 us, and 7.5 instead of 6.4 us on 96 tensors of 20000.  A chunk of one tensor's elements is a
// block's; a thread takes 8 elements in a row: one 32-byte access for each fp32
// operand, and the 16 lanes that share a scale find its maximum with four
// shuffles.  A table in device memory, written once per list, names the tensor of
// each chunk.
#pragma once

#include "bulk.cuh"
#include "common.cuh"

namespace moe {
namespace adamw {

constexpr int THREADS = 256;
constexpr int PER = 8;                       // elements of a thread
constexpr int SPAN = THREADS * PER;          // elements of a block at a time
constexpr int BLOCK = 128;                   // elements that share a scale
constexpr int ROUNDS = 7;
constexpr uint32_t KEY_STEP = 0x9E3779B9u;   // Philox key increment (Weyl)
constexpr uint32_t PHILOX_M = 0xD256D193u;

constexpr int GRAD_BF16 = 1;                 // Entry::flags
constexpr int ALIGNED = 2;                   // every address fits the vector accesses
constexpr int STATE8 = 4;

// The ring of spans of a block with 8-bit states: p, the gradient and both codes of
// a span.
constexpr uint32_t RING_BYTES = 49152;       // 3 spans with bf16 gradients, 2 with fp32
constexpr int RING_MAX = 3;
__host__ __device__ constexpr uint32_t span_bytes(bool bf16) {
  return SPAN * ((bf16 ? 2 : 4) + 4 + 2);
}

struct alignas(16) Entry {
  float* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  __nv_bfloat16* pb;
  long long n;
  int first;                                 // its first chunk
  int flags;
  float decay;
  int spans;                                 // spans of each of its chunks
};

// What a step adds to the hyperparameters.
struct Coef {
  float lr, alpha, root_mul;                 // lr / (1 - b1^t), (1 - b2^t)^-1/2
  uint32_t key[ROUNDS];
};

struct Args {
  const Entry* entries;
  const int* tensor_of;                      // [chunks]
  const int* step_dev;                       // read instead of coef when given
  const float* lr_dev;
  double lr, beta1, beta2;
  float b1, b2, c1, c2, eps;                 // betas and 1 - betas
  uint32_t seed;
  int host_step;                             // without step_dev
  Coef coef;
};

// b^t by squaring: t is at most 31 bits, and the relative error t 2^-53 is far
// below the fp32 rounding of the result
__host__ __device__ inline double power(double b, uint32_t t) {
  double r = 1.0;
  for (; t; t >>= 1, b *= b)
    if (t & 1u) r *= b;
  return r;
}
__host__ __device__ inline Coef coef_of(double lr, double beta1, double beta2, uint32_t seed,
                                        uint32_t step) {
  Coef c;
  c.lr = (float)lr;
  c.alpha = (float)(lr / (1.0 - power(beta1, step)));
  c.root_mul = (float)(1.0 / sqrt(1.0 - power(beta2, step)));
  uint32_t key = seed + step * KEY_STEP;
  for (int r = 0; r < ROUNDS; ++r, key += KEY_STEP) c.key[r] = key;
  return c;
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

__device__ __forceinline__ void load4(const void* p, uint32_t* v) {
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "l"(p));
}
__device__ __forceinline__ void load2(const void* p, uint32_t* v) {
  asm volatile("ld.global.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p));
}

// sqrt(x) and 1 / x to within 2^-23 (x > 0 and normal for the inverse, 0 beyond
// 2^126): next to the rounding of the p that they move by lr at most, nothing
__device__ __forceinline__ float root_of(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float inverse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / x with one Newton step on the approximation (Markstein, as for roots8): the
// nearest float for every x from 2^-100 to 2^14, compared one by one with __frcp_rn,
// which the other branch of encode8 takes
__device__ __forceinline__ float inverse_step(float x) {
  const float near = inverse(x);
  return fmaf(fmaf(-x, near, 1.0f), near, near);
}

// The larger and the smaller magnitude of three; a NaN wins the maximum.
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max8(const float (&x)[8]) {
  return max_nan(max_nan(max_nan(x[0], x[1], x[2]), x[3], x[4]), x[5], max_nan(x[6], x[7], 0.f));
}
__device__ __forceinline__ float min8(const float (&x)[8]) {
  return min3(min3(min3(x[0], x[1], x[2]), x[3], x[4]), x[5], min3(x[6], x[7], x[7]));
}
// over the 16 lanes that share a scale
__device__ __forceinline__ float block_max(float most) {
#pragma unroll
  for (int o = 8; o; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o), 0.f);
  return most;
}

// E4M3 codes, each in the top byte of a word and rounded up with the probability
// of its distance from the code below; r4: 16 random bits, shifted left by 4.
// From 2^-6 on a code is the upper bits of the float's exponent and mantissa less
// 960; the 20 mantissa bits below decide against the random ones, a carry makes
// the next code.
__device__ __forceinline__ uint32_t encode(float y, uint32_t r4) {
  const float a = fabsf(y);
  uint32_t c = min(__float_as_uint(a) - (960u << 20) + r4, 0x07efffffu) << 4;
  // below it codes are multiples of 2^-9
  if (a < 0x1p-6f) c = (uint32_t)fmaf(a, 512.0f, (float)r4 * 0x1p-20f) << 24;
  return c | (__float_as_uint(y) & 0x80000000u);
}

// 8 codes of x 448 / most in blocks whose largest magnitude is `most`, or of 0
// where that is below 2^-100 (448 / most would leave fp32's range); r4(j): the
// random bits of element j.  Without SIGNED, x >= 0 and a positive x is not held
// as 0.
//
// The common case has most <= 2^14 and all of the eight products at 2^-6 or above.
// Its inverse is the hardware's approximation and one Newton step, which rounds it
// (inverse_step).  Scaled by 2^-120 too (an exact factor, as 448 / most is not below 2^-6),
// the product's bits are those of `encode` less 960 << 20 without subtracting
// them.
template <bool SIGNED, typename R>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float most, R r4) {
  uint32_t c[8];
  float y[8];
  const float inv120 = inverse_step(most) * 448.0f * 0x1p-120f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = (SIGNED ? fabsf(x[j]) : x[j]) * inv120;
    c[j] = min(__float_as_uint(y[j]) + r4(j), 0x07efffffu) << 4;
    if (SIGNED) c[j] |= __float_as_uint(x[j]) & 0x80000000u;
  }
  if (!(min8(y) >= 0x1p-126f && most >= 0x1p-100f && most <= 0x1p14f)) {
    const float inv = most < 0x1p-100f ? 0.f : __frcp_rn(most) * 448.0f;
    const bool bad = !(most <= 3.402823466e38f);    // an infinity or a NaN: no scale, NaN codes
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = bad ? 0x7f000000u : encode(x[j] * inv, r4(j));
      if (!SIGNED && x[j] > 0.f) c[j] = max(c[j], 1u << 24);
    }
  }
  auto top4 = [](const uint32_t* b) {
    return __byte_perm(__byte_perm(b[0], b[1], 0x0073), __byte_perm(b[2], b[3], 0x0073), 0x5410);
  };
  return make_uint2(top4(c), top4(c + 4));
}

__device__ __forceinline__ void decode4(uint32_t codes, float s, float* out) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw raw =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> (16 * h)), __NV_E4M3);
    const float2 f = __half22float2(__half2(raw));
    out[2 * h] = f.x * s;
    out[2 * h + 1] = f.y * s;
  }
}

// Rounded roots of 8 values >= 0 without a branch for each: r = v y with y the
// hardware's approximation of v^-1/2 is close enough for one Newton step,
// r + (v - r r) y / 2 with the residual exact in a fused multiply-add, to round
// to the nearest float (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990).  Zeros come out as zeros; values whose
// residual would be subnormal, infinities and NaN take the general root.  Compared
// with __fsqrt_rn for every float from 0 up.
__device__ __forceinline__ float roots8(const float (&v)[8], float (&root)[8]) {
  constexpr float LEAST = 0x1p-100f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(v[j], LEAST)));
    const float r = v[j] * y;
    root[j] = fmaf(fmaf(-r, r, v[j]), 0.5f * y, r);
  }
  float most = max8(root);
  if (!(most <= 3.402823466e38f) || (min8(v) < LEAST && most > 0.f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) root[j] = __fsqrt_rn(v[j]);
    most = max8(root);
  }
  return most;
}

// A thread's 8 elements as they are stored.  WHOLE: the block's are all there and
// aligned; GRAD: 0 fp32, 1 bf16, 2 as the entry says.
template <bool STATES8, bool WHOLE, int GRAD>
struct Held {
  static constexpr int STATE_WORDS = STATES8 ? 2 : 8;
  float p[8], m_scale, v_scale;
  uint32_t g[8];                             // bf16: the first four
  uint32_t m[STATE_WORDS], v[STATE_WORDS];
  int here;                                  // elements that are there
  bool vectors;                              // all, and aligned
  __device__ __forceinline__ void load(const Entry& e, long long at) {
    here = WHOLE ? PER : (int)min((long long)PER, max(0ll, e.n - at));
    vectors = WHOLE || ((e.flags & ALIGNED) && here == PER);
    const bool bf16 = GRAD == 2 ? (e.flags & GRAD_BF16) != 0 : GRAD;
    if (STATES8 && (WHOLE || here > 0)) {
      m_scale = e.m_scale[at / BLOCK];
      v_scale = e.v_scale[at / BLOCK];
    }
    if (vectors) {
      load8(e.p + at, p);
      if (bf16) load4(static_cast<const __nv_bfloat16*>(e.g) + at, g);
      else load8(static_cast<const float*>(e.g) + at, reinterpret_cast<float(&)[8]>(g));
      if constexpr (STATES8) {
        load2(static_cast<const uint8_t*>(e.m) + at, m);
        load2(static_cast<const uint8_t*>(e.v) + at, v);
      } else {
        load8(static_cast<const float*>(e.m) + at, reinterpret_cast<float(&)[8]>(m));
        load8(static_cast<const float*>(e.v) + at, reinterpret_cast<float(&)[8]>(v));
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < STATE_WORDS; ++i) m[i] = v[i] = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool there = j < here;
      p[j] = there ? e.p[at + j] : 0.f;
      if (bf16) {
        const uint32_t x = there ? static_cast<const uint16_t*>(e.g)[at + j] : 0u;
        if (j & 1) g[j >> 1] |= x << 16;
        else g[j >> 1] = x;
      }
      if constexpr (STATES8) {
        if (there) {
          m[j >> 2] |= (uint32_t)static_cast<const uint8_t*>(e.m)[at + j] << (8 * (j & 3));
          v[j >> 2] |= (uint32_t)static_cast<const uint8_t*>(e.v)[at + j] << (8 * (j & 3));
        }
      } else {
        m[j] = there ? static_cast<const uint32_t*>(e.m)[at + j] : 0u;
        v[j] = there ? static_cast<const uint32_t*>(e.v)[at + j] : 0u;
      }
    }
    if (!bf16)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        g[j] = j < here ? static_cast<const uint32_t*>(e.g)[at + j] : 0u;
    if (here <= 0) m_scale = v_scale = 0.f;
  }
  // from a span in shared memory; the scales are loaded already
  __device__ __forceinline__ void load_span(const uint8_t* span) {
    constexpr uint32_t GB = GRAD == 1 ? 2 : 4;
    const int at = threadIdx.x * PER;
    here = PER;
    vectors = true;
    const float4* ps = reinterpret_cast<const float4*>(span) + at / 4;
    const float4 a = ps[0], b = ps[1];
    p[0] = a.x; p[1] = a.y; p[2] = a.z; p[3] = a.w;
    p[4] = b.x; p[5] = b.y; p[6] = b.z; p[7] = b.w;
    const uint4* gs = reinterpret_cast<const uint4*>(span + SPAN * 4 + at * GB);
#pragma unroll
    for (int i = 0; i < (int)GB / 2; ++i) {
      const uint4 x = gs[i];
      g[4 * i] = x.x; g[4 * i + 1] = x.y; g[4 * i + 2] = x.z; g[4 * i + 3] = x.w;
    }
    const uint2 x = *reinterpret_cast<const uint2*>(span + SPAN * (4 + GB) + at);
    const uint2 y = *reinterpret_cast<const uint2*>(span + SPAN * (5 + GB) + at);
    m[0] = x.x; m[1] = x.y;
    v[0] = y.x; v[1] = y.y;
  }
  __device__ __forceinline__ void values(const Entry& e, float (&gf)[8], float (&mf)[8],
                                         float (&vf)[8]) const {
    const bool bf16 = GRAD == 2 ? (e.flags & GRAD_BF16) != 0 : GRAD;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      gf[j] = __uint_as_float(!bf16 ? g[j] : (j & 1) ? g[j >> 1] & 0xffff0000u : g[j >> 1] << 16);
    if constexpr (STATES8) {
      decode4(m[0], m_scale, mf);
      decode4(m[1], m_scale, mf + 4);
      decode4(v[0], v_scale, vf);
      decode4(v[1], v_scale, vf + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mf[j] = __uint_as_float(m[j]);
        vf[j] = __uint_as_float(v[j]);
      }
    }
  }
};

// The chunk of block blockIdx.x, tensor t of the list.  Whole chunks with 8-bit
// states come through a ring in shared memory, filled with bulk copies: what the
// threads hold in registers for a span, and for the next, is too little in flight
// to cover memory's latency beside 75 instructions an element (1146 us instead of
// 1074 us for 360M elements, measured in turn).
template <bool STATES8, bool WHOLE, int GRAD>
__device__ __forceinline__ void step_chunk(const Args& a, const Coef& c, const Entry& e, int t,
                                           uint8_t* ring, uint64_t* full, volatile int* abort) {
  constexpr bool RING = STATES8 && WHOLE;
  const float keep = fmaf(-c.lr, e.decay, 1.0f);
  const int size = e.spans * SPAN;
  const long long first = (long long)((int)blockIdx.x - e.first) * size;
  constexpr uint32_t BYTES = span_bytes(GRAD == 1);
  constexpr int STAGES = RING_BYTES / BYTES;
  static_assert(STAGES <= RING_MAX, "");
  auto fetch = [&](int i) {
    uint64_t* bar = &full[i % STAGES];
    uint8_t* to = ring + (i % STAGES) * BYTES;
    const long long from = first + (long long)i * SPAN;
    constexpr uint32_t GB = GRAD == 1 ? 2 : 4;
    mbar_arrive_expect_tx(bar, BYTES);
    bulk_load_1d(to, e.p + from, SPAN * 4, bar);
    bulk_load_1d(to + SPAN * 4, static_cast<const uint8_t*>(e.g) + from * GB, SPAN * GB, bar);
    bulk_load_1d(to + SPAN * (4 + GB), static_cast<const uint8_t*>(e.m) + from, SPAN, bar);
    bulk_load_1d(to + SPAN * (5 + GB), static_cast<const uint8_t*>(e.v) + from, SPAN, bar);
  };
  if constexpr (RING) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
      *abort = 0;
      fence_barrier_init();
      fence_proxy_async_smem();
      for (int i = 0; i < STAGES && i < e.spans; ++i) fetch(i);
    }
    __syncthreads();
  }
  Held<STATES8, WHOLE, GRAD> held;
  float m_scale = 0.f, v_scale = 0.f;        // of the next span
  const long long mine = first + threadIdx.x * PER;
  if constexpr (RING) {
    m_scale = e.m_scale[mine / BLOCK];
    v_scale = e.v_scale[mine / BLOCK];
  }
#pragma unroll 1
  for (int i = 0; i < e.spans && first + (long long)i * SPAN < e.n; ++i) {
    const long long at = mine + (long long)i * SPAN;
    if constexpr (RING) {
      // a wait that ran out is reported, and the rest of the chunk left as it is
      const bool there = mbar_wait(&full[i % STAGES], (uint32_t)(i / STAGES) & 1u, abort);
      held.load_span(ring + (i % STAGES) * BYTES);
      held.m_scale = m_scale;
      held.v_scale = v_scale;
      if (i + 1 < e.spans) {
        m_scale = e.m_scale[(at + SPAN) / BLOCK];
        v_scale = e.v_scale[(at + SPAN) / BLOCK];
      }
      if (!__syncthreads_and(there)) {         // the span is in registers
        const int issued = min(i + STAGES, e.spans);
        if (threadIdx.x == 0)
          bulk_drain(full, issued % STAGES, (uint32_t)(issued / STAGES) & 1u, STAGES);
        return;
      }
      if (threadIdx.x == 0 && i + STAGES < e.spans) fetch(i + STAGES);
    } else {
      held.load(e, at);
    }
    const int here = held.here;
    const bool vectors = held.vectors;
    float (&p)[8] = held.p;
    float g[8], m[8], v[8];
    held.values(e, g, m, v);

    float root[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (STATES8) {
        // each operation of the formulas rounded by itself: the codes are drawn
        // from these values, and a last bit that differs can change a code
        v[j] = __fmul_rn(v[j], v[j]);
        m[j] = __fadd_rn(__fmul_rn(a.b1, m[j]), __fmul_rn(a.c1, g[j]));
        v[j] = __fadd_rn(__fmul_rn(a.b2, v[j]), __fmul_rn(a.c2, __fmul_rn(g[j], g[j])));
      } else {
        m[j] = fmaf(a.c1, g[j], a.b1 * m[j]);
        v[j] = fmaf(a.c2, g[j] * g[j], a.b2 * v[j]);
        root[j] = root_of(v[j]);
      }
    }
    const float here_v = STATES8 ? roots8(v, root) : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      p[j] = fmaf(p[j], keep, -(m[j] * c.alpha) * inverse(fmaf(root[j], c.root_mul, a.eps)));

    if (vectors) {
      store8(e.p + at, p);
      if (e.pb) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(p[2 * j], p[2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(e.pb + at) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < here) {
          e.p[at + j] = p[j];
          if (e.pb) e.pb[at + j] = __float2bfloat16_rn(p[j]);
        }
    }
    if (!STATES8) {
      if (vectors) {
        store8(static_cast<float*>(e.m) + at, m);
        store8(static_cast<float*>(e.v) + at, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < here) {
            static_cast<float*>(e.m)[at + j] = m[j];
            static_cast<float*>(e.v)[at + j] = v[j];
          }
      }
      continue;
    }

    const float most_m = block_max(max8(m)), most_v = block_max(here_v);
    if ((threadIdx.x & 15) == 0 && here > 0) {
      e.m_scale[at / BLOCK] = most_m < 0x1p-100f ? 0.f : most_m * (1.0f / 448.0f);
      e.v_scale[at / BLOCK] = most_v < 0x1p-100f ? 0.f : most_v * (1.0f / 448.0f);
    }
    uint32_t word[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const unsigned long long pair = ((unsigned long long)at >> 1) + q;
      uint32_t x = (uint32_t)pair, y = ((uint32_t)t << 8) ^ (uint32_t)(pair >> 32);
#pragma unroll
      for (int r = 0; r < ROUNDS; ++r) {
        const unsigned long long prod = (unsigned long long)x * PHILOX_M;
        x = (uint32_t)(prod >> 32) ^ c.key[r] ^ y;
        y = (uint32_t)prod;
      }
      word[2 * q] = x;
      word[2 * q + 1] = y;
    }
    const uint2 cm = encode8<true>(m, most_m,
                                   [&](int j) { return (word[j] << 4) & 0xffff0u; });
    const uint2 cv = encode8<false>(root, most_v,
                                   [&](int j) { return (word[j] >> 12) & 0xffff0u; });
    if (vectors) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(e.m) + at) = cm;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(e.v) + at) = cv;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < here) {
          static_cast<uint8_t*>(e.m)[at + j] = (uint8_t)((j < 4 ? cm.x : cm.y) >> (8 * (j & 3)));
          static_cast<uint8_t*>(e.v)[at + j] = (uint8_t)((j < 4 ? cv.x : cv.y) >> (8 * (j & 3)));
        }
    }
  }
}

template <bool STATES8, bool FROM_DEVICE>
__global__ void __launch_bounds__(THREADS, 4) k_adamw(const Args a) {
  grid_dep_sync();
  __shared__ Coef from_device;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[RING_MAX];
  __shared__ int abort_word;
  const int t = a.tensor_of[blockIdx.x];
  const Entry e = a.entries[t];
  if (((e.flags & STATE8) != 0) != STATES8) {    // a table of the other kind
    if (threadIdx.x == 0) set_status(MOE_ERR_DEVICE_CHECK);
    return;
  }
  if (FROM_DEVICE) {
    const int step = a.step_dev ? *a.step_dev : a.host_step;
    if (step < 1) {
      if (threadIdx.x == 0) set_status(MOE_ERR_DEVICE_CHECK);
      return;
    }
    if (threadIdx.x == 0)
      from_device = coef_of(a.lr_dev ? (double)*a.lr_dev : a.lr, a.beta1, a.beta2, a.seed,
                            (uint32_t)step);
    __syncthreads();
  }
  const Coef& c = FROM_DEVICE ? from_device : a.coef;
  // Blocks with a tensor's end, or of a tensor that is not aligned, look at every
  // element.  One loop for both would issue the element accesses with false
  // predicates in every block: 81 instructions an element with 8-bit states
  // instead of 75.
  const int size = e.spans * SPAN;
  if (!(e.flags & ALIGNED) || e.n - (long long)((int)blockIdx.x - e.first) * size < size)
    step_chunk<STATES8, false, 2>(a, c, e, t, ring, full, &abort_word);
  else if (e.flags & GRAD_BF16)
    step_chunk<STATES8, true, 1>(a, c, e, t, ring, full, &abort_word);
  else
    step_chunk<STATES8, true, 0>(a, c, e, t, ring, full, &abort_word);
}

}  // namespace adamw
}  // namespace moe
