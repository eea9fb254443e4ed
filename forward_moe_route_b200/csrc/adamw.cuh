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
// Bound by memory: 24 to 28 bytes an element with fp32 states, 14 with 8-bit
// ones.  A chunk of one tensor's elements is a block's; a thread takes
// 8 elements in a row: one 32-byte access for each fp32 operand, and the 16
// lanes that share a scale find its maximum with four shuffles.  A table in
// device memory, written once per list, names the tensor of each chunk.
#pragma once

#include "common.cuh"

namespace moe {
namespace adamw {

constexpr int THREADS = 256;
constexpr int PER = 8;                       // elements of a thread
constexpr int SPAN = THREADS * PER;          // elements of a block at a time
constexpr int CHUNK = SPAN, CHUNK8 = 2 * SPAN;   // elements of a block, fp32 and 8-bit states
constexpr int BLOCK = 128;                   // elements that share a scale
constexpr int ROUNDS = 7;
constexpr uint32_t KEY_STEP = 0x9E3779B9u;   // Philox key increment (Weyl)
constexpr uint32_t PHILOX_M = 0xD256D193u;

constexpr int GRAD_BF16 = 1;                 // Entry::flags
constexpr int ALIGNED = 2;                   // every address fits the vector accesses
constexpr int STATE8 = 4;

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
  int spare;
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

// E4M3 code of |x| <= 448 (up to rounding) in the top byte, rounded up with the
// probability of its distance from the code below; r: 16 random bits, shifted
// left by 4.  The 20 mantissa bits below E4M3's three decide against them: a
// carry makes the next code.  Only for |x| >= 2^-6.
template <bool SIGNED>
__device__ __forceinline__ uint32_t encode_top(float x, uint32_t r4) {
  const uint32_t a = __float_as_uint(x) & (SIGNED ? 0x7fffffffu : 0xffffffffu);
  const uint32_t c = min(a - (960u << 20) + r4, 0x07efffffu) << 4;
  return SIGNED ? c | (__float_as_uint(x) & 0x80000000u) : c;
}
// the same below 2^-6, where codes are multiples of 2^-9
__device__ __forceinline__ uint32_t encode_small_top(float x, uint32_t r4) {
  const uint32_t c = (uint32_t)fmaf(fabsf(x), 512.0f, (float)r4 * 0x1p-20f);
  return (c << 24) | (__float_as_uint(x) & 0x80000000u);
}

// 8 codes of x * inv; r4(j): the random bits of element j.  Without SIGNED, x >= 0
// and a positive x is not held as 0.
template <bool SIGNED, typename R>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv, float most, R r4) {
  uint32_t c[8];
  float y[8], least = 1.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = x[j] * inv;
    c[j] = encode_top<SIGNED>(y[j], r4(j));
    least = fminf(least, fabsf(y[j]));
  }
  if (least < 0.015625f) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (fabsf(y[j]) < 0.015625f) {
        c[j] = encode_small_top(y[j], r4(j));
        if (!SIGNED && x[j] > 0.f) c[j] = max(c[j], 1u << 24);
      }
  }
  // an infinity or a NaN leaves its block without a scale: NaN codes
  if (!(most <= 3.402823466e38f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = 0x7f000000u;
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

// the larger magnitude; a NaN wins
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max8(const float (&x)[8]) {
  float most = fabsf(x[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) most = max_nan(most, fabsf(x[j]));
  return most;
}
// over the 16 lanes that share a scale
__device__ __forceinline__ float block_max(float most) {
#pragma unroll
  for (int o = 8; o; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
  return most;
}

// Rounded roots of 8 values >= 0 without a branch for each: r = v y with y the
// hardware's approximation of v^-1/2 is close enough for one Newton step,
// r + (v - r r) y / 2 with the residual exact in a fused multiply-add, to round
// to the nearest float (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990).  Zeros come out as zeros; values whose
// residual would be subnormal, infinities and NaN take the general root.
__device__ __forceinline__ float roots8(const float (&v)[8], float (&root)[8]) {
  constexpr float LEAST = 0x1p-100f;
  float least = v[0];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(v[j], LEAST)));
    const float r = v[j] * y;
    root[j] = fmaf(fmaf(-r, r, v[j]), 0.5f * y, r);
    least = fminf(least, v[j]);
  }
  float most = max8(root);
  if (!(most <= 3.402823466e38f) || (least < LEAST && most > 0.f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) root[j] = __fsqrt_rn(v[j]);
    most = max8(root);
  }
  return most;
}

template <bool STATES8, bool FROM_DEVICE>
__global__ void __launch_bounds__(THREADS, 4) k_adamw(const Args a) {
  grid_dep_sync();
  __shared__ Coef from_device;
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
  const float keep = fmaf(-c.lr, e.decay, 1.0f);
#pragma unroll 1
  for (int part = 0; part < (STATES8 ? CHUNK8 : CHUNK); part += SPAN) {
    const long long at = (long long)((int)blockIdx.x - e.first) * (STATES8 ? CHUNK8 : CHUNK) +
                         part + threadIdx.x * PER;
    const int here = (int)min((long long)PER, max(0ll, e.n - at));   // elements of this thread
    const bool whole = (e.flags & ALIGNED) && here == PER;
    float p[8], g[8], m[8], v[8];
    if (whole) {
      load8(e.p + at, p);
      if (e.flags & GRAD_BF16) {
        const uint4 raw = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(e.g) + at);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g[2 * j] = __uint_as_float(w[j] << 16);
          g[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      } else {
        load8(static_cast<const float*>(e.g) + at, g);
      }
      if (STATES8) {
        const uint2 cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(e.m) + at);
        const uint2 cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(e.v) + at);
        const float sm = e.m_scale[at / BLOCK], sv = e.v_scale[at / BLOCK];
        decode4(cm.x, sm, m);
        decode4(cm.y, sm, m + 4);
        decode4(cv.x, sv, v);
        decode4(cv.y, sv, v + 4);
      } else {
        load8(static_cast<const float*>(e.m) + at, m);
        load8(static_cast<const float*>(e.v) + at, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = g[j] = m[j] = v[j] = 0.f;
        if (j >= here) continue;
        p[j] = e.p[at + j];
        g[j] = (e.flags & GRAD_BF16)
                   ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.g)[at + j])
                   : static_cast<const float*>(e.g)[at + j];
        if (STATES8) {
          float one[4];
          decode4(static_cast<const uint8_t*>(e.m)[at + j], e.m_scale[at / BLOCK], one);
          m[j] = one[0];
          decode4(static_cast<const uint8_t*>(e.v)[at + j], e.v_scale[at / BLOCK], one);
          v[j] = one[0];
        } else {
          m[j] = static_cast<const float*>(e.m)[at + j];
          v[j] = static_cast<const float*>(e.v)[at + j];
        }
      }
    }

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

    if (whole) {
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
      if (whole) {
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

    // scale and its inverse; a block below 2^-100 counts as zero (448 / max
    // would leave fp32's range)
    const float most_m = block_max(max8(m)), most_v = block_max(here_v);
    const bool there_m = !(most_m < 0x1p-100f), there_v = !(most_v < 0x1p-100f);
    const float inv_m = there_m ? __frcp_rn(most_m) * 448.0f : 0.f;
    const float inv_v = there_v ? __frcp_rn(most_v) * 448.0f : 0.f;
    if ((threadIdx.x & 15) == 0 && here > 0) {
      e.m_scale[at / BLOCK] = there_m ? most_m * (1.0f / 448.0f) : 0.f;
      e.v_scale[at / BLOCK] = there_v ? most_v * (1.0f / 448.0f) : 0.f;
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
    const uint2 cm = encode8<true>(m, inv_m, most_m,
                                    [&](int j) { return (word[j] << 4) & 0xffff0u; });
    const uint2 cv = encode8<false>(root, inv_v, most_v,
                                   [&](int j) { return (word[j] >> 12) & 0xffff0u; });
    if (whole) {
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

}  // namespace adamw
}  // namespace moe
