// AdamW over many tensors at once, with the moments in 32 or in 8 bits, and
// the global norm of the gradients with its clipping.
//
//   t <- t + 1,  c = min(1, max_norm / (|g| + 1e-6)),  g' = c g
//   m <- b1 m + (1 - b1) g',  v <- b2 v + (1 - b2) g'^2
//   w <- w (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// w is an f32 weight, or the f32 master of a bf16 weight that gets its
// rounding.  8-bit moments: m and sqrt(v) as E4M3 codes, one E8M0 scale 2^e per
// 32 elements with e the smallest that keeps the block's largest value at or
// below 448 2^e.  (sqrt(v), because the codes span 2^17 from the smallest to
// the largest and v's elements twice as many octaves.)  Codes are rounded up or
// down by 16 random bits: with b2 = 0.999 a step changes sqrt(v) by 0.05%, a
// code is 6% to 12% wide, and rounding to the nearest would keep it where it is
// for ever; by chance it moves by as much on average as it should.  A sqrt(v)
// that is not zero keeps the smallest code, so that a weight with m and without
// gradient does not divide by eps.
//
// The state after a step is the one of the 64-bit formula: m is formed with
// the rounding errors of its first product (b1 m and (1 - b1) g' may cancel),
// good to two steps of fp32, and where that comes within 8 steps of the point
// at which the random bits turn a code (or the block's largest value one of its
// scale), the element is done again in 64 bits.  That happens to one element in
// 30,000; it matters, because gradients and codes of few bits put sums exactly
// on those points more often than chance would.
//
// Memory bound: 28 bytes per element with bf16 weights and 32-bit moments, 16
// with 8-bit ones.  One launch for all tensors: a table of (tensor, chunk),
// built once, splits them into chunks of CHUNK elements, and the gradients'
// addresses (they differ from step to step) come as a kernel parameter.  The
// norm and the step's scalars are kernels in front of it that it overlaps.
//
// Measured, a step per graph: 99.6 million bf16 weights in four tensors, clipped,
// 483 us: the norm 47 (4.2 TB/s, while the step before still writes back), the
// step 437 (6.4 TB/s; a plain copy reaches 6.1).  With 8-bit moments 352 us, the
// step 303 (5.3 TB/s, with 83 instructions per element at 63% of the issue slots).
// 95,000 weights 6.2 us.
#include <cmath>

#include "common.cuh"
#include "host_common.h"

namespace moeglu {
namespace adamw {

constexpr int THREADS = 256, PER = 8, CHUNK = 2048;  // elements per thread at a time, per chunk
// gradient addresses in a launch's parameters (32,764 bytes at most, each byte copied per launch)
constexpr int FEW = 64, SOME = 512, MANY = 4000;
constexpr int BLOCK = 32;                            // elements per scale
constexpr int MAX_PARTS = 2048;                      // CTAs of the norm's kernel
constexpr int NEAR = 8;  // fp32 steps around a turning point inside which 64 bits decide

struct Entry {
  uint32_t tensor, chunk;
};
template <int N>
struct Grads {
  const void* p[N];
};

// What a step's scalars are, written once per step.
struct Short {
  float b1h, b1l, a1h, a1l, b2f, a2f;  // a1 and a2 with c and c^2
  float down;                          // a power of two that the gradients are multiplied by first
  float step, root, lr, eps;           // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t key;
  int32_t skip;  // the gradients' norm is not finite
};
struct Scalars : Short {
  double b1, a1, b2, a2, c;  // a = 1 - b; c without `down`
};
// the workspace: the scalars, then the norm's partial sums
constexpr size_t PARTS_AT = 256;

// A published 32-bit hash of two multiplications (shifts and factors are those of
// Wellons' "lowbias32"); the header states it, callers may form the bits themselves.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

// ---------------------------------------------------------------------------
// Loads and stores of PER consecutive elements: whole vectors where the
// address allows, element by element at a tensor's end or off alignment.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void ld_f32x8(const float* p, float* v) {
  asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void st_f32x8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
               "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ bool on(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// n: elements left from p on (at least 1); whole: PER of them and aligned
__device__ __forceinline__ void load8(const float* p, int64_t n, bool whole, float* v) {
  if (whole) {
    ld_f32x8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
}
__device__ __forceinline__ void unpack8(uint4 q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int64_t n, bool whole, float* v) {
  if (whole) {
    unpack8(*reinterpret_cast<const uint4*>(p), v);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ void store8(float* p, int64_t n, bool whole, const float* v) {
  if (whole) {
    st_f32x8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int64_t n, bool whole, const float* v) {
  if (whole) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                              pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < n) p[i] = __float2bfloat16_rn(v[i]);
  }
}

// ---------------------------------------------------------------------------
// The gradients' norm
// ---------------------------------------------------------------------------
__device__ __forceinline__ double warp_sum(double s) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  return s;
}

// parts[CTA] = sum of squares of its chunks, AT_ONCE of them loaded together.
// Eight squares are added in fp32 (of bf16 values they are exact), these sums
// with their rounding errors.
constexpr int AT_ONCE = 2;
template <int N>
__global__ void __launch_bounds__(THREADS, 8) k_adamw_norm(const __grid_constant__ Grads<N> grads,
                                                        const moe_adamw_tensor_t* __restrict__ tensors,
                                                        const Entry* __restrict__ table, uint32_t chunks, int first,
                                                        double* __restrict__ parts) {
  launch_dependents();
  float hi = 0.0f, lo = 0.0f;
  for (uint32_t i = blockIdx.x; i < chunks; i += AT_ONCE * gridDim.x) {
    Entry e[AT_ONCE];
    float g[AT_ONCE][PER];
    bool packed[AT_ONCE];  // g holds eight bf16 values in its first four words: taken apart when all loads are under way
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) e[k] = i + k * gridDim.x < chunks ? table[i + k * gridDim.x] : Entry{0xFFFFFFFFu, 0};
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      int64_t n = 0, at = 0;
      packed[k] = false;
      if (e[k].tensor != 0xFFFFFFFFu) {
        at = (int64_t)e[k].chunk * CHUNK + threadIdx.x * PER;
        n = tensors[e[k].tensor].n - at;
      }
      if (n > 0) {
        const void* p = grads.p[e[k].tensor - first];
        if (tensors[e[k].tensor].grad_bf16) {
          const auto* q = static_cast<const __nv_bfloat16*>(p) + at;
          if (n >= PER && on(q, 16)) {
            packed[k] = true;
            asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(g[k][0]), "=f"(g[k][1]), "=f"(g[k][2]), "=f"(g[k][3]) : "l"(q));
          } else {
            load8(q, n, false, g[k]);
          }
        } else {
          const auto* q = static_cast<const float*>(p) + at;
          load8(q, n, n >= PER && on(q, 32), g[k]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) g[k][j] = 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k)
      if (packed[k])
        unpack8(make_uint4(__float_as_uint(g[k][0]), __float_as_uint(g[k][1]), __float_as_uint(g[k][2]), __float_as_uint(g[k][3])),
                g[k]);
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      float q = g[k][0] * g[k][0];
#pragma unroll
      for (int j = 1; j < PER; ++j) q = fmaf(g[k][j], g[k][j], q);
      const float s = hi + q, bb = s - hi;
      lo += (hi - (s - bb)) + (q - bb);
      hi = s;
    }
  }
  // (an infinite or NaN hi stays so: its error term, NaN, is left out)
  double s = warp_sum(fabsf(hi) <= 3.4e38f ? (double)hi + (double)lo : (double)hi);
  __shared__ double warp[THREADS / 32];
  if ((threadIdx.x & 31) == 0) warp[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < THREADS / 32; ++w) s += warp[w];
    parts[blockIdx.x] = s;
  }
}

// sqrt(x) and a / x to about 2^-45: an fp32 guess and one step of Newton's
// method in 64 bits (whose own root and division take microseconds here).
__device__ __forceinline__ double root64(double x) {
  if (!(x > 1e-30 && x < 1e38)) return sqrt(x);
  const double r = (double)rsqrtf((float)x), y = x * r;
  return fma(fma(-y, y, x), 0.5 * r, y);
}
__device__ __forceinline__ double over64(double a, double x) {
  if (!(x > 1e-30 && x < 1e38)) return a / x;
  const double r = (double)(1.0f / (float)x), y = a * r;
  return fma(fma(-y, x, a), r, y);
}

// One CTA: the norm from its parts, the step count and the step's scalars,
// which come as they are for c = 1.
__global__ void __launch_bounds__(256) k_adamw_scalars(Scalars o, double max_norm, double ln_b1, double ln_b2, uint32_t seed,
                                                       const float* __restrict__ lr, int64_t* __restrict__ t,
                                                       const double* __restrict__ parts, int n_parts,
                                                       float* __restrict__ norm, Scalars* __restrict__ out) {
  launch_dependents();
  __shared__ double warp[8];
  const int lane = threadIdx.x & 31;
  const int64_t now = *t + 1;
  // 1 - b^t = -expm1(t ln b): as near as fp32 gets for every t
  const float away1 = -expm1f((float)((double)now * ln_b1)), away2 = -expm1f((float)((double)now * ln_b2));
  o.lr = *lr;
  o.step = o.lr / away1;
  o.root = 1.0f / sqrtf(away2);
  o.key = mix(mix((uint32_t)now) ^ seed);
  o.skip = 0;
  if (max_norm > 0.0) {
    wait_for_primary();  // (of the norm's kernel)
    double s = 0.0;
    for (int i = threadIdx.x; i < n_parts; i += 256) s += parts[i];
    s = warp_sum(s);
    if (lane == 0) warp[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    s = lane < 8 ? warp[lane] : 0.0;
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s = root64(s);
    o.skip = !(s <= 1.7e308);
    o.c = fmin(1.0, over64(max_norm, s + 1e-6));
    // Gradients far larger than max_norm: c's square would leave fp32's range, although c g is an ordinary number.  The part of
    // c below 2^-25 is a power of two of its own, which multiplies the gradients exactly.
    const int ex = (int)((__double_as_longlong(o.c) >> 52) & 0x7FF) - 1023;
    if (ex < -25) {
      const int k = max(ex + 25, -126);
      o.down = __uint_as_float((uint32_t)(k + 127) << 23);
      o.c *= __longlong_as_double((int64_t)(1023 - k) << 52);
    }
    const double a1 = o.a1 * o.c;
    o.a1h = (float)a1;
    o.a1l = (float)(a1 - (double)o.a1h);
    o.a2f = (float)(o.a2 * o.c * o.c);
    if (lane == 0 && norm) *norm = (float)s;
  }
  if (threadIdx.x != 0) return;
  if (!o.skip) *t = now;
  *out = o;
}

// ---------------------------------------------------------------------------
// 8-bit moments
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// The scale byte e + 127 for a block whose largest magnitude has these bits:
// 448 = 1.75 * 2^8.  `above`: the 64-bit value lies above 1.75 of its power of
// two (asked where the fp32 one is within NEAR of it).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, bool above) {
  if (amax >= 0x7F800000u) return 0xFFu;
  const int b = (int)(amax >> 23) - 8 + (above ? 1 : 0);
  return b > 0 ? (uint32_t)b : 0u;
}

// The code (no sign) of a = |x| 2^-e <= 448, up or down by r16, in 64 bits.
__device__ __noinline__ uint32_t code_exact(double a, uint32_t r16) {
  if (a <= 0.0) return 0u;
  const double lowest = 0.015625;  // 2^-6, the smallest normal value: below it codes lie as far apart as above
  const int ex = a < lowest ? -6 : (int)((__double_as_longlong(a) >> 52) & 0x7FF) - 1023;
  const double u = a * __longlong_as_double((int64_t)(3 - ex + 1023) << 52);  // in units of the codes' distance
  const double f = floor(u);
  const uint32_t k = (uint32_t)f + ((u - f) + (double)r16 * (1.0 / 65536.0) >= 1.0 ? 1u : 0u);
  return (uint32_t)(ex + 6) * 8u + k;  // (a normal value's k has its leading one: 8 to 16)
}

// Quantises one moment of a thread's PER elements; four neighbouring threads
// share a block.  x: the fp32 values, ex(i): the 64-bit value of element i.
// SHIFT: which half of the random bits.
//
// The fp32 pattern of x 2^-e, four places up (its sign and the exponent's high
// bits fall off the word) and with 8 added to the exponent (the two biases, 127
// and 7, differ by 24 modulo the 32 that are left), has the code of a normal
// value in its top byte and what lies above it in the 24 bits below; 16 random
// bits in the upper ones carry into it.  The elements whose low bits come within NEAR fp32 steps of a
// carry, and those below the normal codes, are found together and done again
// one by one.
template <bool LEAST, int SHIFT, class Exact>
__device__ __forceinline__ uint2 quantise(const float2* x, const uint32_t* bits, Exact ex, uint32_t& sbyte) {
  float peak = 0.0f;
#pragma unroll
  for (int i = 0; i < PER / 2; ++i) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(peak) : "f"(LEAST ? x[i].x : fabsf(x[i].x)));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(peak) : "f"(LEAST ? x[i].y : fabsf(x[i].y)));
  }
  uint32_t top = __float_as_uint(peak) & 0x7FFFFFFFu;
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  bool above = (top & 0x7FFFFFu) > 0x600000u;
  const bool near = (top & 0x7FFFFFu) - (0x600000u - NEAR) <= 2u * NEAR && top < 0x7F800000u;
  auto at = [&](int i) { return i & 1 ? x[i >> 1].y : x[i >> 1].x; };
  if (__any_sync(0xFFFFFFFFu, near)) {
    // the whole group of four looks at its elements near the limit in 64 bits
    const double limit = (double)__uint_as_float((top & 0x7F800000u) | 0x600000u);
    bool over = false;
    if (near) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (abs_bits(at(i)) + 2 * NEAR >= top) over |= fabs(ex(i)) > limit;
    }
    const uint32_t votes = __ballot_sync(0xFFFFFFFFu, over) >> (threadIdx.x & 28);
    if (near) above = (votes & 15u) != 0;
  }
  sbyte = scale_byte(top, above);
  if (sbyte == 0xFFu) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float inv = mx_inv_scale(sbyte);
  constexpr float LOWEST = 0.015625f;  // 2^-6, the smallest normal code's value
  uint32_t y[PER], close = 0xFFFFFFFFu;
  float least = 1e30f;
#pragma unroll
  for (int i = 0; i < PER / 2; ++i) {
    const float2 a = __fmul2_rn(x[i], both(inv));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float f = k ? a.y : a.x;
      const uint32_t v = __float_as_uint(f) * 16u + __byte_perm(bits[2 * i + k], 0x40u, SHIFT ? 0x4325 : 0x4105);
      least = fminf(least, fabsf(f));
      close = min(close, v * 256u + 16u * NEAR * 256u);
      y[2 * i + k] = LEAST ? v : v | (__float_as_uint(f) & 0x80000000u);
    }
  }
  uint2 w = make_uint2(__byte_perm(__byte_perm(y[0], y[1], 0x73), __byte_perm(y[2], y[3], 0x73), 0x5410),
                       __byte_perm(__byte_perm(y[4], y[5], 0x73), __byte_perm(y[6], y[7], 0x73), 0x5410));
  if (least < LOWEST || close < 32u * NEAR * 256u) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t low = y[i] & 0xFFFFFFu;
      if (fabsf(at(i) * inv) >= LOWEST && ((low + 16u * NEAR) & 0xFFFFFFu) >= 32u * NEAR) continue;
      uint32_t code = 0;
      if (at(i) != 0.0f) {
        code = code_exact(fabs(ex(i)) * (double)inv, SHIFT ? bits[i] >> 16 : bits[i] & 0xFFFFu);
        if (LEAST && code == 0) code = 1;
        if (!LEAST) code |= (__float_as_uint(at(i)) >> 24) & 0x80u;
      }
      uint32_t& word = i < 4 ? w.x : w.y;
      word = (word & ~(0xFFu << (8 * (i & 3)))) | code << (8 * (i & 3));
    }
  }
  return w;
}

// m or sqrt(v) of PER elements from their codes; the block's scale is one of
// the 32 elements from at on.
__device__ __forceinline__ void decode8(uint2 w, uint32_t sbyte, float2* x) {
  // (0 stands for 2^-127, a subnormal; 255 only beside codes that are NaN themselves)
  const float f = __uint_as_float(max(sbyte << 23, 0x00400000u));
  const float2 f2 = make_float2(f, f);
  x[0] = __fmul2_rn(e4m3x2_value(w.x & 0xFFFFu), f2);
  x[1] = __fmul2_rn(e4m3x2_value(w.x >> 16), f2);
  x[2] = __fmul2_rn(e4m3x2_value(w.y & 0xFFFFu), f2);
  x[3] = __fmul2_rn(e4m3x2_value(w.y >> 16), f2);
}

__device__ __forceinline__ float sqrt_hw(float x) {  // (v below 2^-126, a subnormal, as 0)
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_hw(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// w <- w - (lr wd w + step m / (sqrt(v) root + eps)): the quotient and the
// root by the hardware's approximations, good to two fp32 steps; what is taken
// off is small beside w, so that w is rounded once.
__device__ __forceinline__ float2 updated(const Short& s, float decay, float2 w, float2 m, float2 root_v) {
  const float2 den = __ffma2_rn(root_v, both(s.root), both(s.eps));
  const float2 q = __fmul2_rn(m, make_float2(rcp_hw(den.x), rcp_hw(den.y)));
  const float2 d = __ffma2_rn(q, both(s.step), __fmul2_rn(w, both(decay)));
  return __ffma2_rn(d, both(-1.0f), w);
}

// The moments in 64 bits (calls, so that the rare path costs the usual one no registers).
__device__ __noinline__ double exact_m(float m, float g, const Scalars* s) {
  return __dadd_rn(__dmul_rn((double)m, s->b1), __dmul_rn(__dmul_rn((double)g, s->c), s->a1));
}
__device__ __noinline__ double exact_root(float root, float g, const Scalars* s) {
  const double gc = __dmul_rn((double)g, s->c), r = (double)root;
  return sqrt(__dadd_rn(__dmul_rn(r * r, s->b2), __dmul_rn(__dmul_rn(gc, gc), s->a2)));
}

template <bool STATE8, bool W16, class G>
__device__ __forceinline__ void step8(const Short& s, const Scalars* all, const moe_adamw_tensor_t& t, const G* grad,
                                      int64_t at, int64_t n, uint32_t key) {
  float2 g[PER / 2], w[PER / 2], m[PER / 2], v[PER / 2];
  // a thread past the tensor's end works on zeros: its neighbours' block needs it in the exchange
  const bool live = n > 0;
  // whole vectors everywhere: one test for all of a thread's loads and stores
  float* wide = W16 ? t.master : static_cast<float*>(t.w);
  const bool whole = n >= PER && on(wide + at, 32) && on(grad + at, sizeof(G) * PER) && (!W16 || on(static_cast<__nv_bfloat16*>(t.w) + at, 16)) &&
                     (STATE8 || (on(static_cast<const float*>(t.m) + at, 32) && on(static_cast<const float*>(t.v) + at, 32)));
#pragma unroll
  for (int i = 0; i < PER / 2; ++i) g[i] = w[i] = m[i] = v[i] = both(0.0f);
  if (live) {
    // (the gradient last: its bf16 values are taken apart as they come, when all other loads are under way)
    if (STATE8) {
      const uint2 qm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + at);
      const uint2 qv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + at);
      const uint32_t sm = t.m_scale[at / BLOCK], sv = t.v_scale[at / BLOCK];
      load8(wide + at, n, whole, &w[0].x);
      load8(grad + at, n, whole, &g[0].x);
      decode8(qm, sm, m);
      decode8(qv, sv, v);
    } else {
      load8(wide + at, n, whole, &w[0].x);
      load8(static_cast<const float*>(t.m) + at, n, whole, &m[0].x);
      load8(static_cast<const float*>(t.v) + at, n, whole, &v[0].x);
      load8(grad + at, n, whole, &g[0].x);
    }
  }
  if (s.down != 1.0f) {
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) g[i] = __fmul2_rn(g[i], both(s.down));
  }
  const float decay = s.lr * t.weight_decay;
  float2 om[PER / 2], ov[PER / 2];
#pragma unroll
  for (int i = 0; i < PER / 2; ++i) {
    if (STATE8) {
      // b1 m + a1 g: the first product's error, and the low parts of both factors
      const float2 p = __fmul2_rn(m[i], both(s.b1h)), minus = __fmul2_rn(m[i], both(-s.b1h));
      const float2 rest = __ffma2_rn(g[i], both(s.a1l), __ffma2_rn(m[i], both(s.b1l), __ffma2_rn(m[i], both(s.b1h), minus)));
      om[i] = __fadd2_rn(__ffma2_rn(g[i], both(s.a1h), p), rest);
      const float2 q = __ffma2_rn(__fmul2_rn(v[i], v[i]), both(s.b2f), __fmul2_rn(__fmul2_rn(g[i], g[i]), both(s.a2f)));
      ov[i] = make_float2(sqrt_hw(q.x), sqrt_hw(q.y));
      w[i] = updated(s, decay, w[i], om[i], ov[i]);
    } else {
      om[i] = __ffma2_rn(m[i], both(s.b1h), __fmul2_rn(g[i], both(s.a1h)));
      ov[i] = __ffma2_rn(v[i], both(s.b2f), __fmul2_rn(__fmul2_rn(g[i], g[i]), both(s.a2f)));
      w[i] = updated(s, decay, w[i], om[i], make_float2(sqrt_hw(ov[i].x), sqrt_hw(ov[i].y)));
    }
  }
  if (live) {
    store8(wide + at, n, whole, &w[0].x);
    if (W16) store8(static_cast<__nv_bfloat16*>(t.w) + at, n, whole, &w[0].x);
  }
  if (STATE8) {
    uint32_t bits[PER];
    const uint32_t k = mix(key + (uint32_t)(at >> 32)) + (uint32_t)at;
#pragma unroll
    for (int i = 0; i < PER; ++i) bits[i] = mix(k + i);
    uint32_t sm, sv;
    const auto of = [](const float2* x, int i) { return i & 1 ? x[i >> 1].y : x[i >> 1].x; };
    const uint2 qm = quantise<false, 1>(om, bits, [&](int i) { return exact_m(of(m, i), of(g, i), all); }, sm);
    const uint2 qv = quantise<true, 0>(ov, bits, [&](int i) { return exact_root(of(v, i), of(g, i), all); }, sv);
    if (live) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + at) = qm;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + at) = qv;
      if ((threadIdx.x & 3) == 0) {
        t.m_scale[at / BLOCK] = (uint8_t)sm;
        t.v_scale[at / BLOCK] = (uint8_t)sv;
      }
    }
  } else if (live) {
    store8(static_cast<float*>(t.m) + at, n, whole, &om[0].x);
    store8(static_cast<float*>(t.v) + at, n, whole, &ov[0].x);
  }
}

template <int N, bool STATE8>
__global__ void __launch_bounds__(THREADS, STATE8 ? 3 : 4) k_adamw_step(const __grid_constant__ Grads<N> grads,
                                                        const moe_adamw_tensor_t* __restrict__ tensors,
                                                        const Entry* __restrict__ table, uint32_t chunks, int first,
                                                        const Scalars* __restrict__ scalars) {
  wait_for_primary();
  const Short s = *scalars;
  if (s.skip) return;
  // backwards: the norm's kernel has read the last gradients last, and finds them in L2
  Entry next = table[chunks - 1 - blockIdx.x];
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const Entry e = next;
    if (i + gridDim.x < chunks) next = table[chunks - 1 - i - gridDim.x];
    const moe_adamw_tensor_t t = tensors[e.tensor];
    const void* g = grads.p[e.tensor - first];
    const int64_t at = (int64_t)e.chunk * CHUNK + threadIdx.x * PER, n = t.n - at;
    const uint32_t key = mix(s.key + e.tensor);
    if (t.w_bf16) {
      if (t.grad_bf16)
        step8<STATE8, true>(s, scalars, t, static_cast<const __nv_bfloat16*>(g), at, n, key);
      else
        step8<STATE8, true>(s, scalars, t, static_cast<const float*>(g), at, n, key);
    } else {
      if (t.grad_bf16)
        step8<STATE8, false>(s, scalars, t, static_cast<const __nv_bfloat16*>(g), at, n, key);
      else
        step8<STATE8, false>(s, scalars, t, static_cast<const float*>(g), at, n, key);
    }
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
size_t chunks_of(const moe_adamw_tensor_t& t) { return (size_t)((t.n + CHUNK - 1) / CHUNK); }

bool valid(const moe_adamw_tensor_t* t, int n, int state8) {
  if (n < 0 || n > (1 << 20) || (n > 0 && !t)) return false;
  size_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].n < 0 || t[i].n > ((int64_t)1 << 42)) return false;
    if (t[i].n == 0) continue;
    chunks += chunks_of(t[i]);
    if (!t[i].w || !t[i].m || !t[i].v || (t[i].w_bf16 && !t[i].master)) return false;
    const auto off = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; };
    if (off(t[i].w, t[i].w_bf16 ? 2 : 4) || (t[i].w_bf16 && off(t[i].master, 4))) return false;
    if (state8 ? off(t[i].m, 8) || off(t[i].v, 8) || !t[i].m_scale || !t[i].v_scale : off(t[i].m, 4) || off(t[i].v, 4))
      return false;
    if (!(t[i].weight_decay >= 0.0f)) return false;
  }
  return chunks < ((size_t)1 << 31);
}

// Tensors [first, first + count) as one launch each of the norm's part
// (parts != null) or of the step.
template <int N>
moe_status_t launch_group(const moe_adamw_tensor_t* dev, const Entry* table, uint32_t chunks, const void* const* grads,
                          int first, int count, int state8, const Scalars* sc, double* parts, int n_parts,
                          bool behind_scalars, cudaStream_t stream) {
  Grads<N> g;
  for (int i = 0; i < count; ++i) g.p[i] = grads[first + i];
  if (parts) return launch_kernel(k_adamw_norm<N>, n_parts, 0, THREADS, 0, false, stream, g, dev, table, chunks, first, parts);
  const auto k = state8 ? k_adamw_step<N, true> : k_adamw_step<N, false>;
  const int per_sm = max_active_blocks((const void*)k, THREADS, 0), sms = sm_count();
  if (per_sm < 1 || sms < 1) return MOE_ERR_CUDA;
  const uint32_t most = per_sm * sms;
  return launch_kernel(k, chunks < most ? chunks : most, 0, THREADS, 0, behind_scalars, stream, g, dev, table, chunks, first, sc);
}

int parts_of(uint32_t chunks) {
  const int n = sm_count() * 8;
  const int most = n < MAX_PARTS ? n : MAX_PARTS;
  return chunks < (uint32_t)most ? (int)chunks : most;
}

int groups_of(int n) { return (n + MANY - 1) / MANY; }

}  // namespace adamw
}  // namespace moeglu

using namespace moeglu;
using namespace moeglu::adamw;

extern "C" size_t moe_adamw_plan_size(const moe_adamw_tensor_t* tensors, int n) {
  if (n < 0 || (n > 0 && !tensors)) return 0;
  size_t c = 0;
  for (int i = 0; i < n; ++i) c += tensors[i].n > 0 ? chunks_of(tensors[i]) : 0;
  return n * sizeof(moe_adamw_tensor_t) + c * sizeof(Entry);
}

extern "C" moe_status_t moe_adamw_plan(const moe_adamw_tensor_t* tensors, int n, int state, void* host_plan, size_t bytes) {
  if ((state != MOE_MOMENTS_F32 && state != MOE_MOMENTS_MXFP8) || !valid(tensors, n, state)) return MOE_ERR_ARG;
  if (bytes < moe_adamw_plan_size(tensors, n) || (n > 0 && !host_plan)) return MOE_ERR_ARG;
  auto* t = static_cast<moe_adamw_tensor_t*>(host_plan);
  auto* e = reinterpret_cast<Entry*>(t + n);
  for (int i = 0; i < n; ++i) {
    t[i] = tensors[i];
    const size_t c = chunks_of(tensors[i]);
    for (size_t j = 0; j < c; ++j) *e++ = {(uint32_t)i, (uint32_t)j};
  }
  return MOE_OK;
}

extern "C" size_t moe_adamw_workspace_size(int n) {
  return n < 0 ? 0 : PARTS_AT + (size_t)MAX_PARTS * sizeof(double) * (groups_of(n) < 1 ? 1 : groups_of(n));
}

extern "C" moe_status_t moe_adamw_step(const moe_adamw_tensor_t* tensors, const void* const* grads, int n, const void* plan,
                                       const moe_adamw_params_t* p, const float* lr, int64_t* t, float* norm, void* ws,
                                       size_t ws_bytes, moe_stream_t stream_) {
  if (!p || !lr || !t || !ws || (reinterpret_cast<uintptr_t>(ws) & 15u) || ws_bytes < moe_adamw_workspace_size(n))
    return MOE_ERR_ARG;
  if (!(p->beta1 >= 0.0 && p->beta1 < 1.0 && p->beta2 >= 0.0 && p->beta2 < 1.0 && p->eps >= 0.0 && p->max_norm >= 0.0) ||
      (p->state != MOE_MOMENTS_F32 && p->state != MOE_MOMENTS_MXFP8) || !valid(tensors, n, p->state))
    return MOE_ERR_ARG;
  if (n > 0 && (!grads || !plan || (reinterpret_cast<uintptr_t>(plan) & 7u))) return MOE_ERR_ARG;
  for (int i = 0; i < n; ++i)
    if (tensors[i].n > 0 && (!grads[i] || (reinterpret_cast<uintptr_t>(grads[i]) & (tensors[i].grad_bf16 ? 1u : 3u))))
      return MOE_ERR_ARG;
  static_assert(sizeof(Scalars) <= PARTS_AT, "the scalars' part of the workspace");
  const cudaStream_t stream = as_stream(stream_);
  auto* sc = static_cast<Scalars*>(ws);
  auto* parts = reinterpret_cast<double*>(static_cast<char*>(ws) + PARTS_AT);
  const auto* dev = static_cast<const moe_adamw_tensor_t*>(plan);
  const auto* table = reinterpret_cast<const Entry*>(dev + n);
  int n_parts = 0;
  bool pass0 = false;  // the norm's last launch is right in front of the scalars'
  for (int pass = p->max_norm > 0.0 ? 0 : 1; pass < 2; ++pass) {
    if (pass == 1) {
      Scalars c1 = {};
      c1.b1 = p->beta1;
      c1.a1 = 1.0 - p->beta1;
      c1.b2 = p->beta2;
      c1.a2 = 1.0 - p->beta2;
      c1.c = 1.0;
      c1.down = 1.0f;
      c1.b1h = (float)c1.b1;
      c1.b1l = (float)(c1.b1 - (double)c1.b1h);
      c1.a1h = (float)c1.a1;
      c1.a1l = (float)(c1.a1 - (double)c1.a1h);
      c1.b2f = (float)c1.b2;
      c1.a2f = (float)c1.a2;
      c1.eps = (float)p->eps;
      const auto ln = [](double b) { return b > 0.0 ? std::log(b) : -1e9; };  // (of 0: a power of 0)
      if (const moe_status_t e = launch_kernel(k_adamw_scalars, 1, 0, p->max_norm > 0.0 ? 256 : 32, 0, pass0, stream, c1,
                                               p->max_norm, ln(p->beta1), ln(p->beta2), p->seed, lr, t, parts, n_parts, norm, sc))
        return e;
    }
    const Entry* at = table;
    bool behind = true;  // only the launch right behind the scalars' may start before it ends
    for (int first = 0; first < n; first += MANY) {
      const int count = n - first < MANY ? n - first : MANY;
      size_t c = 0;
      for (int i = 0; i < count; ++i) c += chunks_of(tensors[first + i]);
      if (c == 0) continue;
      double* to = pass == 0 ? parts + n_parts : nullptr;
      const int np = parts_of((uint32_t)c);
      if (np < 1) return MOE_ERR_CUDA;
      const moe_status_t e =
          count <= FEW
              ? launch_group<FEW>(dev, at, (uint32_t)c, grads, first, count, p->state, sc, to, np, behind, stream)
          : count <= SOME
              ? launch_group<SOME>(dev, at, (uint32_t)c, grads, first, count, p->state, sc, to, np, behind, stream)
              : launch_group<MANY>(dev, at, (uint32_t)c, grads, first, count, p->state, sc, to, np, behind, stream);
      if (e) return e;
      behind = false;
      if (pass == 0) n_parts += np, pass0 = true;
      at += c;
    }
  }
  return MOE_OK;
}
