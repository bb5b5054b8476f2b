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
// addresses (they differ from step to step) come as a kernel parameter.
#include "common.cuh"
#include "host_common.h"

namespace moeglu {
namespace adamw {

constexpr int THREADS = 256, PER = 8, CHUNK = 2048;  // elements per thread at a time, per chunk
constexpr int FEW = 64, MANY = 4000;                 // gradient addresses in a launch's parameters (32,764 bytes at most)
constexpr int BLOCK = 32;                            // elements per scale
constexpr int MAX_PARTS = 1024;                      // CTAs of the norm's kernel
constexpr int NEAR = 8;  // fp32 steps around a turning point inside which 64 bits decide

struct Entry {
  uint32_t tensor, chunk;
};
template <int N>
struct Grads {
  const void* p[N];
};

// What a step's scalars are, written once per step.
struct Scalars {
  double b1, a1, b2, a2, c;            // a = 1 - b
  float b1h, b1l, a1h, a1l, b2f, a2f;  // a1 and a2 with c and c^2
  float step, root, lr, eps;           // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t key;
  int32_t skip;  // the gradients' norm is not finite
};
// the workspace: the scalars, then the norm's partial sums
constexpr size_t PARTS_AT = 256;

struct Params {
  double b1, b2, eps, max_norm;
  uint32_t seed;
};

__device__ __forceinline__ uint32_t mix(uint32_t x) {  // a 32-bit hash: two multiplications
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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

// n: elements left from p on (at least 1)
__device__ __forceinline__ void load8(const float* p, int64_t n, float* v) {
  if (n >= PER && on(p, 32)) {
    ld_f32x8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int64_t n, float* v) {
  if (n >= PER && on(p, 16)) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ void store8(float* p, int64_t n, const float* v) {
  if (n >= PER && on(p, 32)) {
    st_f32x8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int64_t n, const float* v) {
  if (n >= PER && on(p, 16)) {
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

// parts[CTA] = sum of squares of its chunks.  Eight squares are added in fp32
// (of bf16 values they are exact), these sums with their rounding errors.
template <int N>
__global__ void __launch_bounds__(THREADS) k_adamw_norm(const __grid_constant__ Grads<N> grads,
                                                        const moe_adamw_tensor_t* __restrict__ tensors,
                                                        const Entry* __restrict__ table, uint32_t chunks, int first,
                                                        double* __restrict__ parts) {
  float hi = 0.0f, lo = 0.0f;
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const Entry e = table[i];
    const moe_adamw_tensor_t& t = tensors[e.tensor];
    const int64_t at = (int64_t)e.chunk * CHUNK + threadIdx.x * PER, n = t.n - at;
    if (n <= 0) continue;
    float g[PER];
    const void* p = grads.p[e.tensor - first];
    if (t.grad_bf16)
      load8(static_cast<const __nv_bfloat16*>(p) + at, n, g);
    else
      load8(static_cast<const float*>(p) + at, n, g);
    float q = g[0] * g[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) q = fmaf(g[j], g[j], q);
    const float s = hi + q, bb = s - hi;
    lo += (hi - (s - bb)) + (q - bb);
    hi = s;
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

// One CTA: the norm from its parts, the step count and the step's scalars.
__global__ void __launch_bounds__(32) k_adamw_scalars(Params p, const float* __restrict__ lr, int64_t* __restrict__ t,
                                                      const double* __restrict__ parts, int n_parts,
                                                      float* __restrict__ norm, Scalars* __restrict__ out) {
  launch_dependents();
  double s = 0.0;
  for (int i = threadIdx.x; i < n_parts; i += 32) s += parts[i];
  s = sqrt(warp_sum(s));
  if (threadIdx.x != 0) return;
  double c = 1.0;
  bool skip = false;
  if (p.max_norm > 0.0) {
    skip = !(s <= 1.7e308);
    c = fmin(1.0, p.max_norm / (s + 1e-6));
    if (norm) *norm = (float)s;
  }
  if (!skip) *t += 1;
  const int64_t now = *t;
  Scalars o;
  o.b1 = p.b1;
  o.a1 = 1.0 - p.b1;
  o.b2 = p.b2;
  o.a2 = 1.0 - p.b2;
  o.c = c;
  const double a1 = o.a1 * c;
  o.b1h = (float)p.b1;
  o.b1l = (float)(p.b1 - (double)o.b1h);
  o.a1h = (float)a1;
  o.a1l = (float)(a1 - (double)o.a1h);
  o.b2f = (float)p.b2;
  o.a2f = (float)(o.a2 * c * c);
  o.lr = *lr;
  o.step = (float)((double)o.lr / (1.0 - pow(p.b1, (double)now)));
  o.root = (float)(1.0 / sqrt(1.0 - pow(p.b2, (double)now)));
  o.eps = (float)p.eps;
  o.key = mix(mix((uint32_t)now) ^ p.seed);
  o.skip = skip;
  *out = o;
}

// ---------------------------------------------------------------------------
// 8-bit moments
// ---------------------------------------------------------------------------
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

// The code (no sign) of a >= 0 within a few fp32 steps; false where 64 bits
// have to decide (or the value is below the normal codes).
__device__ __forceinline__ bool code_fast(float a, uint32_t r16, uint32_t& code) {
  const uint32_t b = __float_as_uint(a), x = b + (r16 << 4);
  code = (x >> 20) - (120u << 3);
  return b >= 0x3C800000u && ((x + NEAR) & 0xFFFFFu) >= 2u * NEAR;
}

// Quantises one moment of a thread's PER elements; four neighbouring threads
// share a block.  x: the fp32 values, ex(i): the 64-bit value of element i.
// SHIFT: which half of the random bits.
template <bool LEAST, int SHIFT, class Exact>
__device__ __forceinline__ uint2 quantise(const float* x, const uint32_t* bits, Exact ex, uint32_t& sbyte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = max(top, abs_bits(x[i]));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  bool above = (top & 0x7FFFFFu) > 0x600000u;
  const bool near = (top & 0x7FFFFFu) - (0x600000u - NEAR) <= 2u * NEAR && top < 0x7F800000u;
  if (__any_sync(0xFFFFFFFFu, near)) {
    // the whole group of four looks at its elements near the limit in 64 bits
    const double limit = (double)__uint_as_float((top & 0x7F800000u) | 0x600000u);
    bool over = false;
    if (near) {
      for (int i = 0; i < PER; ++i)
        if (abs_bits(x[i]) + 2 * NEAR >= top) over |= fabs(ex(i)) > limit;
    }
    const uint32_t votes = __ballot_sync(0xFFFFFFFFu, over) >> (threadIdx.x & 28);
    if (near) above = (votes & 15u) != 0;
  }
  sbyte = scale_byte(top, above);
  if (sbyte == 0xFFu) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float inv = mx_inv_scale(sbyte);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t r16 = SHIFT ? bits[i] >> 16 : bits[i] & 0xFFFFu;
    uint32_t code;
    if (!code_fast(fabsf(x[i]) * inv, r16, code)) {
      if (x[i] == 0.0f) {
        code = 0;
      } else {
        code = code_exact(fabs(ex(i)) * (double)inv, r16);
        if (LEAST && code == 0) code = 1;
      }
    }
    if (!LEAST) code |= (__float_as_uint(x[i]) >> 24) & 0x80u;
    w[i >> 2] |= code << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

// m and sqrt(v) of PER elements from their codes; the block's scale is one of
// the 32 elements from at on.
__device__ __forceinline__ void decode8(const uint8_t* q, const uint8_t* s, int64_t at, float* x) {
  const uint2 w = *reinterpret_cast<const uint2*>(q + at);
  const float f = e8m0_value(s[at / BLOCK]);
  const uint32_t h[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = e4m3x2_value(h[i]);
    x[2 * i] = p.x * f;
    x[2 * i + 1] = p.y * f;
  }
}

__device__ __forceinline__ float sqrt_hw(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// w <- w - (lr wd w + step m / (sqrt(v) root + eps)): the quotient and the
// root by the hardware's approximations, good to two fp32 steps; what is taken
// off is small beside w, so that w is rounded once.
__device__ __forceinline__ float updated(const Scalars& s, float decay, float w, float m, float root_v) {
  return w - fmaf(s.step, __fdividef(m, fmaf(root_v, s.root, s.eps)), w * decay);
}

template <bool STATE8, bool W16, class G>
__device__ __forceinline__ void step8(const Scalars& s, const moe_adamw_tensor_t& t, const G* grad, int64_t at, int64_t n,
                                      uint32_t key) {
  float g[PER], w[PER], m[PER], v[PER];
  // a thread past the tensor's end works on zeros: its neighbours' block needs it in the exchange
  const bool live = n > 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) g[i] = w[i] = m[i] = v[i] = 0.0f;
  float* wide = W16 ? t.master : static_cast<float*>(t.w);
  if (live) {
    load8(grad + at, n, g);
    load8(wide + at, n, w);
    if (STATE8) {
      decode8(static_cast<const uint8_t*>(t.m), t.m_scale, at, m);
      decode8(static_cast<const uint8_t*>(t.v), t.v_scale, at, v);
    } else {
      load8(static_cast<const float*>(t.m) + at, n, m);
      load8(static_cast<const float*>(t.v) + at, n, v);
    }
  }
  const float decay = s.lr * t.weight_decay;
  float om[PER], ov[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (STATE8) {
      // b1 m + a1 g: the first product's error, and the low parts of both factors
      const float p = s.b1h * m[i];
      const float rest = fmaf(s.a1l, g[i], fmaf(s.b1l, m[i], fmaf(s.b1h, m[i], -p)));
      om[i] = fmaf(s.a1h, g[i], p) + rest;
      ov[i] = sqrt_hw(fmaf(s.b2f, v[i] * v[i], s.a2f * (g[i] * g[i])));
      w[i] = updated(s, decay, w[i], om[i], ov[i]);
    } else {
      om[i] = fmaf(s.b1h, m[i], s.a1h * g[i]);
      ov[i] = fmaf(s.b2f, v[i], s.a2f * (g[i] * g[i]));
      w[i] = updated(s, decay, w[i], om[i], sqrt_hw(ov[i]));
    }
  }
  if (live) {
    store8(wide + at, n, w);
    if (W16) store8(static_cast<__nv_bfloat16*>(t.w) + at, n, w);
  }
  if (STATE8) {
    uint32_t bits[PER];
    const uint32_t k = mix(key + (uint32_t)(at >> 32));
#pragma unroll
    for (int i = 0; i < PER; ++i) bits[i] = mix(k + (uint32_t)at + i);
    uint32_t sm, sv;
    const uint2 qm = quantise<false, 1>(
        om, bits,
        [&](int i) { return __dadd_rn(__dmul_rn((double)m[i], s.b1), __dmul_rn(__dmul_rn((double)g[i], s.c), s.a1)); }, sm);
    const uint2 qv = quantise<true, 0>(
        ov, bits,
        [&](int i) {
          const double gc = __dmul_rn((double)g[i], s.c), r = (double)v[i];
          return sqrt(__dadd_rn(__dmul_rn(r * r, s.b2), __dmul_rn(__dmul_rn(gc, gc), s.a2)));
        },
        sv);
    if (live) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + at) = qm;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + at) = qv;
      if ((threadIdx.x & 3) == 0) {
        t.m_scale[at / BLOCK] = (uint8_t)sm;
        t.v_scale[at / BLOCK] = (uint8_t)sv;
      }
    }
  } else if (live) {
    store8(static_cast<float*>(t.m) + at, n, om);
    store8(static_cast<float*>(t.v) + at, n, ov);
  }
}

template <int N, bool STATE8>
__global__ void __launch_bounds__(THREADS) k_adamw_step(const __grid_constant__ Grads<N> grads,
                                                        const moe_adamw_tensor_t* __restrict__ tensors,
                                                        const Entry* __restrict__ table, uint32_t chunks, int first,
                                                        const Scalars* __restrict__ scalars) {
  wait_for_primary();
  const Scalars s = *scalars;
  if (s.skip) return;
  // backwards: the norm's kernel has read the last gradients last, and finds them in L2
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const Entry e = table[chunks - 1 - i];
    const moe_adamw_tensor_t t = tensors[e.tensor];
    const void* g = grads.p[e.tensor - first];
    const int64_t at = (int64_t)e.chunk * CHUNK + threadIdx.x * PER, n = t.n - at;
    const uint32_t key = mix(s.key + e.tensor);
    if (t.w_bf16) {
      if (t.grad_bf16)
        step8<STATE8, true>(s, t, static_cast<const __nv_bfloat16*>(g), at, n, key);
      else
        step8<STATE8, true>(s, t, static_cast<const float*>(g), at, n, key);
    } else {
      if (t.grad_bf16)
        step8<STATE8, false>(s, t, static_cast<const __nv_bfloat16*>(g), at, n, key);
      else
        step8<STATE8, false>(s, t, static_cast<const float*>(g), at, n, key);
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

template <int N, bool STATE8>
moe_status_t launch_step(const Grads<N>& g, const moe_adamw_tensor_t* dev, const Entry* table, uint32_t chunks, int first,
                         const Scalars* sc, bool behind_scalars, cudaStream_t stream) {
  auto* k = k_adamw_step<N, STATE8>;
  const int per_sm = max_active_blocks((const void*)k, THREADS, 0), sms = sm_count();
  if (per_sm < 1 || sms < 1) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(chunks < (uint32_t)(per_sm * sms) ? chunks : (uint32_t)(per_sm * sms));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = behind_scalars ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, k, g, dev, table, chunks, first, sc) != cudaSuccess) return MOE_ERR_CUDA;
  count_launch();
  return launch_status();
}

// Tensors [first, first + count) as one launch each of the norm's part
// (parts != null) or of the step.
template <int N>
moe_status_t launch_group(const moe_adamw_tensor_t* dev, const Entry* table, uint32_t chunks, const void* const* grads,
                          int first, int count, int state8, const Scalars* sc, double* parts, int n_parts,
                          bool behind_scalars, cudaStream_t stream) {
  Grads<N> g;
  for (int i = 0; i < count; ++i) g.p[i] = grads[first + i];
  if (parts) {
    k_adamw_norm<N><<<n_parts, THREADS, 0, stream>>>(g, dev, table, chunks, first, parts);
    count_launch();
    return launch_status();
  }
  return state8 ? launch_step<N, true>(g, dev, table, chunks, first, sc, behind_scalars, stream)
                : launch_step<N, false>(g, dev, table, chunks, first, sc, behind_scalars, stream);
}

int parts_of(uint32_t chunks) {
  const int n = sm_count() * 6;
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
  for (int pass = p->max_norm > 0.0 ? 0 : 1; pass < 2; ++pass) {
    if (pass == 1) {
      const Params q = {p->beta1, p->beta2, p->eps, p->max_norm, p->seed};
      k_adamw_scalars<<<1, 32, 0, stream>>>(q, lr, t, parts, n_parts, norm, sc);
      count_launch();
      if (const moe_status_t e = launch_status()) return e;
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
              : launch_group<MANY>(dev, at, (uint32_t)c, grads, first, count, p->state, sc, to, np, behind, stream);
      if (e) return e;
      behind = false;
      if (pass == 0) n_parts += np;
      at += c;
    }
  }
  return MOE_OK;
}
