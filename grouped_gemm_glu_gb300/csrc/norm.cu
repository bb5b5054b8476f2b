// Residual addition and RMS norm in front of the expert MLP, forward and
// backward, and the read-back of MXFP8 rows.
//
//   h = bf16(x + residual)            (the residual stream; h = x without one)
//   r = 1 / sqrt(mean_i h_i^2 + eps)
//   y_i = (h_i r) gamma_i             -> bf16 and / or MXFP8 rows (one E8M0
//                                        scale per 32 columns)
//   backward, t_i = dy_i gamma_i:
//   dx_i = r (t_i - h_i r^2 mean_j(t_j h_j)) + dres_i
//   dgamma_i = sum over tokens of dy_i h_i r
//
// All arithmetic between the bf16 loads and the stores is fp32; h is rounded
// to bf16 once, and the norm uses the rounded value, so that the backward,
// which reads h back, sees the number the forward used.  MXFP8 is quantised
// from the fp32 y, as in the fused epilogues.
//
// Memory bound: the forward must read x and residual and write h and y (8
// bytes per element, 1.03 more for MXFP8), the backward reads dy, h and dres
// and writes dx (8 bytes per element).  A row is held in registers by its
// threads (packed bf16) between the reduction and the output, so every byte
// crosses HBM once.
//
// One CTA per SM walks the rows in G groups of wpr warps, one row per group
// at a time.  A reduction and its barrier stand between a row's loads and its
// stores, so loads issued row by row leave HBM idle; each thread therefore
// copies the columns it owns of the next rows into its own slots of shared
// memory (cp.async, `stages` rows ahead: about 170 KB in flight per SM).  The
// slots are private to the thread: no barrier guards them.  A call of few
// rows (at most FEW_ROWS) takes one CTA per row instead, spread over as many
// warps as it has vectors for, because there one row's latency is the call's
// time.
//
// Measured: 8192 x 7168 with residual forward 89 us (bf16 and MXFP8 out; 5.9
// TB/s), backward 81 us and 6.4 for dgamma's last sum (5.4 TB/s together); one
// row of 2880 2.2 us.
#include "common.cuh"
#include "host_common.h"

namespace moeglu {
namespace norm {

constexpr int MAX_H = 16384;  // 16 warps x 4 vectors of 8 columns a lane
// threads per CTA: with more than one vector a thread's registers allow 16 warps
template <int V>
constexpr int max_threads() { return V == 1 ? 1024 : 512; }
constexpr int MAX_T = 1 << 30;  // row indexes stay in 32 bits a few grids past the end
// of a call of few rows, at most: 32 warps on each of the 152 SMs (a constant, because the workspace's size is host
// arithmetic that has to give the launch's split without asking a device)
constexpr int FEW_ROWS = 512, FEW_WARPS = 152 * 32;
constexpr int RING_BYTES = 200 * 1024;  // of the 227 KB a CTA may have

// Eight bf16 values as four float pairs (the packed fp32 instructions of
// sm_100 work on pairs).
__device__ __forceinline__ void unpack8(const uint4 q, float2* v) {
  v[0] = make_float2(bf16_lo(q.x), bf16_hi(q.x));
  v[1] = make_float2(bf16_lo(q.y), bf16_hi(q.y));
  v[2] = make_float2(bf16_lo(q.z), bf16_hi(q.z));
  v[3] = make_float2(bf16_lo(q.w), bf16_hi(q.w));
}
__device__ __forceinline__ uint4 pack8(const float2* v) {
  return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                    pack_bf16x2(v[3].x, v[3].y));
}
__device__ __forceinline__ float2 pair_of(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
// The larger magnitude, NaN if either is.
__device__ __forceinline__ float max_abs(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `ahead` (0..3) of the thread's newest groups are in flight.
__device__ __forceinline__ void cp_async_wait(int ahead) {
  if (ahead == 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (ahead == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (ahead == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// A float and the rounding error of the sum it came from.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {  // a + b = hi + lo exactly (Knuth)
  const float s = a + b, bb = s - a;
  return {s, (a - (s - bb)) + (b - bb)};
}

// Adds the squares of v to the sums hi + lo of the two halves, keeping the
// rounding errors (a square of a bf16 value is exact in fp32).
__device__ __forceinline__ void add_squares(float2 v, float2& hi, float2& lo) {
  const float2 q = __fmul2_rn(v, v);
  const float2 s = __fadd2_rn(hi, q), bb = __fadd2_rn(s, neg2(hi));
  lo = __fadd2_rn(lo, __fadd2_rn(__fadd2_rn(hi, neg2(__fadd2_rn(s, neg2(bb)))), __fadd2_rn(q, neg2(bb))));
  hi = s;
}

// Adds another lane's pair; EXACT keeps the rounding errors of the sums.
template <bool EXACT>
__device__ __forceinline__ Pair lane_add(Pair s, int d) {
  const float oh = __shfl_xor_sync(0xFFFFFFFFu, s.hi, d);
  if (!EXACT) return {s.hi + oh, 0.0f};
  const float ol = __shfl_xor_sync(0xFFFFFFFFu, s.lo, d);
  const Pair q = two_sum(s.hi, oh);
  return {q.hi, q.lo + (s.lo + ol)};
}

// Sum over a group's wpr warps, in the same order for every thread.  red: two
// sets of one pair per warp of the CTA, used in turn (par), so that one
// barrier per row is enough: a warp writes a set again only after the barrier
// of the row between.
template <bool EXACT>
__device__ __forceinline__ Pair row_sum(Pair s, float2* red, int par, int group, int wpr) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s = lane_add<EXACT>(s, d);
  if (wpr == 1) return s;
  const int lane = threadIdx.x & 31;
  red += par * 32;
  if (lane == 0) red[threadIdx.x >> 5] = make_float2(s.hi, s.lo);
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(32 * wpr) : "memory");
  const float2 o = lane < wpr ? red[group * wpr + lane] : make_float2(0.0f, 0.0f);
  s = {o.x, o.y};
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (d < 2 * wpr) s = lane_add<EXACT>(s, d);
  // (lane 0's is the sum of lanes 0 .. 2^j - 1 with 2^j >= wpr)
  s.hi = __shfl_sync(0xFFFFFFFFu, s.hi, 0);
  s.lo = __shfl_sync(0xFFFFFFFFu, s.lo, 0);
  return s;
}

// 1 / sqrt(ss / n + eps) as hi + lo, good to about 2^-29: the quantised
// outputs round y on a coarse grid, where an error of y of one fp32 step
// already moves some value of a large batch across a rounding boundary (36
// of 58.7 million codes with everything in fp32).
__device__ __forceinline__ Pair inv_rms(Pair ss, float n, float eps) {
  const float q = ss.hi / n;
  const float q_lo = (fmaf(-q, n, ss.hi) + ss.lo) / n;
  Pair w = two_sum(q, eps);
  w.lo += q_lo;
  const float r = 1.0f / sqrtf(w.hi);
  const float a = w.hi * r;                       // Newton: r (1 + e / 2), e = 1 - w r^2
  const float a_lo = fmaf(w.hi, r, -a);
  const float e = fmaf(-a, r, 1.0f) - fmaf(w.lo, r, a_lo) * r;
  return {r, fabsf(e) < 1e-3f ? 0.5f * r * e : 0.0f};  // (no correction for 0, Inf, NaN)
}

// y = p (r.hi + r.lo) rounded to fp32; if it sits on the middle of two E4M3
// values and the rounding dropped something, the neighbour on that side.  (Normal
// E4M3 values: below 2^-14 of its block's largest element a y keeps the fp32
// rounding.)
__device__ __forceinline__ float off_middle(float y, float p, Pair r) {
  if ((__float_as_uint(y) & 0xFFFFFu) != 0x80000u) return y;
  const float rest = fmaf(p, r.hi, -y) + p * r.lo;
  if (rest == 0.0f || rest != rest) return y;
  return __uint_as_float(__float_as_uint(y) + ((rest > 0.0f) == (y > 0.0f) ? 1u : 0xFFFFFFFFu));
}

// V: 16-byte vectors of a row per thread; vector j of a thread is column
// group t + j * 32 wpr of the row.  h_out may be x or res: a thread stores
// only the columns that it alone reads, after it has read them (so those three
// are not __restrict__; the backward's dy, dres and dx likewise).
template <int V>
__global__ void __launch_bounds__(max_threads<V>()) k_rmsnorm_fwd(
    const uint4* x, const uint4* res, const uint4* __restrict__ gamma, float eps, int T,
    int H8, int wpr, int groups, int stages, uint4* h_out, uint4* __restrict__ y, uint8_t* __restrict__ q,
    uint8_t* __restrict__ s, float* __restrict__ rstd) {
  extern __shared__ __align__(16) uint4 ring[];  // [stages][inputs][V][threads]
  __shared__ float2 red[64];
  const int tpr = 32 * wpr, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
  const int nin = res != nullptr ? 2 : 1, nthr = blockDim.x;
  const int slot0 = blockIdx.x * groups + group, slots = gridDim.x * groups;
  auto fetch = [&](int row, int stage) {  // always one group, so that the counts of groups match
    if (row < T) {
      const size_t base = (size_t)row * H8;
      uint4* d = ring + (size_t)stage * nin * V * nthr + threadIdx.x;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = t + j * tpr;
        if (c < H8) {
          cp_async16(d + j * nthr, x + base + c);
          if (nin == 2) cp_async16(d + (V + j) * nthr, res + base + c);
        }
      }
    }
    cp_async_commit();
  };
  uint4 gm[V];
#pragma unroll
  for (int j = 0; j < V; ++j) gm[j] = t + j * tpr < H8 ? __ldg(gamma + t + j * tpr) : make_uint4(0, 0, 0, 0);
  for (int st = 0; st < stages; ++st) fetch(slot0 + st * slots, st);
  int stage = 0, par = 0;
  for (int row = slot0; row < T; row += slots) {
    const size_t base = (size_t)row * H8;
    cp_async_wait(stages - 1);
    const uint4* d = ring + (size_t)stage * nin * V * nthr + threadIdx.x;
    uint4 hv[V];
    float2 hi = pair_of(0.0f), lo = pair_of(0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * tpr;
      hv[j] = make_uint4(0, 0, 0, 0);
      float2 v[4];
      if (c < H8) {
        hv[j] = d[j * nthr];
        if (nin == 2) {
          float2 b[4];
          unpack8(hv[j], v);
          unpack8(d[(V + j) * nthr], b);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = __fadd2_rn(v[i], b[i]);
          hv[j] = pack8(v);
          h_out[base + c] = hv[j];
        }
      }
      unpack8(hv[j], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) add_squares(v[i], hi, lo);
    }
    Pair part = two_sum(hi.x, hi.y);
    part.lo += lo.x + lo.y;
    const Pair sum = row_sum<true>(part, red, par, group, wpr);  // (the row's slots have been read)
    fetch(row + stages * slots, stage);
    if (++stage == stages) stage = 0;
    par ^= 1;
    const Pair r = inv_rms(sum, (float)(8 * H8), eps);
    const float2 rhi = pair_of(r.hi), rlo = pair_of(r.lo);
    if (rstd != nullptr && t == 0) rstd[row] = r.hi + r.lo;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * tpr;
      const bool in = c < H8;
      float2 v[4], g[4];
      unpack8(hv[j], v);
      unpack8(gm[j], g);
      uint32_t mid = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g[i] = __fmul2_rn(v[i], g[i]);  // exact: two 8-bit significands
        v[i] = __ffma2_rn(g[i], rhi, __fmul2_rn(g[i], rlo));
        mid = min(mid, min((__float_as_uint(v[i].x) ^ 0x80000u) & 0xFFFFFu, (__float_as_uint(v[i].y) ^ 0x80000u) & 0xFFFFFu));
      }
      // a y that was rounded onto the middle of two codes (20 bits below E4M3's three: a 1 and zeros): what
      // the rounding dropped decides the code
      if (q != nullptr && mid == 0u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i].x = off_middle(v[i].x, g[i].x, r);
          v[i].y = off_middle(v[i].y, g[i].y, r);
        }
      }
      if (in && y != nullptr) y[base + c] = pack8(v);
      if (q != nullptr) {
        // a 32-column block is four consecutive lanes (H % 32 == 0: all four are in range, or none)
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max_abs(max_abs(m, v[i].x), v[i].y);
        m = max_abs(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max_abs(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const uint32_t sb = e8m0_from_amax_bits(abs_bits(m));
        uint2 code = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        if (sb != 0xFFu) {
          const float2 inv = pair_of(mx_inv_scale(sb));
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = __fmul2_rn(v[i], inv);
          code.x = e4m3x2(v[0].x, v[0].y) | (e4m3x2(v[1].x, v[1].y) << 16);
          code.y = e4m3x2(v[2].x, v[2].y) | (e4m3x2(v[3].x, v[3].y) << 16);
        }
        if (in) {
          reinterpret_cast<uint2*>(q)[base + c] = code;
          if ((c & 3) == 0) s[(base + c) >> 2] = (uint8_t)sb;
        }
      }
    }
  }
}

// Backward.  Every thread keeps the dgamma sums of its own columns over the
// rows it sees (fp32, in row order); they leave as one line per group,
// part[slot][H], and k_dgamma_sum adds the lines in slot order: the result
// does not depend on timing.
template <int V>
__global__ void __launch_bounds__(max_threads<V>()) k_rmsnorm_bwd(
    const uint4* dy, const uint4* dres, const uint4* __restrict__ h,
    const uint4* __restrict__ gamma, const float* __restrict__ rstd, int T, int H8, int wpr, int groups, int stages,
    uint4* dx, float* __restrict__ part) {
  extern __shared__ __align__(16) uint4 ring[];  // [stages][inputs][V][threads]
  __shared__ float2 red[64];
  const int tpr = 32 * wpr, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
  const int nin = dres != nullptr ? 3 : 2, nthr = blockDim.x;
  const int slot0 = blockIdx.x * groups + group, slots = gridDim.x * groups;
  const float inv_h = 1.0f / (float)(8 * H8);
  auto fetch = [&](int row, int stage) {
    if (row < T) {
      const size_t base = (size_t)row * H8;
      uint4* d = ring + (size_t)stage * nin * V * nthr + threadIdx.x;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = t + j * tpr;
        if (c < H8) {
          cp_async16(d + j * nthr, dy + base + c);
          cp_async16(d + (V + j) * nthr, h + base + c);
          if (nin == 3) cp_async16(d + (2 * V + j) * nthr, dres + base + c);
        }
      }
    }
    cp_async_commit();
  };
  float2 acc[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = pair_of(0.0f);
  for (int st = 0; st < stages; ++st) fetch(slot0 + st * slots, st);
  int stage = 0, par = 0;
  float r = slot0 < T ? __ldg(rstd + slot0) : 0.0f;
  for (int row = slot0; row < T; row += slots) {
    const size_t base = (size_t)row * H8;
    const float r_next = row + slots < T ? __ldg(rstd + row + slots) : 0.0f;
    cp_async_wait(stages - 1);
    const uint4* b = ring + (size_t)stage * nin * V * nthr + threadIdx.x;
    uint4 dv[V], hv[V], ev[V];
    float2 dot2 = pair_of(0.0f);
    const float2 r2 = pair_of(r);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * tpr;
      dv[j] = hv[j] = ev[j] = make_uint4(0, 0, 0, 0);
      if (c >= H8) continue;
      dv[j] = b[j * nthr];
      hv[j] = b[(V + j) * nthr];
      if (nin == 3) ev[j] = b[(2 * V + j) * nthr];
      float2 d[4], v[4], g[4];
      unpack8(dv[j], d);
      unpack8(hv[j], v);
      unpack8(__ldg(gamma + c), g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dot2 = __ffma2_rn(__fmul2_rn(d[i], g[i]), v[i], dot2);
        acc[j][i] = __ffma2_rn(d[i], __fmul2_rn(v[i], r2), acc[j][i]);
      }
    }
    const float dot = row_sum<false>(Pair{dot2.x + dot2.y, 0.0f}, red, par, group, wpr).hi;
    fetch(row + stages * slots, stage);
    if (++stage == stages) stage = 0;
    par ^= 1;
    const float2 k = pair_of(-(r * r * (dot * inv_h)));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * tpr;
      if (c >= H8) continue;
      float2 d[4], v[4], g[4], e[4];
      unpack8(dv[j], d);
      unpack8(hv[j], v);
      unpack8(ev[j], e);
      unpack8(__ldg(gamma + c), g);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = __ffma2_rn(r2, __ffma2_rn(v[i], k, __fmul2_rn(d[i], g[i])), e[i]);
      dx[base + c] = pack8(d);
    }
    r = r_next;
  }
  if (part != nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * tpr;
      if (c >= H8) continue;
      float4* d = reinterpret_cast<float4*>(part + (size_t)slot0 * H8 * 8) + 2 * c;
      d[0] = make_float4(acc[j][0].x, acc[j][0].y, acc[j][1].x, acc[j][1].y);
      d[1] = make_float4(acc[j][2].x, acc[j][2].y, acc[j][3].x, acc[j][3].y);
    }
  }
}

// dgamma[c] = sum over the slots of part[slot][c], in a fixed order: warp w
// of 32 takes lines w, w + 32, ... of 32 columns (a few loads each, all in
// flight: a launch of this size is latency), then the warps' sums are added
// in warp order.
__global__ void __launch_bounds__(1024) k_dgamma_sum(const float* __restrict__ part, int slots, int H,
                                                     float* __restrict__ dgamma) {
  __shared__ float sm[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int sl = warp; sl < slots; sl += 32) a += __ldg(part + (size_t)sl * H + c);
  }
  sm[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < H) {
    a = sm[0][lane];
#pragma unroll
    for (int w = 1; w < 32; ++w) a += sm[w][lane];
    dgamma[c] = a;
  }
}

// MXFP8 rows back to bf16: e4m3 * 2^(s - 127) has at most 4 significant bits,
// so the result is exact (unless it leaves bf16's range).  A thread converts 8
// codes at a time (8 bytes in, 16 out, neighbouring threads neighbouring
// codes).
constexpr int DQ_UNROLL = 8;  // loads in flight per thread
__global__ void __launch_bounds__(256) k_dequant_mxfp8(const uint2* __restrict__ q, const uint8_t* __restrict__ s,
                                                       size_t n8, uint4* __restrict__ out) {
  const size_t step = (size_t)gridDim.x * blockDim.x;
  for (size_t i0 = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i0 < n8; i0 += DQ_UNROLL * step) {
    uint2 w[DQ_UNROLL];
    uint32_t sb[DQ_UNROLL];
#pragma unroll
    for (int u = 0; u < DQ_UNROLL; ++u) {
      const size_t i = i0 + u * step;
      w[u] = make_uint2(0, 0);
      sb[u] = 0;
      if (i < n8) {
        w[u] = __ldg(q + i);
        sb[u] = __ldg(s + (i >> 2));
      }
    }
#pragma unroll
    for (int u = 0; u < DQ_UNROLL; ++u) {
      const size_t i = i0 + u * step;
      if (i >= n8) break;
      const float2 sc = pair_of(e8m0_value(sb[u]));
      const float2 v[4] = {__fmul2_rn(e4m3x2_value(w[u].x & 0xFFFFu), sc), __fmul2_rn(e4m3x2_value(w[u].x >> 16), sc),
                           __fmul2_rn(e4m3x2_value(w[u].y & 0xFFFFu), sc), __fmul2_rn(e4m3x2_value(w[u].y >> 16), sc)};
      out[i] = pack8(v);
    }
  }
}

// How the rows are laid over the GPU (see the head of the file).
struct Split {
  bool few;
  int V, wpr, groups, threads;
};
static Split split(int H8, int T) {
  const int lanes = (H8 + 31) / 32;  // warps needed at one vector per thread (<= 64)
  Split p{};
  // Few rows: what runs in one wave.  Two warps' columns of H = 512: 2.3 us
  // against 2.6 at 512 rows (forward), 3.6 against 2.7 at 1024; 2880: 4.0
  // against 4.4 at 320 rows, 4.9 against 4.4 at 512; 7168: 3.6 against 4.4 at
  // 128 rows, 6.1 against 4.4 at 256.  (The backward's crossings are the same.)
  const bool few = T <= FEW_ROWS && T * (lanes < 32 ? lanes : 32) <= FEW_WARPS;
  p.few = few;
  // four vectors of each input per thread where the row is wide enough for two warps of them
  p.V = few ? (lanes > 32 ? 4 : 1) : lanes >= 8 ? 4 : lanes >= 4 ? 2 : 1;
  p.wpr = (lanes + p.V - 1) / p.V;
  p.groups = few ? 1 : 16 / p.wpr;
  if (p.wpr > 1 && p.groups > 15) p.groups = 15;  // one named barrier per group
  p.threads = 32 * p.wpr * p.groups;
  return p;
}
static int ring_stage(const Split& p, int inputs) { return inputs * p.V * p.threads * 16; }
static int ring_stages(const Split& p, int inputs) {
  if (p.few) return 1;
  const int n = RING_BYTES / ring_stage(p, inputs);
  return n < 1 ? 1 : n > 4 ? 4 : n;
}

constexpr int SM_BOUND = 256;  // workspace bound: one CTA per SM of the largest device
static int ctas(int T, int sms, const Split& p) {
  const int need = (T + p.groups - 1) / p.groups;
  const int most = p.few ? FEW_ROWS : sms < SM_BOUND ? sms : SM_BOUND;
  return need < most ? need : most;
}

}  // namespace norm
}  // namespace moeglu

using namespace moeglu;

extern "C" moe_status_t moe_rmsnorm_fwd(const moe_bf16* x, const moe_bf16* residual, const moe_bf16* gamma, float eps,
                                        int T, int H, moe_bf16* h, moe_bf16* y, uint8_t* q, uint8_t* s, float* rstd,
                                        moe_stream_t stream) {
  using namespace norm;
  if (T < 0 || T > MAX_T || H <= 0 || (H & 7) || !(eps >= 0.0f)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !gamma || (residual != nullptr) != (h != nullptr) || (q == nullptr) != (s == nullptr)) return MOE_ERR_ARG;
  if (!y && !q) return MOE_ERR_ARG;
  if (q && (H & 31)) return MOE_ERR_ARG;
  if (H > MAX_H) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(gamma) || (residual && (!aligned16(residual) || !aligned16(h))) ||
      (y && !aligned16(y)) || (q && (reinterpret_cast<uintptr_t>(q) & 7)))
    return MOE_ERR_ARG;
  const int sms = sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  const int H8 = H / 8, inputs = residual ? 2 : 1;
  const Split p = split(H8, T);
  const int stages = ring_stages(p, inputs), smem = stages * ring_stage(p, inputs);
  auto run = [&](auto kernel) {
    if (!set_smem_limit((const void*)kernel, RING_BYTES)) return MOE_ERR_CUDA;
    kernel<<<ctas(T, sms, p), p.threads, smem, as_stream(stream)>>>(
        reinterpret_cast<const uint4*>(x), reinterpret_cast<const uint4*>(residual),
        reinterpret_cast<const uint4*>(gamma), eps, T, H8, p.wpr, p.groups, stages, reinterpret_cast<uint4*>(h),
        reinterpret_cast<uint4*>(y), q, s, rstd);
    count_launch();
    return launch_status();
  };
  return p.V == 1 ? run(k_rmsnorm_fwd<1>) : p.V == 2 ? run(k_rmsnorm_fwd<2>) : run(k_rmsnorm_fwd<4>);
}

extern "C" size_t moe_rmsnorm_bwd_workspace_size(int T, int H) {
  using namespace norm;
  if (T <= 0 || H <= 0 || (H & 7) || H > MAX_H) return 0;
  // one line of dgamma sums per row group of the largest grid
  const Split p = split(H / 8, T);
  return (size_t)ctas(T, SM_BOUND, p) * p.groups * (size_t)H * sizeof(float);
}

extern "C" moe_status_t moe_rmsnorm_bwd(const moe_bf16* dy, const moe_bf16* dres, const moe_bf16* h,
                                        const moe_bf16* gamma, const float* rstd, int T, int H, moe_bf16* dx,
                                        float* dgamma, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace norm;
  if (T < 0 || T > MAX_T || H <= 0 || (H & 7)) return MOE_ERR_ARG;
  if (T == 0) {
    if (dgamma && cudaMemsetAsync(dgamma, 0, (size_t)H * sizeof(float), as_stream(stream)) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!dy || !h || !gamma || !rstd || !dx) return MOE_ERR_ARG;
  if (H > MAX_H) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(dy) || !aligned16(h) || !aligned16(gamma) || !aligned16(dx) || (dres && !aligned16(dres)))
    return MOE_ERR_ARG;
  if (dgamma && (!ws || !aligned16(ws) || ws_bytes < moe_rmsnorm_bwd_workspace_size(T, H))) return MOE_ERR_ARG;
  const int sms = sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  const int H8 = H / 8, inputs = dres ? 3 : 2;
  const Split p = split(H8, T);
  const int grid = ctas(T, sms, p);
  const int stages = ring_stages(p, inputs), smem = stages * ring_stage(p, inputs);
  float* part = dgamma ? static_cast<float*>(ws) : nullptr;
  auto run = [&](auto kernel) {
    if (!set_smem_limit((const void*)kernel, RING_BYTES)) return MOE_ERR_CUDA;
    kernel<<<grid, p.threads, smem, as_stream(stream)>>>(
        reinterpret_cast<const uint4*>(dy), reinterpret_cast<const uint4*>(dres), reinterpret_cast<const uint4*>(h),
        reinterpret_cast<const uint4*>(gamma), rstd, T, H8, p.wpr, p.groups, stages, reinterpret_cast<uint4*>(dx),
        part);
    count_launch();
    return launch_status();
  };
  const moe_status_t rc = p.V == 1 ? run(k_rmsnorm_bwd<1>) : p.V == 2 ? run(k_rmsnorm_bwd<2>) : run(k_rmsnorm_bwd<4>);
  if (rc != MOE_OK || !dgamma) return rc;
  k_dgamma_sum<<<(H + 31) / 32, 1024, 0, as_stream(stream)>>>(part, grid * p.groups, H, dgamma);
  count_launch();
  return launch_status();
}

extern "C" moe_status_t moe_dequantize_mxfp8(const uint8_t* q, const uint8_t* s, size_t blocks, moe_bf16* out,
                                             moe_stream_t stream) {
  using namespace norm;
  if (blocks == 0) return MOE_OK;
  if (!q || !s || !out || !aligned16(q) || !aligned16(out)) return MOE_ERR_ARG;
  const size_t n8 = 4 * blocks;
  size_t grid = (n8 + 255) / 256;
  const size_t cap = (size_t)sm_count() * 8;
  if (cap == 0) return MOE_ERR_CUDA;
  if (grid > cap) grid = cap;
  k_dequant_mxfp8<<<(int)grid, 256, 0, as_stream(stream)>>>(reinterpret_cast<const uint2*>(q), s, n8,
                                                           reinterpret_cast<uint4*>(out));
  count_launch();
  return launch_status();
}
