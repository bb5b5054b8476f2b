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
#include "common.cuh"
#include "host_common.h"

namespace moeglu {
namespace norm {

constexpr int MAX_H = 16384;  // 16 warps x 4 vectors of 8 columns a lane
// threads per CTA: with more than one vector a thread's registers allow 16 warps
template <int V>
constexpr int max_threads() { return V == 1 ? 1024 : 512; }

__device__ __forceinline__ void unpack8(const uint4 q, float* v) {
  v[0] = bf16_lo(q.x);
  v[1] = bf16_hi(q.x);
  v[2] = bf16_lo(q.y);
  v[3] = bf16_hi(q.y);
  v[4] = bf16_lo(q.z);
  v[5] = bf16_hi(q.z);
  v[6] = bf16_lo(q.w);
  v[7] = bf16_hi(q.w);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Sum over the `wpr` warps of a row (a CTA holds whole rows).  red: one float
// per warp of the CTA.  Every thread gets the sum, added in the same order.
__device__ __forceinline__ float row_sum(float v, float* red, int wpr) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if (wpr == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int first = warp / wpr * wpr;
  float s = lane < wpr ? red[first + lane] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  __syncthreads();  // red is free again
  return s;
}

// V: 16-byte vectors of a row per thread.  A row belongs to wpr warps, a CTA
// to blockDim / (32 wpr) rows; vector j of a thread is column group
// t + j * 32 wpr of the row.
template <int V>
__global__ void __launch_bounds__(max_threads<V>()) k_rmsnorm_fwd(const uint4* __restrict__ x, const uint4* __restrict__ res,
                              const uint4* __restrict__ gamma, float eps, int T, int H8, int wpr,
                              uint4* __restrict__ h_out, uint4* __restrict__ y, uint8_t* __restrict__ q,
                              uint8_t* __restrict__ s, float* __restrict__ rstd) {
  __shared__ float red[32];
  const int tpr = 32 * wpr, t = threadIdx.x % tpr, rows = blockDim.x / tpr;
  const int row = blockIdx.x * rows + threadIdx.x / tpr;
  const bool on = row < T;
  const size_t base = (size_t)row * H8;
  uint4 hv[V];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = t + j * tpr;
    hv[j] = make_uint4(0, 0, 0, 0);
    if (on && c < H8) {
      hv[j] = __ldg(x + base + c);
      if (res != nullptr) {
        float a[8], b[8];
        unpack8(hv[j], a);
        unpack8(__ldg(res + base + c), b);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] += b[i];
        hv[j] = pack8(a);
        h_out[base + c] = hv[j];
      }
    }
    float v[8];
    unpack8(hv[j], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
  }
  ss = row_sum(ss, red, wpr);
  const float r = 1.0f / sqrtf(ss / (float)(8 * H8) + eps);
  if (on && rstd != nullptr && t == 0) rstd[row] = r;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = t + j * tpr;
    const bool in = on && c < H8;
    float v[8], g[8];
    unpack8(hv[j], v);
    unpack8(in ? __ldg(gamma + c) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * r * g[i];
    if (in && y != nullptr) y[base + c] = pack8(v);
    if (q != nullptr) {
      // a 32-column block is four consecutive lanes (H % 32 == 0: all four are in range, or none)
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const uint32_t sb = e8m0_from_amax_bits(m);
      uint2 code = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
      if (sb != 0xFFu) {
        const float inv = mx_inv_scale(sb);
        code.x = e4m3x2(v[0] * inv, v[1] * inv) | (e4m3x2(v[2] * inv, v[3] * inv) << 16);
        code.y = e4m3x2(v[4] * inv, v[5] * inv) | (e4m3x2(v[6] * inv, v[7] * inv) << 16);
      }
      if (in) {
        reinterpret_cast<uint2*>(q)[base + c] = code;
        if ((c & 3) == 0) s[(base + c) >> 2] = (uint8_t)sb;
      }
    }
  }
}

// Backward.  A CTA walks rows blockIdx.x * rows + ..., and every thread keeps
// the dgamma sums of its own columns over the rows it sees (fp32, in row
// order); they leave as one line per row slot of the CTA, part[slot][H], and
// k_dgamma_sum adds the lines in slot order: the result does not depend on
// timing.
template <int V>
__global__ void __launch_bounds__(max_threads<V>()) k_rmsnorm_bwd(const uint4* __restrict__ dy, const uint4* __restrict__ dres,
                              const uint4* __restrict__ h, const uint4* __restrict__ gamma,
                              const float* __restrict__ rstd, int T, int H8, int wpr, uint4* __restrict__ dx,
                              float* __restrict__ part) {
  __shared__ float red[32];
  const int tpr = 32 * wpr, t = threadIdx.x % tpr, rows = blockDim.x / tpr;
  const int slot = blockIdx.x * rows + threadIdx.x / tpr, slots = gridDim.x * rows;
  const float inv_h = 1.0f / (float)(8 * H8);
  float acc[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
  const int steps = (T + slots - 1) / slots;  // the same for every thread: the row sum has barriers
  for (int st = 0; st < steps; ++st) {
    const int row = slot + st * slots;
    const bool on = row < T;
    const size_t base = (size_t)row * H8;
    uint4 dv[V], hv[V];
    float dot = 0.0f;
    const float r = on ? __ldg(rstd + row) : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * tpr;
      dv[j] = hv[j] = make_uint4(0, 0, 0, 0);
      if (on && c < H8) {
        dv[j] = __ldg(dy + base + c);
        hv[j] = __ldg(h + base + c);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * tpr;
      float d[8], v[8], g[8];
      unpack8(dv[j], d);
      unpack8(hv[j], v);
      unpack8(c < H8 ? __ldg(gamma + c) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot = fmaf(d[i] * g[i], v[i], dot);
        acc[j][i] = fmaf(d[i], v[i] * r, acc[j][i]);
      }
    }
    dot = row_sum(dot, red, wpr);
    const float k = r * r * (dot * inv_h);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * tpr;
      if (!on || c >= H8) continue;
      float d[8], v[8], g[8], o[8];
      unpack8(dv[j], d);
      unpack8(hv[j], v);
      unpack8(__ldg(gamma + c), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = r * (d[i] * g[i] - v[i] * k);
      if (dres != nullptr) {
        float e[8];
        unpack8(__ldg(dres + base + c), e);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += e[i];
      }
      dx[base + c] = pack8(o);
    }
  }
  if (part != nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * tpr;
      if (c >= H8) continue;
      float4* d = reinterpret_cast<float4*>(part + (size_t)slot * H8 * 8) + 2 * c;
      d[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      d[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
  }
}

// dgamma[c] = sum over the slots of part[slot][c], in a fixed order: 8 warps
// take every eighth line of 32 columns, then their sums are added in warp order.
__global__ void __launch_bounds__(256) k_dgamma_sum(const float* __restrict__ part, int slots, int H,
                                                    float* __restrict__ dgamma) {
  __shared__ float sm[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.0f;
  if (c < H)
    for (int sl = warp; sl < slots; sl += 8) a += __ldg(part + (size_t)sl * H + c);
  sm[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < H) {
    a = sm[0][lane];
#pragma unroll
    for (int w = 1; w < 8; ++w) a += sm[w][lane];
    dgamma[c] = a;
  }
}

// MXFP8 rows back to bf16: e4m3 * 2^(s - 127) has at most 4 significant bits,
// so the result is exact (unless it leaves bf16's range).  One thread per 16
// codes (16 bytes in, 32 out).
__global__ void __launch_bounds__(256) k_dequant_mxfp8(const uint4* __restrict__ q, const uint8_t* __restrict__ s,
                                                       size_t n16, uint4* __restrict__ out) {
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n16; i += (size_t)gridDim.x * blockDim.x) {
    const uint4 w = __ldg(q + i);
    const uint32_t sb = __ldg(s + (i >> 1));
    const float sc = e8m0_value(sb);
    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
    float v[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = e4m3x2_value(c[j] & 0xFFFFu), b = e4m3x2_value(c[j] >> 16);
      v[4 * j] = a.x * sc;
      v[4 * j + 1] = a.y * sc;
      v[4 * j + 2] = b.x * sc;
      v[4 * j + 3] = b.y * sc;
    }
    out[2 * i] = pack8(v);
    out[2 * i + 1] = pack8(v + 8);
  }
}

// How a row is split: V vectors per thread and wpr warps per row.  Rows wide
// enough take four vectors per thread, so that a thread has four 16-byte
// loads of each input in flight; a call of few rows spreads each over as many
// warps as it has vectors for, because then one row's latency is the call's
// time.
constexpr int FEW_ROWS = 256;
struct Split {
  int V, wpr, threads, rows;  // rows per CTA
};
static Split split(int H8, int T) {
  const int lanes = (H8 + 31) / 32;  // warps needed at one vector per thread (<= 64)
  Split p{};
  p.V = T <= FEW_ROWS ? (lanes > 32 ? 4 : 1) : lanes >= 8 ? 4 : lanes >= 4 ? 2 : 1;
  const int need = (lanes + p.V - 1) / p.V;
  p.wpr = 1;
  while (p.wpr < need) p.wpr *= 2;
  p.threads = p.wpr >= 8 ? 32 * p.wpr : 256;
  p.rows = p.threads / (32 * p.wpr);
  return p;
}

// CTAs of the backward: a few per SM, so that each walks many rows and the
// partial sums stay a small share of the traffic; never more than BWD_CTAS
constexpr int BWD_CTAS = 1024;
static int bwd_ctas(int T, int sms, const Split& p) {
  const int need = (T + p.rows - 1) / p.rows;
  int c = sms * (p.threads > 256 ? 2 : 4);
  if (c > BWD_CTAS) c = BWD_CTAS;
  return need < c ? need : c;
}

}  // namespace norm
}  // namespace moeglu

using namespace moeglu;

extern "C" moe_status_t moe_rmsnorm_fwd(const moe_bf16* x, const moe_bf16* residual, const moe_bf16* gamma, float eps,
                                        int T, int H, moe_bf16* h, moe_bf16* y, uint8_t* q, uint8_t* s, float* rstd,
                                        moe_stream_t stream) {
  using namespace norm;
  if (T < 0 || H <= 0 || (H & 7) || !(eps >= 0.0f)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !gamma || (residual != nullptr) != (h != nullptr) || (q == nullptr) != (s == nullptr)) return MOE_ERR_ARG;
  if (!y && !q) return MOE_ERR_ARG;
  if (q && (H & 31)) return MOE_ERR_ARG;
  if (H > MAX_H) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(gamma) || (residual && (!aligned16(residual) || !aligned16(h))) ||
      (y && !aligned16(y)) || (q && (reinterpret_cast<uintptr_t>(q) & 7)))
    return MOE_ERR_ARG;
  const int H8 = H / 8;
  const Split p = split(H8, T);
  const int grid = (T + p.rows - 1) / p.rows;
  auto run = [&](auto kernel) {
    kernel<<<grid, p.threads, 0, as_stream(stream)>>>(
        reinterpret_cast<const uint4*>(x), reinterpret_cast<const uint4*>(residual),
        reinterpret_cast<const uint4*>(gamma), eps, T, H8, p.wpr, reinterpret_cast<uint4*>(h),
        reinterpret_cast<uint4*>(y), q, s, rstd);
  };
  if (p.V == 1)
    run(k_rmsnorm_fwd<1>);
  else if (p.V == 2)
    run(k_rmsnorm_fwd<2>);
  else
    run(k_rmsnorm_fwd<4>);
  count_launch();
  return launch_status();
}

extern "C" size_t moe_rmsnorm_bwd_workspace_size(int T, int H) {
  using namespace norm;
  if (T <= 0 || H <= 0 || (H & 7) || H > MAX_H) return 0;
  // one line of dgamma sums per row slot of the largest grid
  const Split p = split(H / 8, T);
  const int need = (T + p.rows - 1) / p.rows;
  return (size_t)(need < BWD_CTAS ? need : BWD_CTAS) * p.rows * (size_t)H * sizeof(float);
}

extern "C" moe_status_t moe_rmsnorm_bwd(const moe_bf16* dy, const moe_bf16* dres, const moe_bf16* h,
                                        const moe_bf16* gamma, const float* rstd, int T, int H, moe_bf16* dx,
                                        float* dgamma, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace norm;
  if (T < 0 || H <= 0 || (H & 7)) return MOE_ERR_ARG;
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
  const int H8 = H / 8;
  const Split p = split(H8, T);
  const int ctas = bwd_ctas(T, sms, p);
  float* part = dgamma ? static_cast<float*>(ws) : nullptr;
  auto run = [&](auto kernel) {
    kernel<<<ctas, p.threads, 0, as_stream(stream)>>>(
        reinterpret_cast<const uint4*>(dy), reinterpret_cast<const uint4*>(dres), reinterpret_cast<const uint4*>(h),
        reinterpret_cast<const uint4*>(gamma), rstd, T, H8, p.wpr, reinterpret_cast<uint4*>(dx), part);
  };
  if (p.V == 1)
    run(k_rmsnorm_bwd<1>);
  else if (p.V == 2)
    run(k_rmsnorm_bwd<2>);
  else
    run(k_rmsnorm_bwd<4>);
  count_launch();
  if (dgamma) {
    k_dgamma_sum<<<(H + 31) / 32, 256, 0, as_stream(stream)>>>(part, ctas * p.rows, H, dgamma);
    count_launch();
  }
  return launch_status();
}

extern "C" moe_status_t moe_dequantize_mxfp8(const uint8_t* q, const uint8_t* s, size_t blocks, moe_bf16* out,
                                             moe_stream_t stream) {
  using namespace norm;
  if (blocks == 0) return MOE_OK;
  if (!q || !s || !out || !aligned16(q) || !aligned16(out)) return MOE_ERR_ARG;
  const size_t n16 = 2 * blocks;
  size_t grid = (n16 + 255) / 256;
  const size_t cap = (size_t)sm_count() * 16;
  if (cap == 0) return MOE_ERR_CUDA;
  if (grid > cap) grid = cap;
  k_dequant_mxfp8<<<(int)grid, 256, 0, as_stream(stream)>>>(reinterpret_cast<const uint4*>(q), s, n16,
                                                           reinterpret_cast<uint4*>(out));
  count_launch();
  return launch_status();
}
