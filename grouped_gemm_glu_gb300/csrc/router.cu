// The router: expert choice and weights from the logits of a batch, and the
// gradient of the weights with respect to the logits.
//
//   s_e  = softmax(x)_e or sigmoid(x_e)
//   key  = s_e + bias_e; without a bias the logit itself, which orders the
//          experts as the scores do
//   group score = sum of the group_top best keys of a group (its best key, or
//          its two best scores); experts outside the topk_group best groups
//          are out
//   the k largest keys, ties to the lowest index; weight = the score,
//   renormalised over the chosen experts if asked, times scale
//
// One warp per token, lane l holding experts l, l + 32, ...: keys are the
// floats' bits mapped to unsigned integers of the same order, so that a
// round of the choice is a max over the lane's registers and two warp
// reductions (redux.sync): the largest key, then the lowest index that has
// it.  An expert with a logit (or bias) of -inf is never chosen.
//
// Memory: each logit is read once (4 or 2 bytes), 8 bytes leave per chosen
// expert.  A batch of 8192 x 256 fp32 logits is 8.4 MB, so the instructions
// of the k rounds bound the kernel, not HBM.
#include <type_traits>

#include "common.cuh"
#include "host_common.h"

namespace moeglu {
namespace router {

constexpr int N_MAX = 1024, K_MAX = 32, G_MAX = 32;
constexpr int WARPS = 8;
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;  // ordered_key(-inf): keys at or below it are not chosen

struct Params {
  int n, k, score, renorm, G, keep, gtop;
  float scale;
};

// Unsigned integers in the order of the floats: -inf < ... < -0 = +0 < ... <
// +inf < NaN (a NaN is chosen first, so that it shows in the weights).
__device__ __forceinline__ uint32_t ordered_key(float f) {
  if (f != f) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(f + 0.0f);  // -0 + 0 = +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

__device__ __forceinline__ float load_logit(const void* p, size_t i, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16)
              : __ldg(static_cast<const float*>(p) + i);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  return v;
}

// Scores of the lane's VL logits (x, -inf past n), and for softmax the row's
// sums; every form rounds as the formula written out in fp32 does.
template <int VL>
__device__ __forceinline__ void scores(const float* x, int score, float* s) {
  if (score == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < VL; ++i) s[i] = 1.0f / (1.0f + expf(-x[i]));
    return;
  }
  float m = x[0];
#pragma unroll
  for (int i = 1; i < VL; ++i) m = fmaxf(m, x[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.0f;  // a row without experts: every score is 0
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VL; ++i) {
    s[i] = expf(x[i] - m);
    sum += s[i];
  }
  sum = warp_sum(sum);
  const float d = fmaxf(sum, 1e-38f);
#pragma unroll
  for (int i = 0; i < VL; ++i) s[i] = sum != sum ? sum : s[i] / d;
}

template <int VL>
__global__ void __launch_bounds__(32 * WARPS) k_router_fwd(const void* __restrict__ logits, int bf16,
                                                           const float* __restrict__ bias,
                                                           const uint8_t* __restrict__ mask, int T, const Params p,
                                                           int32_t* __restrict__ idx, float* __restrict__ prob,
                                                           int32_t* __restrict__ load) {
  extern __shared__ int32_t hist[];  // [n] when load is counted
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (load != nullptr) {
    for (int e = threadIdx.x; e < p.n; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const int n = p.n;
  for (int t = blockIdx.x * WARPS + warp; t < T; t += gridDim.x * WARPS) {
    const bool live = mask == nullptr || __ldg(mask + t) != 0;
    float x[VL], s[VL];
    uint32_t key[VL];
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int e = lane + 32 * i;
      x[i] = e < n ? load_logit(logits, (size_t)t * n + e, bf16) : -INFINITY;
    }
    // scores are needed for the weights (unless they are the softmax of the
    // chosen logits alone), for a bias and for sums of group scores
    const bool need_s = p.score == MOE_SCORE_SIGMOID || !p.renorm || bias != nullptr || p.gtop > 1;
    if (need_s) scores<VL>(x, p.score, s);
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int e = lane + 32 * i;
      float f = x[i];
      if (bias != nullptr && e < n && f != -INFINITY) f = s[i] + __ldg(bias + e);
      key[i] = e < n ? ordered_key(f) : 0u;
    }
    if (p.G > 1) {
      // group scores: lane g ends with the score of group g
      const int gs = n / p.G;
      float mine = -INFINITY;
      for (int g = 0; g < p.G; ++g) {
        const int lo = g * gs, hi = lo + gs;
        uint32_t b1 = 0, b2 = 0;  // the lane's best two of the group
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          const int e = lane + 32 * i;
          if (e >= lo && e < hi) {
            uint32_t kk = key[i];
            if (p.gtop > 1 && bias == nullptr) kk = x[i] == -INFINITY ? KEY_NEG_INF : ordered_key(s[i]);
            b2 = max(b2, min(b1, kk));
            b1 = max(b1, kk);
          }
        }
        const uint32_t m1 = __reduce_max_sync(0xFFFFFFFFu, b1);
        float sc = key_value(m1);
        if (p.gtop > 1 && gs > 1) {
          const unsigned who = __ballot_sync(0xFFFFFFFFu, b1 == m1);
          const uint32_t rest = (lane == __ffs(who) - 1) ? b2 : b1;
          sc += key_value(__reduce_max_sync(0xFFFFFFFFu, rest));
        }
        if (lane == g) mine = sc;
      }
      // keep the topk_group best: lane g counts the groups that come before it
      const uint32_t gk = lane < p.G ? ordered_key(mine) : 0u;
      int before = 0;
      for (int g = 0; g < p.G; ++g) {
        const uint32_t o = __shfl_sync(0xFFFFFFFFu, gk, g);
        before += (o > gk || (o == gk && g < lane)) ? 1 : 0;
      }
      const unsigned kept = __ballot_sync(0xFFFFFFFFu, lane < p.G && before < p.keep);
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const int e = lane + 32 * i;
        if (e < n && !((kept >> (e / gs)) & 1u)) key[i] = 0u;
      }
    }
    // the choice: lane j keeps the j-th expert
    int my_idx = -1;
    float my_val = 0.0f;
    if (live) {
      for (int j = 0; j < p.k; ++j) {
        uint32_t b = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < VL; ++i)
          if (key[i] > b) {
            b = key[i];
            bi = i;
          }
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, b);
        if (m <= KEY_NEG_INF) break;
        const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, b == m ? (uint32_t)(lane + 32 * bi) : 0xFFFFFFFFu);
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < VL; ++i)
          if (e == (uint32_t)(lane + 32 * i)) {
            key[i] = 0u;
            v = need_s && !(p.renorm && p.score == MOE_SCORE_SOFTMAX) ? s[i] : x[i];
          }
        v = __shfl_sync(0xFFFFFFFFu, v, e & 31u);
        if (lane == j) {
          my_idx = (int)e;
          my_val = v;
        }
      }
    }
    if (p.renorm) {
      if (p.score == MOE_SCORE_SOFTMAX) {
        const float m = warp_max(my_idx >= 0 ? my_val : -INFINITY);
        const float ex = my_idx >= 0 ? expf(my_val - m) : 0.0f;
        const float sum = warp_sum(ex);
        my_val = my_idx >= 0 ? ex / sum : 0.0f;
      } else {
        my_val = my_val / (warp_sum(my_val) + 1e-20f);
      }
    }
    if (lane < p.k) {
      idx[(size_t)t * p.k + lane] = my_idx;
      prob[(size_t)t * p.k + lane] = my_val * p.scale;
      if (load != nullptr && my_idx >= 0) atomicAdd(&hist[my_idx], 1);
    }
  }
  if (load != nullptr) {
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += blockDim.x)
      if (hist[e] != 0) atomicAdd(load + e, hist[e]);  // integers: the order does not matter
  }
}

__device__ __forceinline__ void store_logit(void* p, size_t i, float v, int bf16) {
  if (bf16)
    static_cast<uint16_t*>(p)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  else
    static_cast<float*>(p)[i] = v;
}

// Backward, one warp per token; lane j < k holds the j-th chosen expert with
// g_j = scale * dprob_j.  With w the weights before the factor:
//   softmax, renormalised:   dx_j = w_j (g_j - sum g w)            (chosen only)
//   softmax:                 dx_e = [e chosen] g s_e - s_e sum_j g_j s_j
//   sigmoid, renormalised:   dx_j = (g_j - sum g w) / D * s_j (1 - s_j),  D = sum s + 1e-20
//   sigmoid:                 dx_j = g_j s_j (1 - s_j)
// Experts without a gradient get 0; only the plain softmax reads every logit.
template <int VL>
__global__ void __launch_bounds__(32 * WARPS) k_router_bwd(const void* __restrict__ logits, int bf16,
                                                           const int32_t* __restrict__ idx,
                                                           const float* __restrict__ dprob, int T, const Params p,
                                                           void* __restrict__ dlogits) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = p.n;
  for (int t = blockIdx.x * WARPS + warp; t < T; t += gridDim.x * WARPS) {
    int e = -1;
    float g = 0.0f, xe = -INFINITY;
    if (lane < p.k) {
      e = __ldg(idx + (size_t)t * p.k + lane);
      if (e < 0 || e >= n) e = -1;
      if (e >= 0) {
        g = p.scale * __ldg(dprob + (size_t)t * p.k + lane);
        xe = load_logit(logits, (size_t)t * n + e, bf16);
      }
    }
    float out[VL];
#pragma unroll
    for (int i = 0; i < VL; ++i) out[i] = 0.0f;
    float d;  // gradient of the lane's chosen logit
    if (p.score == MOE_SCORE_SIGMOID) {
      const float s = e >= 0 ? 1.0f / (1.0f + expf(-xe)) : 0.0f;
      const float s1 = 1.0f / (1.0f + expf(xe));  // 1 - s without the cancellation
      if (p.renorm) {
        const float D = warp_sum(s) + 1e-20f;
        const float in = warp_sum(g * (s / D));
        d = (g - in) / D * s * s1;
      } else {
        d = g * s * s1;
      }
    } else if (p.renorm) {
      const float m = warp_max(xe);
      const float ex = e >= 0 ? expf(xe - m) : 0.0f;
      const float w = ex / fmaxf(warp_sum(ex), 1e-38f);
      d = w * (g - warp_sum(g * w));
    } else {
      float x[VL], s[VL];
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const int c = lane + 32 * i;
        x[i] = c < n ? load_logit(logits, (size_t)t * n + c, bf16) : -INFINITY;
      }
      scores<VL>(x, p.score, s);
      float se = 0.0f;  // the score of the lane's chosen expert
      for (int j = 0; j < p.k; ++j) {
        const int ej = __shfl_sync(0xFFFFFFFFu, e, j);
        if (ej < 0) continue;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < VL; ++i)
          if (ej == lane + 32 * i) v = s[i];
        v = __shfl_sync(0xFFFFFFFFu, v, ej & 31);
        if (lane == j) se = v;
      }
      d = g * se;
      const float in = warp_sum(d);
#pragma unroll
      for (int i = 0; i < VL; ++i) out[i] = -s[i] * in;
    }
    for (int j = 0; j < p.k; ++j) {
      const int ej = __shfl_sync(0xFFFFFFFFu, e, j);
      const float dj = __shfl_sync(0xFFFFFFFFu, d, j);
      if (ej < 0) continue;
#pragma unroll
      for (int i = 0; i < VL; ++i)
        if (ej == lane + 32 * i) out[i] += dj;
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int c = lane + 32 * i;
      if (c < n) store_logit(dlogits, (size_t)t * n + c, out[i], bf16);
    }
  }
}

static bool params_ok(const moe_router_params_t* q, int n, int k) {
  return q && (q->score == MOE_SCORE_SOFTMAX || q->score == MOE_SCORE_SIGMOID) && n > 0 && n <= N_MAX && k > 0 &&
         k <= K_MAX && k <= n && q->n_group >= 1 && q->n_group <= G_MAX && n % q->n_group == 0 &&
         q->topk_group >= 1 && q->topk_group <= q->n_group && (q->group_top == 1 || q->group_top == 2) &&
         k <= n / q->n_group * q->topk_group && q->scale == q->scale;
}

static int grid_of(int T) {
  const long long need = ((long long)T + WARPS - 1) / WARPS, cap = (long long)sm_count() * 8;
  return (int)(need < cap ? need : cap);
}

// lane registers for n experts: the next power of two of n / 32
template <class F>
static void dispatch(int n, F&& f) {
  const int vl = (n + 31) / 32;
  if (vl <= 1)
    f(std::integral_constant<int, 1>{});
  else if (vl <= 2)
    f(std::integral_constant<int, 2>{});
  else if (vl <= 4)
    f(std::integral_constant<int, 4>{});
  else if (vl <= 8)
    f(std::integral_constant<int, 8>{});
  else if (vl <= 16)
    f(std::integral_constant<int, 16>{});
  else
    f(std::integral_constant<int, 32>{});
}

}  // namespace router
}  // namespace moeglu

using namespace moeglu;

extern "C" moe_status_t moe_router_fwd(const void* logits, int logits_bf16, const float* bias,
                                       const uint8_t* token_mask, int T, int n, int k,
                                       const moe_router_params_t* params, int32_t* topk_idx, float* topk_prob,
                                       int32_t* load, moe_stream_t stream) {
  using namespace router;
  if (T < 0 || !params_ok(params, n, k)) return MOE_ERR_ARG;
  if ((int64_t)T * k > (int64_t)INT32_MAX / 2) return MOE_ERR_ARG;
  if (T > 0 && (!logits || !topk_idx || !topk_prob)) return MOE_ERR_ARG;
  cudaStream_t st = as_stream(stream);
  if (load && cudaMemsetAsync(load, 0, (size_t)n * sizeof(int32_t), st) != cudaSuccess) return MOE_ERR_CUDA;
  if (T == 0) return MOE_OK;
  const Params p{n, k, params->score, params->renorm ? 1 : 0, params->n_group, params->topk_group, params->group_top,
                 params->scale};
  const int grid = grid_of(T);
  if (grid <= 0) return MOE_ERR_CUDA;
  dispatch(n, [&](auto vl) {
    k_router_fwd<decltype(vl)::value><<<grid, 32 * WARPS, load ? n * sizeof(int32_t) : 0, st>>>(
        logits, logits_bf16 ? 1 : 0, bias, token_mask, T, p, topk_idx, topk_prob, load);
  });
  count_launch();
  return launch_status();
}

extern "C" moe_status_t moe_router_bwd(const void* logits, int logits_bf16, const int32_t* topk_idx,
                                       const float* dprob, int T, int n, int k, const moe_router_params_t* params,
                                       void* dlogits, moe_stream_t stream) {
  using namespace router;
  if (T < 0 || !params_ok(params, n, k)) return MOE_ERR_ARG;
  if ((int64_t)T * k > (int64_t)INT32_MAX / 2) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !dprob || !dlogits) return MOE_ERR_ARG;
  const Params p{n, k, params->score, params->renorm ? 1 : 0, params->n_group, params->topk_group, params->group_top,
                 params->scale};
  const int grid = grid_of(T);
  if (grid <= 0) return MOE_ERR_CUDA;
  dispatch(n, [&](auto vl) {
    k_router_bwd<decltype(vl)::value><<<grid, 32 * WARPS, 0, as_stream(stream)>>>(
        logits, logits_bf16 ? 1 : 0, topk_idx, dprob, T, p, dlogits);
  });
  count_launch();
  return launch_status();
}
