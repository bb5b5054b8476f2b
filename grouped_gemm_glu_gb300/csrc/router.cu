// The router: expert choice and weights from the logits of a batch, and the
// gradient of the weights with respect to the logits.
//
//   s_e  = softmax(x)_e or sigmoid(x_e)
//   key  = s_e + bias_e; without a bias the logit itself, which orders the
//          experts as the scores do
//   group score = sum of the group_top best keys of a group (its best key, or
//          its two best scores; -inf where fewer are left); experts outside
//          the topk_group best groups are out
//   the k largest keys, ties to the lowest index; weight = the score,
//   renormalised over the chosen experts if asked, times scale
//
// One warp per token; lane l holds the VL neighbouring experts l VL .. l VL +
// VL - 1 (VL = 1, 2, 4, ... with 32 VL >= n), so that a row is read in one or
// two vector loads per lane, a group of experts is a run of lanes whose best
// keys meet in a few shuffles, and the lowest lane among equal keys holds the
// lowest index.  Keys are the floats' bits mapped to unsigned integers of the
// same order, sorted within each lane by min / max: a round of the choice is
// one warp reduction (redux.sync) over the lanes' best keys and a ballot, and
// the lane that held the winner moves its list up.  Which of that lane's
// experts had the key is settled once, after the rounds, by lane j for the
// j-th choice from a copy of the keys in shared memory; lane j then computes
// the weight from the expert's logit.  An
// expert with a logit (or bias) of -inf is never chosen.
//
// Memory: each logit is read once (4 or 2 bytes), 8 bytes leave per chosen
// expert; at 8192 x 256 that is 1.3 us of HBM time.  What bounds the kernel is
// the latency of the chain from the loads over the scores and the k rounds:
// 12.6 us with 8 groups, bias and top-8 (issue slots 45% busy, half of the
// warps resident on average: 8192 tokens are 1.7 rounds of 152 x 32 warps), 9.6
// us for 32768 x 64 top-6 (41%), 4.4 us for one token.  Backward of 32768 x 64
// 8.7 us (46%; half of the stalls wait for its loads).
#include <type_traits>

#include "common.cuh"
#include "host_common.h"

namespace moeglu {
namespace router {

constexpr int N_MAX = 1024, K_MAX = 32, G_MAX = 32;
template <int VL>
constexpr int max_warps() { return VL <= 8 ? 32 : VL < 32 ? 16 : 8; }  // per CTA: registers, and 32 KB of keys
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;  // ordered_key(-inf): keys at or below it are not chosen

struct Params {
  int n, k, score, renorm, G, keep, gtop;
  float scale;
  // set by dispatch(): experts per group; log2 of the lanes per group where
  // groups are whole runs of 2^j lanes, else -1; whether the logits' and the
  // bias's rows start on a lane's vector
  int gs, seg_log, vec, vec_bias;
};

// Unsigned integers in the order of the floats: -inf < ... < -0 = +0 < ... <
// +inf < NaN (a NaN is chosen first, so that it shows in the weights).
__device__ __forceinline__ uint32_t ordered_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);  // -0 + 0 = +0
  return f != f ? 0xFFFFFFFFu : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, size_t i) {
  return BF16 ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16)
              : __ldg(static_cast<const float*>(p) + i);
}

// The lane's VL logits of row t, -inf past n.  vec: rows start on the
// alignment of one lane's vector, and n is a multiple of VL.
template <int VL, bool BF16>
__device__ __forceinline__ void load_row(const void* p, size_t t, int n, int lane, bool vec, float* x) {
  const int e0 = lane * VL;
  if (vec) {
#pragma unroll
    for (int i = 0; i < VL; ++i) x[i] = -INFINITY;
    if (e0 >= n) return;
    if (BF16) {
      const uint16_t* s = static_cast<const uint16_t*>(p) + t * n + e0;
      if (VL == 1) {
        x[0] = __uint_as_float((uint32_t)__ldg(s) << 16);
      } else if (VL == 2) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(s));
        x[0] = bf16_lo(w);
        x[VL - 1] = bf16_hi(w);
      } else if (VL == 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(s));
        x[0] = bf16_lo(w.x);
        x[1 % VL] = bf16_hi(w.x);
        x[2 % VL] = bf16_lo(w.y);
        x[3 % VL] = bf16_hi(w.y);
      } else {
#pragma unroll
        for (int c = 0; c < VL / 8; ++c) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(s) + c);
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) x[(8 * c + i) % VL] = (i & 1) ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]);
        }
      }
    } else {
      const float* s = static_cast<const float*>(p) + t * n + e0;
      if (VL == 1) {
        x[0] = __ldg(s);
      } else if (VL == 2) {
        const float2 w = __ldg(reinterpret_cast<const float2*>(s));
        x[0] = w.x;
        x[VL - 1] = w.y;
      } else {
#pragma unroll
        for (int c = 0; c < VL / 4; ++c) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(s) + c);
          x[(4 * c) % VL] = w.x;
          x[(4 * c + 1) % VL] = w.y;
          x[(4 * c + 2) % VL] = w.z;
          x[(4 * c + 3) % VL] = w.w;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < VL; ++i) x[i] = e0 + i < n ? load_logit<BF16>(p, t * n + e0 + i) : -INFINITY;
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

// Each rounds as the formula 1 / (1 + exp(-x)) in fp32 does (a correctly
// rounded reciprocal is the quotient of 1).
__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.0f + expf(-x)); }

// Softmax of the row: its largest logit (0 for a row without experts) and
// the sum of the exponentials; a score is expf(x - m) / d.
struct Soft {
  float m, d;
};
template <int VL>
__device__ __forceinline__ Soft softmax_of(const float* x) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < VL; ++i) m = fmaxf(m, x[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VL; ++i) sum += expf(x[i] - m);
  sum = warp_sum(sum);
  return {m, sum != sum ? sum : fmaxf(sum, 1e-38f)};
}
__device__ __forceinline__ float soft_score(const Soft& s, float x) { return expf(x - s.m) / s.d; }

// The counts of this CTA into load (whole CTA).  A lone CTA has every count;
// otherwise load was cleared by the kernel before this one, which the launch
// overlaps with this one up to here (programmatic dependent launch).
__device__ __forceinline__ void flush_load(const int32_t* hist, int n, int32_t* load) {
  __syncthreads();
  if (gridDim.x > 1) wait_for_primary();
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    if (gridDim.x == 1)
      load[e] = hist[e];
    else if (hist[e] != 0)
      atomicAdd(load + e, hist[e]);  // integers: the order does not matter
  }
}
__global__ void k_router_clear(int32_t* __restrict__ load, int n) {
  launch_dependents();
  for (int e = threadIdx.x; e < n; e += blockDim.x) load[e] = 0;
}

// Descending order of VL keys (Batcher's odd-even merge sort, unrolled).
template <int VL>
__device__ __forceinline__ void sort_desc(uint32_t* v) {
#pragma unroll
  for (int p = 1; p < VL; p *= 2) {
#pragma unroll
    for (int k = p; k >= 1; k /= 2) {
#pragma unroll
      for (int j = k % p; j + k < VL; j += 2 * k) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
          if (i + j + k < VL && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t hi = max(v[i + j], v[i + j + k]), lo = min(v[i + j], v[i + j + k]);
            v[i + j] = hi;
            v[i + j + k] = lo;
          }
        }
      }
    }
  }
}

// Dynamic shared memory: the keys of the warps' rows ([warps][32 VL]), then
// the histogram [n] when load is counted.
template <int VL, bool BF16>
__global__ void __launch_bounds__(32 * max_warps<VL>()) k_router_fwd(const void* __restrict__ logits,
                                                           const float* __restrict__ bias,
                                                           const uint8_t* __restrict__ mask, int T, const Params p,
                                                           int32_t* __restrict__ idx, float* __restrict__ prob,
                                                           int32_t* __restrict__ load) {
  extern __shared__ __align__(16) uint32_t keys_all[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int32_t* hist = reinterpret_cast<int32_t*>(keys_all + warps * 32 * VL);
  uint32_t* keys = keys_all + warp * 32 * VL;
  const int n = p.n, e0 = lane * VL;
  if (load != nullptr) {
    for (int e = threadIdx.x; e < n; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const bool sig = p.score == MOE_SCORE_SIGMOID;
  // scores of all experts are needed for a bias only; sums of group scores
  // without one are made from the logits that the best keys are
  const bool sums = p.G > 1 && p.gtop > 1;
  const int gs = p.gs;
  const bool runs = p.seg_log >= 0;
  for (int t = blockIdx.x * warps + warp; t < T; t += gridDim.x * warps) {
    int mine = -1;  // the lane's chosen expert (lane j: the j-th)
    Soft sm{0.0f, 1.0f};
    if (mask == nullptr || __ldg(mask + t) != 0) {
      float x[VL];
      uint32_t key[VL];
      load_row<VL, BF16>(logits, t, n, lane, p.vec != 0, x);
      if (!sig && (bias != nullptr || sums || !p.renorm)) sm = softmax_of<VL>(x);
      // the key of a group sum: the score behind a key that is a logit
      auto group_key = [&](uint32_t k) {
        if (bias != nullptr || !sums || k <= KEY_NEG_INF) return k;
        const float f = key_value(k);
        return ordered_key(sig ? sigmoid(f) : soft_score(sm, f));
      };
      if (bias != nullptr) {
        float b[VL];
        load_row<VL, false>(bias, 0, n, lane, p.vec_bias != 0, b);  // -inf past n, as the logits
        if (sig) {
#pragma unroll
          for (int i = 0; i < VL; ++i) key[i] = ordered_key(x[i] == -INFINITY ? x[i] : sigmoid(x[i]) + b[i]);
        } else {
#pragma unroll
          for (int i = 0; i < VL; ++i) key[i] = ordered_key(x[i] == -INFINITY ? x[i] : soft_score(sm, x[i]) + b[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VL; ++i) key[i] = ordered_key(x[i]);
      }
      // the topk_group best groups, lane g holding the score of group g
      auto kept_groups = [&](float score) {
        uint32_t gk = lane < p.G ? max(ordered_key(score), 1u) : 0u;
        unsigned kept = 0u;
        for (int r = 0; r < p.keep; ++r) {
          const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, gk);
          const unsigned who = __ballot_sync(0xFFFFFFFFu, gk == m);
          const unsigned best = who & (0u - who);  // the lowest index among equals
          kept |= best;
          if ((best >> lane) & 1u) gk = 0u;
        }
        return kept;
      };
      if (p.G > 1 && !runs) {
        float score = -INFINITY;
        for (int g = 0; g < p.G; ++g) {
          const int lo = g * gs, hi = lo + gs;
          uint32_t b1 = 0, b2 = 0;  // the lane's best two of the group
#pragma unroll
          for (int i = 0; i < VL; ++i) {
            if (e0 + i >= lo && e0 + i < hi) {
              b2 = max(b2, min(b1, key[i]));
              b1 = max(b1, key[i]);
            }
          }
          const uint32_t m1 = __reduce_max_sync(0xFFFFFFFFu, b1);
          float sc = key_value(group_key(m1));
          if (p.gtop > 1 && gs > 1) {
            const unsigned who = __ballot_sync(0xFFFFFFFFu, b1 == m1);
            sc += key_value(group_key(__reduce_max_sync(0xFFFFFFFFu, lane == __ffs(who) - 1 ? b2 : b1)));
          }
          if (lane == g) score = sc;
        }
        const unsigned kept = kept_groups(score);
        int g = e0 / gs, left = gs - (e0 - g * gs);  // the group of expert e0 + i, and what is left of it
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          if (e0 + i < n && !((kept >> g) & 1u)) key[i] = 0u;
          if (--left == 0) {
            ++g;
            left = gs;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < VL; ++i) keys[e0 + i] = key[i];
      sort_desc<VL>(key);
      if (p.G > 1 && runs) {
        uint32_t g1 = key[0], g2 = VL > 1 ? key[1 % VL] : 0u;
        for (int d = 1; d < (1 << p.seg_log); d <<= 1) {
          const uint32_t o1 = __shfl_xor_sync(0xFFFFFFFFu, g1, d), o2 = __shfl_xor_sync(0xFFFFFFFFu, g2, d);
          g2 = max(max(g2, o2), min(g1, o1));
          g1 = max(g1, o1);
        }
        float score = key_value(group_key(g1));
        if (p.gtop > 1 && gs > 1) score += key_value(group_key(g2));
        const unsigned kept = kept_groups(__shfl_sync(0xFFFFFFFFu, score, (lane << p.seg_log) & 31));
        if (!((kept >> (lane >> p.seg_log)) & 1u)) key[0] = 0u;  // (nothing below it is looked at)
      }
      // the choice: lane j keeps the j-th key and the lane it came from
      uint32_t my_key = 0u;
      int my_src = -1, j = 0;
      for (; j < p.k; ++j) {
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, key[0]);
        if (m <= KEY_NEG_INF) break;
        const int src = __ffs(__ballot_sync(0xFFFFFFFFu, key[0] == m)) - 1;
        if (lane == j) {
          my_key = m;
          my_src = src;
        }
        if (lane == src) {
#pragma unroll
          for (int i = 0; i + 1 < VL; ++i) key[i] = key[i + 1];
          key[VL - 1] = 0u;
        }
      }
      // its index: the c-th of the source's experts with that key, c the
      // number of earlier choices of the same key from the same lane
      const unsigned same = __match_any_sync(0xFFFFFFFFu, my_key) & __match_any_sync(0xFFFFFFFFu, my_src);
      int c = __popc(same & ((1u << lane) - 1u));
      if (lane < j) {
        const uint32_t* src = keys + my_src * VL;
#pragma unroll
        for (int i = 0; i < VL; ++i)
          if (src[i] == my_key && c-- == 0) mine = my_src * VL + i;
      }
      __syncwarp();  // the keys have been read
    }
    float w = 0.0f;
    const float xe = mine >= 0 ? load_logit<BF16>(logits, (size_t)t * n + mine) : -INFINITY;
    if (p.renorm && !sig) {
      // the softmax over the chosen logits
      const float m = warp_max(xe);
      const float ex = mine >= 0 ? expf(xe - m) : 0.0f;
      const float sum = warp_sum(ex);
      if (mine >= 0) w = ex / sum;
    } else {
      if (mine >= 0) w = sig ? sigmoid(xe) : soft_score(sm, xe);
      if (p.renorm) w = w / (warp_sum(w) + 1e-20f);
    }
    if (lane < p.k) {
      idx[(size_t)t * p.k + lane] = mine;
      prob[(size_t)t * p.k + lane] = w * p.scale;
      if (load != nullptr && mine >= 0) atomicAdd(&hist[mine], 1);
    }
  }
  if (load != nullptr) flush_load(hist, n, load);
}

// The same choice for few experts without groups (n <= LPT VL, k <= LPT):
// LPT lanes per token, 32 / LPT tokens per warp, so that no lane idles and a
// round serves all of them: with 64 experts on 8 lanes a warp spends about
// the instructions on four tokens that it spent on one.  The reductions are
// shuffles inside the token's lanes.
template <int LPT, int VL, bool BF16>
__global__ void __launch_bounds__(32 * max_warps<VL>()) k_router_small(const void* __restrict__ logits,
                                                                       const float* __restrict__ bias,
                                                                       const uint8_t* __restrict__ mask, int T,
                                                                       const Params p, int32_t* __restrict__ idx,
                                                                       float* __restrict__ prob,
                                                                       int32_t* __restrict__ load) {
  constexpr int TPW = 32 / LPT;
  extern __shared__ __align__(16) uint32_t keys_all[];  // [warps][32 VL] keys, [warps][32] choices (two words), hist
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  uint32_t* keys = keys_all + warp * 32 * VL;
  uint2* picks = reinterpret_cast<uint2*>(keys_all + warps * 32 * VL) + warp * 32;
  int32_t* hist = reinterpret_cast<int32_t*>(keys_all + warps * (32 * VL + 64));
  const int n = p.n, sub = lane & (LPT - 1), first = lane - sub;  // the token's first lane
  const unsigned seg = (LPT == 32 ? 0xFFFFFFFFu : (1u << LPT) - 1u) << first;
  if (load != nullptr) {
    for (int e = threadIdx.x; e < n; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const bool sig = p.score == MOE_SCORE_SIGMOID;
  auto seg_sum = [&](float v) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
  };
  auto seg_max = [&](float v) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
  };
  for (int t0 = (blockIdx.x * warps + warp) * TPW; t0 < T; t0 += gridDim.x * warps * TPW) {
    const int t = t0 + lane / LPT;
    const bool on = t < T && (mask == nullptr || __ldg(mask + t) != 0);
    float x[VL];
    uint32_t key[VL];
    if (on) {
      load_row<VL, BF16>(logits, t, n, sub, p.vec != 0, x);
    } else {
#pragma unroll
      for (int i = 0; i < VL; ++i) x[i] = -INFINITY;
    }
    Soft sm{0.0f, 1.0f};
    if (!sig && (bias != nullptr || !p.renorm)) {
      float m = x[0];
#pragma unroll
      for (int i = 1; i < VL; ++i) m = fmaxf(m, x[i]);
      m = seg_max(m);
      if (m == -INFINITY) m = 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VL; ++i) sum += expf(x[i] - m);
      sum = seg_sum(sum);
      sm = {m, sum != sum ? sum : fmaxf(sum, 1e-38f)};
    }
    if (bias != nullptr) {
      float b[VL];
      load_row<VL, false>(bias, 0, n, sub, p.vec_bias != 0, b);
#pragma unroll
      for (int i = 0; i < VL; ++i)
        key[i] = ordered_key(x[i] == -INFINITY ? x[i] : (sig ? sigmoid(x[i]) : soft_score(sm, x[i])) + b[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VL; ++i) key[i] = ordered_key(x[i]);
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) keys[lane * VL + i] = key[i];
    sort_desc<VL>(key);
    uint32_t last = 0u;
    int again = 0, chosen = 0;  // how often this lane's last winning key has won; choices of the token
    for (int j = 0; j < p.k; ++j) {
      uint32_t m = key[0];
#pragma unroll
      for (int d = LPT / 2; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      const bool got = m > KEY_NEG_INF;
      const unsigned who = __ballot_sync(0xFFFFFFFFu, got && key[0] == m);
      if (who == 0u) break;  // no token of the warp finds another expert
      chosen += got ? 1 : 0;
      if (got && lane == __ffs(who & seg) - 1) {
        again = m == last ? again + 1 : 0;
        last = m;
        picks[first + j] = make_uint2(m, (uint32_t)lane | ((uint32_t)again << 8));
#pragma unroll
        for (int i = 0; i + 1 < VL; ++i) key[i] = key[i + 1];
        key[VL - 1] = 0u;
      }
    }
    __syncwarp();
    // lane `sub` of the token settles its sub-th choice: the c-th of the source lane's experts with that key
    int mine = -1;
    if (sub < chosen) {
      const uint2 pk = picks[first + sub];
      const uint32_t* src = keys + (pk.y & 0xFFu) * VL;
      int c = (int)(pk.y >> 8);
#pragma unroll
      for (int i = 0; i < VL; ++i)
        if (src[i] == pk.x && c-- == 0) mine = (int)((pk.y & (LPT - 1)) * VL) + i;
    }
    __syncwarp();  // keys and picks have been read
    float w = 0.0f;
    const float xe = mine >= 0 ? load_logit<BF16>(logits, (size_t)t * n + mine) : -INFINITY;
    if (p.renorm && !sig) {
      const float m = seg_max(xe);
      const float ex = mine >= 0 ? expf(xe - m) : 0.0f;
      const float sum = seg_sum(ex);
      if (mine >= 0) w = ex / sum;
    } else {
      if (mine >= 0) w = sig ? sigmoid(xe) : soft_score(sm, xe);
      if (p.renorm) w = w / (seg_sum(w) + 1e-20f);
    }
    if (t < T && sub < p.k) {
      idx[(size_t)t * p.k + sub] = mine;
      prob[(size_t)t * p.k + sub] = w * p.scale;
      if (load != nullptr && mine >= 0) atomicAdd(&hist[mine], 1);
    }
  }
  if (load != nullptr) flush_load(hist, n, load);
}

template <bool BF16>
__device__ __forceinline__ void store_logit(void* p, size_t i, float v) {
  if (BF16)
    static_cast<uint16_t*>(p)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  else
    static_cast<float*>(p)[i] = v;
}
// The lane's VL values of row t (see load_row).
template <int VL, bool BF16>
__device__ __forceinline__ void store_row(void* p, size_t t, int n, int lane, bool vec, const float* v) {
  const int e0 = lane * VL;
  if (!vec || VL == 1) {
#pragma unroll
    for (int i = 0; i < VL; ++i)
      if (e0 + i < n) store_logit<BF16>(p, t * n + e0 + i, v[i]);
    return;
  }
  if (e0 >= n) return;
  constexpr int W = BF16 ? VL / 2 : VL;  // 32-bit words
  uint32_t w[W > 0 ? W : 1];
#pragma unroll
  for (int i = 0; i < W; ++i)
    w[i] = BF16 ? pack_bf16x2(v[(2 * i) % VL], v[(2 * i + 1) % VL]) : __float_as_uint(v[i % VL]);
  uint32_t* d = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + (t * n + e0) * (BF16 ? 2 : 4));
  if (W >= 4) {
#pragma unroll
    for (int c = 0; c < W / 4; ++c)
      reinterpret_cast<uint4*>(d)[c] =
          make_uint4(w[(4 * c) % W], w[(4 * c + 1) % W], w[(4 * c + 2) % W], w[(4 * c + 3) % W]);
  } else if (W == 2) {
    *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1 % W]);
  } else {
    *d = w[0];
  }
}

// Backward, one warp per token; lane j < k holds the j-th chosen expert with
// g_j = scale * dprob_j.  With w the weights before the factor:
//   softmax, renormalised:   dx_j = w_j (g_j - sum g w)            (chosen only)
//   softmax:                 dx_e = [e chosen] g s_e - s_e sum_j g_j s_j
//   sigmoid, renormalised:   dx_j = (g_j - sum g w) / D * s_j (1 - s_j),  D = sum s + 1e-20
//   sigmoid:                 dx_j = g_j s_j (1 - s_j)
// Experts without a gradient get 0; only the plain softmax reads every logit.
// The row is written whole, then lane j writes its expert's element over it.
template <int VL, bool BF16>
__global__ void __launch_bounds__(32 * max_warps<VL>()) k_router_bwd(const void* __restrict__ logits,
                                                           const int32_t* __restrict__ idx,
                                                           const float* __restrict__ dprob, int T, const Params p,
                                                           void* __restrict__ dlogits) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int n = p.n;
  for (int t = blockIdx.x * warps + (threadIdx.x >> 5); t < T; t += gridDim.x * warps) {
    int e = -1;
    float g = 0.0f, xe = -INFINITY;
    if (lane < p.k) {
      e = __ldg(idx + (size_t)t * p.k + lane);
      if (e < 0 || e >= n) e = -1;
      if (e >= 0) {
        g = p.scale * __ldg(dprob + (size_t)t * p.k + lane);
        xe = load_logit<BF16>(logits, (size_t)t * n + e);
      }
    }
    float out[VL];
#pragma unroll
    for (int i = 0; i < VL; ++i) out[i] = 0.0f;
    float d;  // gradient of the lane's chosen logit
    if (p.score == MOE_SCORE_SIGMOID) {
      const float s = e >= 0 ? sigmoid(xe) : 0.0f;
      const float s1 = sigmoid(-xe);  // 1 - s without the cancellation
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
    } else if (!__any_sync(0xFFFFFFFFu, e >= 0)) {
      d = 0.0f;  // a token that chose nothing: its logits (masked, perhaps not finite) are not looked at
    } else {
      load_row<VL, BF16>(logits, t, n, lane, p.vec != 0, out);
      const Soft sm = softmax_of<VL>(out);
      const float se = e >= 0 ? soft_score(sm, xe) : 0.0f;
      const float in = warp_sum(g * se);
      d = se * (g - in);
      const float scale = -in / sm.d;
#pragma unroll
      for (int i = 0; i < VL; ++i) out[i] = expf(out[i] - sm.m) * scale;
    }
    store_row<VL, BF16>(dlogits, t, n, lane, p.vec != 0, out);
    __syncwarp();  // orders the row's stores before the chosen experts'
    if (e >= 0) store_logit<BF16>(dlogits, (size_t)t * n + e, d);
  }
}

static bool params_ok(const moe_router_params_t* q, int n, int k) {
  return q && (q->score == MOE_SCORE_SOFTMAX || q->score == MOE_SCORE_SIGMOID) && n > 0 && n <= N_MAX && k > 0 &&
         k <= K_MAX && k <= n && q->n_group >= 1 && q->n_group <= G_MAX && n % q->n_group == 0 &&
         q->topk_group >= 1 && q->topk_group <= q->n_group && (q->group_top == 1 || q->group_top == 2) &&
         k <= n / q->n_group * q->topk_group && q->scale == q->scale;
}

// CTAs and warps per CTA.  Few tokens fit one CTA, which then holds every
// count of the load and needs no cleared buffer and no atomics; otherwise
// `ctas_per_sm` CTAs per SM of as many warps as there is work for: every CTA
// adds its n counts to the same n addresses, and 2432 small CTAs took 12 us
// longer over that than 304 large ones (32768 tokens, 64 experts).
struct Grid {
  int ctas, warps;
};
// 16 tokens of 256 experts take 3.9 us in one CTA against 4.7 spread out, 32
// take 5.1 against 4.7.
static Grid grid_of(int T, int max_warps, int ctas_per_sm) {
  if (T <= 16) return {1, T < max_warps ? T : max_warps};
  const int most = sm_count() * ctas_per_sm;
  if (most <= 0) return {0, 0};
  int w = (T + most - 1) / most;
  if (w > max_warps) w = max_warps;
  const int need = (T + w - 1) / w;
  return {need < most ? need : most, w};
}

// Experts per lane: the power of two that covers n / 32; rows are read in
// vectors where every row starts on a vector's boundary (n a multiple of the
// lane's experts, aligned bases).
static Params make_params(const moe_router_params_t* q, int n, int k, int vl, int bf16, const void* a, const void* b,
                          const float* bias) {
  auto fits = [&](int es, uintptr_t bases) {
    const int unit = vl * es < 16 ? vl * es : 16;
    return n % vl == 0 && ((size_t)n * es) % unit == 0 && (bases & (unit - 1)) == 0;
  };
  Params p{n, k, q->score, q->renorm ? 1 : 0, q->n_group, q->topk_group, q->group_top, q->scale};
  p.gs = n / q->n_group;
  p.seg_log = -1;
  if (p.gs % vl == 0 && (p.gs / vl & (p.gs / vl - 1)) == 0)
    for (p.seg_log = 0; (1 << p.seg_log) < p.gs / vl;) ++p.seg_log;
  p.vec = fits(bf16 ? 2 : 4, reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b));
  p.vec_bias = fits(4, reinterpret_cast<uintptr_t>(bias));
  return p;
}
template <class F>
static void dispatch(const moe_router_params_t* q, int n, int k, int bf16, const void* a, const void* b,
                     const float* bias, F&& f) {
  int vl = 1;
  while (32 * vl < n) vl *= 2;
  const Params p = make_params(q, n, k, vl, bf16, a, b, bias);
  auto typed = [&](auto v) {
    if (bf16)
      f(v, std::true_type{}, p);
    else
      f(v, std::false_type{}, p);
  };
  if (vl == 1)
    typed(std::integral_constant<int, 1>{});
  else if (vl == 2)
    typed(std::integral_constant<int, 2>{});
  else if (vl == 4)
    typed(std::integral_constant<int, 4>{});
  else if (vl == 8)
    typed(std::integral_constant<int, 8>{});
  else if (vl == 16)
    typed(std::integral_constant<int, 16>{});
  else
    typed(std::integral_constant<int, 32>{});
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
  // Few experts without groups: several tokens per warp (lanes per token and
  // experts per lane by n).  64 experts: 6.8 us with one token per warp
  // against 4.9 at 8192 tokens, 16.7 against 9.0 at 32768; below 3000 tokens
  // one per warp would be 0.1 to 0.5 us faster, and is not taken there, because
  // a token's weights would then depend (in their last bit) on the batch's size.
  const int lpt = n <= 64 ? 8 : 16, small_vl = n <= 32 ? 4 : 8;
  const bool small = params->n_group == 1 && n <= 128 && k <= lpt;
  const int units = small ? (T + 32 / lpt - 1) / (32 / lpt) : T;  // warps' worth of work
  const Grid g = T > 0 ? (n <= 256   ? grid_of(units, max_warps<8>(), 1)
                          : n <= 512 ? grid_of(units, max_warps<16>(), 2)
                                     : grid_of(units, max_warps<32>(), 2))
                       : Grid{0, 0};
  if (T > 0 && g.ctas <= 0) return MOE_ERR_CUDA;
  if (T == 0) {
    if (load && cudaMemsetAsync(load, 0, (size_t)n * sizeof(int32_t), st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const bool clear = load && g.ctas > 1;
  if (clear) {
    k_router_clear<<<1, 256, 0, st>>>(load, n);
    count_launch();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.ctas);
  cfg.blockDim = dim3(32 * g.warps);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = clear ? 1 : 0;
  if (small) {
    const Params p = make_params(params, n, k, small_vl, logits_bf16, logits, nullptr, bias);
    cfg.dynamicSmemBytes = (size_t)g.warps * (32 * small_vl + 64) * 4 + (load ? (size_t)n * 4 : 0);  // < 48 KB
    auto run = [&](auto kernel) {
      cudaLaunchKernelEx(&cfg, kernel, logits, bias, token_mask, T, p, topk_idx, topk_prob, load);
    };
    if (n <= 32)
      logits_bf16 ? run(k_router_small<8, 4, true>) : run(k_router_small<8, 4, false>);
    else if (n <= 64)
      logits_bf16 ? run(k_router_small<8, 8, true>) : run(k_router_small<8, 8, false>);
    else
      logits_bf16 ? run(k_router_small<16, 8, true>) : run(k_router_small<16, 8, false>);
    count_launch();
    return launch_status();
  }
  dispatch(params, n, k, logits_bf16, logits, nullptr, bias, [&](auto vl, auto bf16, const Params& p) {
    constexpr int VL = decltype(vl)::value;
    cfg.dynamicSmemBytes = (size_t)g.warps * 32 * VL * 4 + (load ? (size_t)n * 4 : 0);  // at most 36 KB
    cudaLaunchKernelEx(&cfg, k_router_fwd<VL, decltype(bf16)::value>, logits, bias, token_mask, T, p, topk_idx,
                       topk_prob, load);
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
  const Grid g = grid_of(T, 8, 8);
  if (g.ctas <= 0) return MOE_ERR_CUDA;
  dispatch(params, n, k, logits_bf16, logits, dlogits, nullptr, [&](auto vl, auto bf16, const Params& p) {
    k_router_bwd<decltype(vl)::value, decltype(bf16)::value><<<g.ctas, 32 * g.warps, 0, as_stream(stream)>>>(
        logits, topk_idx, dprob, T, p, dlogits);
  });
  count_launch();
  return launch_status();
}
