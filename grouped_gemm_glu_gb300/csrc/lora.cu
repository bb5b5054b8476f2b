// Low-rank adapters of many requests beside a projection that they share.
//
//   h_t = bf16(s_a P_a x_t),  y_t = bf16(base_t + Q_a^T h_t)   for row t with
//   adapter a (P [G][r][K], Q [G][r][N]; rows without one: h = 0, y = base)
//
// The forward has P = A, Q = B.  The backward is the same pair with the roles
// turned (u = bf16(s_a B_a dy), dx = base + A_a^T u), and the adapters'
// gradients are sums over an adapter's rows, dA_a = sum u x^T, dB_a = sum h dy^T.
// h and u are rounded to bf16 because they are tensor-core operands of the
// products behind them; everything else is fp32 until the outputs' rounding.
//
// Memory bound: with r of 8 to 128 each element of x, base and y takes 2 r
// operations.  Three kernels on tcgen05, all over rows grouped by adapter:
//   k_shrink  D[128 rows][r] = X P^T, contracted over K
//   k_expand  D[128 rows][128 columns] = H Q, contracted over r, plus base
//   k_wgrad   D[128 columns][r] = X^T U, contracted over an adapter's rows
// A first kernel (k_group) sorts the row indexes by adapter, stably, and cuts
// each adapter's rows into tiles of 128; the rows themselves stay where they
// are and are gathered by 16-byte asynchronous copies straight into the
// swizzled operand layout, so that any order of rows takes the same path, no
// tile mixes adapters and no work is done for absent ones.
// k_shrink and k_wgrad produce little from much: the CTAs of a cluster share
// a tile's contraction and add their sums through distributed shared memory,
// always in the same order, so equal inputs give equal bits.
// Few rows (decoding) take k_rows instead: one cluster per row, one launch.
#include "common.cuh"
#include "host_common.h"

namespace moeglu {
namespace lora {

constexpr int TILE = 128;      // rows of one adapter per tile
constexpr int MAX_R = 128;
constexpr int KB = 64;         // contraction per stage (128-byte operand rows)
constexpr int LOADERS = 128;   // threads that copy
constexpr int THREADS = 160;   // + the MMA warp

struct Tile {
  int adapter, start, count, pad;
};
// Workspace: the rows by adapter, each adapter's first place, the tiles.
struct Plan {
  int* n_tiles;
  int* first;  // [G + 2]: adapters, then the rows without one
  Tile* tiles;
  int* rows;   // [T]
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;  // (0: the 16 bytes become zero)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 16-byte piece c of 128-byte row `row` of a tile in the 128-byte swizzle
__device__ __forceinline__ uint32_t piece(uint32_t tile, int row, int c) {
  return tile + row * 128 + ((c ^ (row & 7)) << 4);
}
// Operand tile with the contraction across its 128-byte rows (64 elements of
// the kept dimension per row): `block` bytes between blocks of 64 of them.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr, uint32_t block) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
constexpr uint32_t A_MN = 1u << 15, B_MN = 1u << 16;  // instruction descriptor: that operand's layout

__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}

// ---------------------------------------------------------------------------
// Grouping: one CTA; warp w counts and places its stretch of rows
// ---------------------------------------------------------------------------
constexpr int GROUP_THREADS = 1024, GROUP_SMEM = 128 * 1024, MAX_G = GROUP_SMEM / 4 - 1;

__global__ void __launch_bounds__(GROUP_THREADS) k_group(const int32_t* __restrict__ idx, int T, int G, int warps, Plan p) {
  launch_dependents();
  extern __shared__ int hist[];  // [warps][G + 1]
  __shared__ int part[2][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, groups = G + 1;
  for (int i = tid; i < warps * groups; i += GROUP_THREADS) hist[i] = 0;
  __syncthreads();
  const int per = ((T + warps - 1) / warps + 31) & ~31;
  const int lo = warp * per, hi = warp < warps ? min(T, lo + per) : lo;
  int* mine = hist + warp * groups;
  auto group_of = [&](int row) {
    const int a = idx[row];
    return (unsigned)a < (unsigned)G ? a : G;
  };
  for (int b = lo; b < hi; b += 32) {
    const bool ok = b + lane < hi;
    const uint32_t act = __ballot_sync(0xFFFFFFFFu, ok);
    if (ok) {
      const int a = group_of(b + lane);
      const uint32_t same = __match_any_sync(act, a);
      if ((same & ((1u << lane) - 1)) == 0) mine[a] += __popc(same);
    }
    __syncwarp();
  }
  __syncthreads();
  // places: exclusive sums over the groups (rows, tiles), 1024 groups at a time
  int rows0 = 0, tiles0 = 0;
  for (int g0 = 0; g0 < groups; g0 += GROUP_THREADS) {
    const int g = g0 + tid;
    int n = 0;
    if (g < groups)
      for (int w = 0; w < warps; ++w) {
        const int k = hist[w * groups + g];
        hist[w * groups + g] = n;
        n += k;
      }
    const int tiles = (n + TILE - 1) / TILE;
    int rs = n, ts = tiles;
    for (int d = 1; d < 32; d <<= 1) {
      const int r = __shfl_up_sync(0xFFFFFFFFu, rs, d), t = __shfl_up_sync(0xFFFFFFFFu, ts, d);
      if (lane >= d) rs += r, ts += t;
    }
    if (lane == 31) part[0][warp] = rs, part[1][warp] = ts;
    __syncthreads();
    if (warp == 0) {
      int r = part[0][lane], t = part[1][lane];
      for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(0xFFFFFFFFu, r, d), b = __shfl_up_sync(0xFFFFFFFFu, t, d);
        if (lane >= d) r += a, t += b;
      }
      part[0][lane] = r, part[1][lane] = t;
    }
    __syncthreads();
    const int r0 = rows0 + (warp ? part[0][warp - 1] : 0) + rs - n, t0 = tiles0 + (warp ? part[1][warp - 1] : 0) + ts - tiles;
    if (g < groups) {
      for (int w = 0; w < warps; ++w) hist[w * groups + g] += r0;
      p.first[g] = r0;
      for (int i = 0; i < tiles; ++i) p.tiles[t0 + i] = {g < G ? g : -1, r0 + i * TILE, min(TILE, n - i * TILE), 0};
    }
    rows0 += part[0][31];
    tiles0 += part[1][31];
    __syncthreads();
  }
  if (tid == 0) {
    p.first[groups] = rows0;
    *p.n_tiles = tiles0;
  }
  for (int b = lo; b < hi; b += 32) {
    const bool ok = b + lane < hi;
    const uint32_t act = __ballot_sync(0xFFFFFFFFu, ok);
    int a = 0, at = 0;
    uint32_t same = 0;
    if (ok) {
      a = group_of(b + lane);
      same = __match_any_sync(act, a);
      at = mine[a];
      p.rows[at + __popc(same & ((1u << lane) - 1))] = b + lane;
    }
    __syncwarp();
    if (ok && (same & ((1u << lane) - 1)) == 0) mine[a] = at + __popc(same);
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// k_shrink and k_wgrad: the common pipeline
// ---------------------------------------------------------------------------
// RB: the rank's operand rows (64 or 128) that a stage has room for.
template <int RB>
struct Ring {
  static constexpr int STAGES = RB == 64 ? 4 : 3;
  static constexpr int A_BYTES = TILE * 128, B_BYTES = RB * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int BYTES = STAGES * STAGE + 1024;
};
struct Bars {
  uint64_t full[4], empty[4], done;
  int abort;
  uint32_t tmem;
};

// Columns of tensor memory for an accumulator of rp columns (a power of two, at least 32).
__device__ __forceinline__ uint32_t tmem_cols(int rp) { return rp <= 32 ? 32 : rp <= 64 ? 64 : 128; }

// The loaders' side: fill(i, stage address) issues the copies of step i.
template <int STAGES, class Fill>
__device__ __forceinline__ void produce(Bars& b, uint32_t ring, int stage_bytes, int steps, const WaitGuard& g, Fill fill) {
  constexpr int LAG = STAGES - 1;
  int i = 0;
  for (; i < steps; ++i) {
    const int st = i % STAGES;
    if (i >= STAGES && !mbar_wait(&b.empty[st], (i / STAGES - 1) & 1, g)) break;
    fill(i, ring + st * stage_bytes);
    cp_commit();
    if (i >= LAG) {
      cp_wait<LAG>();
      fence_async_shared();
      mbar_arrive(&b.full[(i - LAG) % STAGES]);
    }
  }
  cp_wait<0>();
  fence_async_shared();
  if (i == steps)
    for (int k = max(0, steps - LAG); k < steps; ++k) mbar_arrive(&b.full[k % STAGES]);
}

// Adds the cluster's accumulators [128][rp] (partial: this CTA's copy, as
// float4 [rp/4][128]) and hands each sum of four neighbouring rank elements to
// put(lane of the tile, first rank element, sum).
template <class Put>
__device__ __forceinline__ void cluster_reduce(uint32_t partial, int rp, Put put) {
  const uint32_t size = cluster_size(), rank = cluster_ctarank();
  const int lanes = TILE / size;
  for (int i = threadIdx.x; i < lanes * (rp / 4); i += LOADERS) {
    const int l = rank * lanes + i % lanes, q = i / lanes;
    const uint32_t at = partial + (q * TILE + l) * 16;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (uint32_t c = 0; c < size; ++c) {
      const float4 v = ld_cluster(mapa_shared(at, c));
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    put(l, q * 4, s);
  }
}

// The accumulator to shared memory, by the four loader warps.
__device__ __forceinline__ void spill(uint32_t tmem, unsigned char* partial, int rp, bool any) {
  const int lane = threadIdx.x;  // the accumulator's lane of this thread (warp w holds 32 w ..)
  for (int c = 0; c < rp; c += 32) {
    float v[32];
    if (any) {
      tmem_ld32(tmem + ((uint32_t)(threadIdx.x & 96) << 16) + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 4 * i < rp)
        *reinterpret_cast<float4*>(partial + (((c >> 2) + i) * TILE + lane) * 16) =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

// The dynamic shared memory from its first multiple of 1024 bytes on (the
// swizzle's period; 1024 bytes more are asked for).
__device__ __forceinline__ unsigned char* aligned_smem(unsigned char* p) { return p + ((0u - smem_u32(p)) & 1023u); }

template <int RB>
__device__ __forceinline__ void begin(Bars& b, int rp) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < Ring<RB>::STAGES; ++i) {
      mbar_init(&b.full[i], LOADERS);
      mbar_init(&b.empty[i], 1);
    }
    mbar_init(&b.done, 1);
    b.abort = 0;
    fence_barrier_init();
  }
  if (threadIdx.x >= LOADERS) {
    tmem_alloc(&b.tmem, tmem_cols(rp));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

// The MMA warp's side; step(i, stage address, accumulate) issues step i.
template <int STAGES, class Step>
__device__ __forceinline__ void consume(Bars& b, uint32_t ring, int stage_bytes, int steps, const WaitGuard& g, Step step) {
  if ((threadIdx.x & 31) == 0) {
    for (int i = 0; i < steps; ++i) {
      const int st = i % STAGES;
      if (!mbar_wait(&b.full[st], (i / STAGES) & 1, g)) break;
      tc_fence_after();
      step(i, ring + st * stage_bytes);
      tc_commit(&b.empty[st]);
    }
    tc_commit(&b.done);
  }
  __syncwarp();
}

__device__ __forceinline__ uint2 pack4(float4 s, float f) {
  return make_uint2(pack_bf16x2(s.x * f, s.y * f), pack_bf16x2(s.z * f, s.w * f));
}

// Cluster (tile): h rows of one tile.  X [T][K], P [G][r][K].
template <int RB>
__global__ void __launch_bounds__(THREADS) k_shrink(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ P,
                                                    const float* __restrict__ scale, int K, int r, int rp, Plan plan,
                                                    __nv_bfloat16* __restrict__ h, uint64_t limit_ns, int32_t* status) {
  extern __shared__ unsigned char smem_[];
  unsigned char* smem = aligned_smem(smem_);
  __shared__ Bars b;
  __shared__ int rows[TILE];
  const uint32_t size = cluster_size(), rank = cluster_ctarank();
  const int tile = blockIdx.x / size;
  launch_dependents();
  wait_for_primary();
  if (tile >= *plan.n_tiles) return;  // (the whole cluster)
  const Tile t = plan.tiles[tile];
  if (threadIdx.x < TILE) rows[threadIdx.x] = threadIdx.x < t.count ? plan.rows[t.start + threadIdx.x] : 0;
  if (t.adapter < 0) {  // rows without an adapter
    __syncthreads();
    for (int i = threadIdx.x + rank * THREADS; i < t.count * (r / 8); i += THREADS * size)
      *reinterpret_cast<uint4*>(h + (size_t)rows[i / (r / 8)] * r + (i % (r / 8)) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  begin<RB>(b, rp);
  const WaitGuard g{&b.abort, status, limit_ns};
  const uint32_t ring = smem_u32(smem);
  const int blocks = (K + KB - 1) / KB;
  const int k0 = (int)((int64_t)blocks * rank / size), steps = (int)((int64_t)blocks * (rank + 1) / size) - k0;
  using R = Ring<RB>;
  if (threadIdx.x < LOADERS) {
    const int c = threadIdx.x & 7, row0 = threadIdx.x >> 3;
    const __nv_bfloat16* src[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) src[i] = X + (size_t)rows[row0 + 16 * i] * K + c * 8;
    const __nv_bfloat16* p = P + (size_t)t.adapter * r * K + c * 8;
    produce<R::STAGES>(b, ring, R::STAGE, steps, g, [&](int i, uint32_t at) {
      const int k = (k0 + i) * KB;
      const bool in = k + c * 8 < K;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (row0 + 16 * j < t.count) cp16(piece(at, row0 + 16 * j, c), in ? src[j] + k : X, in);
      for (int j = row0; j < r; j += 16) cp16(piece(at + R::A_BYTES, j, c), in ? p + (size_t)j * K + k : P, in);
    });
  } else {
    const uint32_t idesc = idesc_bf16_f32(TILE, rp);
    consume<R::STAGES>(b, ring, R::STAGE, steps, g, [&](int i, uint32_t at) {
#pragma unroll
      for (int k = 0; k < KB / 16; ++k)
        umma_bf16(b.tmem, sdesc_kmajor_sw128(at + 32 * k), sdesc_kmajor_sw128(at + R::A_BYTES + 32 * k), idesc, i + k > 0);
    });
  }
  mbar_wait(&b.done, 0, g);
  tc_fence_after();
  __syncthreads();  // (every copy has landed and every MMA has read: the ring is free)
  if (threadIdx.x < LOADERS) spill(b.tmem, smem, rp, steps > 0);
  tc_fence_before();
  cluster_sync();
  if (threadIdx.x < LOADERS && !b.abort) {
    const float s = scale[t.adapter];
    cluster_reduce(ring, rp, [&](int l, int q, float4 v) {
      if (l < t.count && q < r) *reinterpret_cast<uint2*>(h + (size_t)rows[l] * r + q) = pack4(v, s);
    });
  }
  cluster_sync();  // (the other CTAs have read this one's sums)
  if (threadIdx.x >= LOADERS) {
    tc_fence_after();
    tmem_dealloc(b.tmem, tmem_cols(rp));
  }
}

// Cluster (adapter, 128 columns of X [T][C]): dP [G][r][C] = U^T X over the
// adapter's rows, U [T][r].
template <int RB>
__global__ void __launch_bounds__(THREADS) k_wgrad(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ U,
                                                   int C, int r, int rp, Plan plan, __nv_bfloat16* __restrict__ dP,
                                                   uint64_t limit_ns, int32_t* status) {
  extern __shared__ unsigned char smem_[];
  unsigned char* smem = aligned_smem(smem_);
  __shared__ Bars b;
  const uint32_t size = cluster_size(), rank = cluster_ctarank();
  const int chunks = (C + TILE - 1) / TILE, unit = blockIdx.x / size, adapter = unit / chunks;
  const int c0 = (unit - adapter * chunks) * TILE;
  launch_dependents();
  wait_for_primary();
  const int first = plan.first[adapter], n = plan.first[adapter + 1] - first;
  begin<RB>(b, rp);
  const WaitGuard g{&b.abort, status, limit_ns};
  const uint32_t ring = smem_u32(smem);
  const int blocks = (n + KB - 1) / KB;
  const int k0 = (int)((int64_t)blocks * rank / size), steps = (int)((int64_t)blocks * (rank + 1) / size) - k0;
  using R = Ring<RB>;
  if (threadIdx.x < LOADERS) {
    const int c = threadIdx.x & 15, row0 = threadIdx.x >> 4;
    const bool col = c0 + c * 8 < C;
    const int pieces = rp / 8;
    produce<R::STAGES>(b, ring, R::STAGE, steps, g, [&](int i, uint32_t at) {
      const int base = (k0 + i) * KB;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = row0 + 8 * j;
        const bool in = col && base + row < n;
        const __nv_bfloat16* s = in ? X + (size_t)plan.rows[first + base + row] * C + c0 + c * 8 : X;
        cp16(piece(at + (c >> 3) * (KB * 128), row, c & 7), s, in);
      }
      for (int j = threadIdx.x; j < KB * pieces; j += LOADERS) {
        const int row = j / pieces, q = j - row * pieces;
        const bool in = base + row < n && q * 8 < r;
        const __nv_bfloat16* s = in ? U + (size_t)plan.rows[first + base + row] * r + q * 8 : U;
        cp16(piece(at + R::A_BYTES + (q >> 3) * (KB * 128), row, q & 7), s, in);
      }
    });
  } else {
    const uint32_t idesc = idesc_bf16_f32(TILE, rp) | A_MN | B_MN;
    consume<R::STAGES>(b, ring, R::STAGE, steps, g, [&](int i, uint32_t at) {
#pragma unroll
      for (int k = 0; k < KB / 16; ++k)
        umma_bf16(b.tmem, sdesc_mnmajor_sw128(at + 2048 * k, KB * 128),
                  sdesc_mnmajor_sw128(at + R::A_BYTES + 2048 * k, KB * 128), idesc, i + k > 0);
    });
  }
  mbar_wait(&b.done, 0, g);
  tc_fence_after();
  __syncthreads();
  if (threadIdx.x < LOADERS) spill(b.tmem, smem, rp, steps > 0);
  tc_fence_before();
  cluster_sync();
  if (threadIdx.x < LOADERS && !b.abort) {
    __nv_bfloat16* out = dP + (size_t)adapter * r * C + c0;
    cluster_reduce(ring, rp, [&](int l, int q, float4 v) {
      if (c0 + l >= C) return;
      const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (q + j < r) out[(size_t)(q + j) * C + l] = __float2bfloat16_rn(w[j]);
    });
  }
  cluster_sync();
  if (threadIdx.x >= LOADERS) {
    tc_fence_after();
    tmem_dealloc(b.tmem, tmem_cols(rp));
  }
}

// ---------------------------------------------------------------------------
// k_expand: y = base + h Q, persistent over (tile, 128 columns)
// ---------------------------------------------------------------------------
template <int RB>
struct Wide {
  static constexpr int STAGES = RB == 32 ? 4 : RB == 64 ? 3 : 2;
  static constexpr int BASE = TILE * 256, Q_BYTES = RB * 256, H_BYTES = TILE * 128 * (RB > 64 ? 2 : 1);
  static constexpr int STAGE = BASE + Q_BYTES + H_BYTES, BYTES = STAGES * STAGE + 1024;
};
struct WideBars {
  uint64_t full[4], empty[4], acc_full[2], acc_empty[2];
  int abort;
  uint32_t tmem;
};
constexpr int WIDE_THREADS = 288;  // 4 warps copy, 4 write out, 1 issues the MMAs

template <int RB>
__global__ void __launch_bounds__(WIDE_THREADS) k_expand(const __nv_bfloat16* __restrict__ H,
                                                         const __nv_bfloat16* __restrict__ Q, const __nv_bfloat16* base,
                                                         int N, int r, int rp, Plan plan, __nv_bfloat16* y,
                                                         uint64_t limit_ns, int32_t* status) {
  extern __shared__ unsigned char smem_[];
  unsigned char* smem = aligned_smem(smem_);
  __shared__ WideBars b;
  using R = Wide<RB>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R::STAGES; ++i) {
      mbar_init(&b.full[i], LOADERS);
      mbar_init(&b.empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.acc_full[i], 1);
      mbar_init(&b.acc_empty[i], 4);
    }
    b.abort = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&b.tmem, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();
  wait_for_primary();
  const WaitGuard g{&b.abort, status, limit_ns};
  const uint32_t ring = smem_u32(smem);
  const int chunks = (N + TILE - 1) / TILE, tiles = *plan.n_tiles;
  const int64_t units = (int64_t)tiles * chunks;
  const int n = units > blockIdx.x ? (int)((units - blockIdx.x + gridDim.x - 1) / gridDim.x) : 0;
  // unit i of this CTA: neighbours in time on the GPU are tiles of the same columns
  auto unit = [&](int i, Tile& t, int& c0) {
    const int64_t u = blockIdx.x + (int64_t)i * gridDim.x;
    const int chunk = (int)(u / tiles);
    t = plan.tiles[u - (int64_t)chunk * tiles];
    c0 = chunk * TILE;
  };
  if (warp < 4) {
    constexpr int LAG = R::STAGES - 1;
    const int c = threadIdx.x & 15, row0 = threadIdx.x >> 4;
    const int pieces = rp / 8;
    int i = 0;
    for (; i < n; ++i) {
      const int st = i % R::STAGES;
      const uint32_t at = ring + st * R::STAGE;
      if (i >= R::STAGES && !mbar_wait(&b.empty[st], (i / R::STAGES - 1) & 1, g)) break;
      Tile t;
      int c0;
      unit(i, t, c0);
      const int* rows = plan.rows + t.start;
      const bool col = c0 + c * 8 < N;
      if (t.adapter >= 0) {
        for (int j = threadIdx.x; j < t.count * pieces; j += LOADERS) {
          const int row = j / pieces, q = j - row * pieces;
          const bool in = q * 8 < r;
          cp16(piece(at + R::BASE + R::Q_BYTES + (q >> 3) * (TILE * 128), row, q & 7),
               in ? H + (size_t)rows[row] * r + q * 8 : H, in);
        }
        const __nv_bfloat16* q = Q + (size_t)t.adapter * r * N + c0 + c * 8;
        for (int j = row0; j < rp; j += 8)
          cp16(piece(at + R::BASE + (c >> 3) * (rp * 128), j, c & 7), col && j < r ? q + (size_t)j * N : Q, col && j < r);
      }
      if (base)
        for (int j = row0; j < t.count; j += 8)
          if (col) cp16(piece(at + (c >> 3) * (TILE * 128), j, c & 7), base + (size_t)rows[j] * N + c0 + c * 8, true);
      cp_commit();
      if (i >= LAG) {
        cp_wait<LAG>();
        fence_async_shared();
        mbar_arrive(&b.full[(i - LAG) % R::STAGES]);
      }
    }
    cp_wait<0>();
    fence_async_shared();
    if (i == n)
      for (int k = max(0, n - LAG); k < n; ++k) mbar_arrive(&b.full[k % R::STAGES]);
  } else if (warp == 8) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(TILE, TILE) | B_MN;
      for (int i = 0; i < n; ++i) {
        const int st = i % R::STAGES, acc = i & 1;
        const uint32_t at = ring + st * R::STAGE;
        if (!mbar_wait(&b.full[st], (i / R::STAGES) & 1, g)) break;
        if (i >= 2 && !mbar_wait(&b.acc_empty[acc], (i / 2 - 1) & 1, g)) break;
        tc_fence_after();
        Tile t;
        int c0;
        unit(i, t, c0);
        if (t.adapter >= 0)
          for (int k = 0; k < rp / 16; ++k)
            umma_bf16(b.tmem + acc * TILE,
                      sdesc_kmajor_sw128(at + R::BASE + R::Q_BYTES + (k >> 2) * (TILE * 128) + 32 * (k & 3)),
                      sdesc_mnmajor_sw128(at + R::BASE + 2048 * k, rp * 128), idesc, k > 0);
        tc_commit(&b.acc_full[acc]);
      }
    }
    __syncwarp();
  } else {
    const int w = warp - 4, quad = w;  // (warps 4..7: tensor-memory lanes 32 w ..)
    for (int i = 0; i < n; ++i) {
      const int st = i % R::STAGES, acc = i & 1;
      Tile t;
      int c0;
      unit(i, t, c0);
      const int mine = t.count - 32 * w;  // rows of this warp
      const int row_id = lane < mine ? plan.rows[t.start + 32 * w + lane] : 0;
      if (!mbar_wait(&b.full[st], (i / R::STAGES) & 1, g)) break;
      if (!mbar_wait(&b.acc_full[acc], (i / 2) & 1, g)) break;
      tc_fence_after();
      const uint32_t at = ring + st * R::STAGE;
      unsigned char* stage = smem + st * R::STAGE;
      if (mine > 0) {
        for (int q = 0; q < 4; ++q) {
          float v[32];
          if (t.adapter >= 0) {
            tmem_ld32(b.tmem + acc * TILE + ((uint32_t)(32 * quad) << 16) + 32 * q, v);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0.0f;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4* at16 = reinterpret_cast<uint4*>(stage + (piece(at + (q >> 1) * (TILE * 128), 32 * w + lane, (q & 1) * 4 + k) - at));
            uint4 o = base ? *at16 : make_uint4(0, 0, 0, 0);
            const float* s = v + 8 * k;
            o.x = pack_bf16x2(bf16_lo(o.x) + s[0], bf16_hi(o.x) + s[1]);
            o.y = pack_bf16x2(bf16_lo(o.y) + s[2], bf16_hi(o.y) + s[3]);
            o.z = pack_bf16x2(bf16_lo(o.z) + s[4], bf16_hi(o.z) + s[5]);
            o.w = pack_bf16x2(bf16_lo(o.w) + s[6], bf16_hi(o.w) + s[7]);
            *at16 = o;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.acc_empty[acc]);
        const int c = lane & 15;
        const bool col = c0 + c * 8 < N;
        for (int j = 0; j < 32 && j < mine; j += 2) {
          const int row = j + (lane >> 4);
          const int id = __shfl_sync(0xFFFFFFFFu, row_id, row);
          if (col && row < mine)
            *reinterpret_cast<uint4*>(y + (size_t)id * N + c0 + c * 8) = *reinterpret_cast<const uint4*>(
                stage + (piece(at + (c >> 3) * (TILE * 128), 32 * w + row, c & 7) - at));
        }
      } else if (lane == 0) {
        mbar_arrive(&b.acc_empty[acc]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.empty[st]);
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(b.tmem, 256);
  }
}

// ---------------------------------------------------------------------------
// k_rows: few rows, one cluster per row, on the CUDA cores
// ---------------------------------------------------------------------------
constexpr int ROW_CTAS = 8, ROW_THREADS = 256;

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(bf16_lo(x[i]), bf16_lo(y[i]), s);
    s = fmaf(bf16_hi(x[i]), bf16_hi(y[i]), s);
  }
  return s;
}
__device__ __forceinline__ void add8(float* s, float f, uint4 q) {
  const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s[2 * i] = fmaf(f, bf16_lo(x[i]), s[2 * i]);
    s[2 * i + 1] = fmaf(f, bf16_hi(x[i]), s[2 * i + 1]);
  }
}

__global__ void __launch_bounds__(ROW_THREADS) k_rows(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ P,
                                                      const __nv_bfloat16* __restrict__ Q, const int32_t* __restrict__ idx,
                                                      const float* __restrict__ scale, const __nv_bfloat16* base, int K,
                                                      int N, int r, int G, __nv_bfloat16* y, __nv_bfloat16* __restrict__ h) {
  __shared__ float sums[ROW_CTAS][MAX_R];  // every CTA's sums over its part of K, from all of them
  __shared__ float hid[MAX_R];
  const int row = blockIdx.x / ROW_CTAS, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int a = idx[row];
  const bool has = (unsigned)a < (unsigned)G;
  const int N8 = N / 8, n0 = (int)((int64_t)N8 * rank / ROW_CTAS), n1 = (int)((int64_t)N8 * (rank + 1) / ROW_CTAS);
  if (has) {
    const int K8 = K / 8, k0 = (int)((int64_t)K8 * rank / ROW_CTAS), k1 = (int)((int64_t)K8 * (rank + 1) / ROW_CTAS);
    const uint4* x = reinterpret_cast<const uint4*>(X + (size_t)row * K);
    const uint4* p = reinterpret_cast<const uint4*>(P + (size_t)a * r * K);
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    bool started = false;  // (the others' shared memory may be written once they have begun)
    for (int j = warp; j < r; j += ROW_THREADS / 32) {
      float s = 0.0f;
      for (int k = k0 + lane; k < k1; k += 32) s = dot8(x[k], p[(size_t)j * K8 + k], s);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      if (!started) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      started = true;
      if (lane < ROW_CTAS)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&sums[rank][j]), lane)), "f"(s) : "memory");
    }
    if (!started) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    cluster_sync();
    if (threadIdx.x < r) {
      float s = 0.0f;
      for (int c = 0; c < ROW_CTAS; ++c) s += sums[c][threadIdx.x];
      const __nv_bfloat16 v = __float2bfloat16_rn(s * scale[a]);
      hid[threadIdx.x] = __bfloat162float(v);
      if (h && rank == 0) h[(size_t)row * r + threadIdx.x] = v;
    }
    __syncthreads();
  } else if (h && rank == 0 && threadIdx.x < r) {
    h[(size_t)row * r + threadIdx.x] = __float2bfloat16_rn(0.0f);
  }
  const uint4* q = reinterpret_cast<const uint4*>(Q + (has ? (size_t)a * r * N : 0));
  for (int n = n0 + threadIdx.x; n < n1; n += ROW_THREADS) {
    float s[8];
    const uint4 o = base ? reinterpret_cast<const uint4*>(base + (size_t)row * N)[n] : make_uint4(0, 0, 0, 0);
    const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    if (has)
      for (int j = 0; j < r; ++j) add8(s, hid[j], q[(size_t)j * N8 + n]);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(bf16_lo(ow[i]) + s[2 * i], bf16_hi(ow[i]) + s[2 * i + 1]);
    reinterpret_cast<uint4*>(y + (size_t)row * N)[n] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int FEW_ROWS = 64;

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
int max_tiles(int T, int G) { return T / TILE + (G + 1 < T ? G + 1 : T); }

size_t plan_bytes(int T, int G) {
  return 256 + up256((size_t)(G + 2) * 4) + up256((size_t)max_tiles(T, G) * sizeof(Tile)) + up256((size_t)T * 4);
}

Plan plan_at(void* ws, int T, int G) {
  char* p = static_cast<char*>(ws);
  Plan q;
  q.n_tiles = reinterpret_cast<int*>(p);
  p += 256;
  q.first = reinterpret_cast<int*>(p);
  p += up256((size_t)(G + 2) * 4);
  q.tiles = reinterpret_cast<Tile*>(p);
  p += up256((size_t)max_tiles(T, G) * sizeof(Tile));
  q.rows = reinterpret_cast<int*>(p);
  return q;
}

template <class... A, class... B>
moe_status_t launch(void (*k)(A...), int ctas, int cluster, int threads, int smem, int smem_limit, bool dependent,
                    cudaStream_t stream, B... args) {
  if (smem_limit && !set_smem_limit((const void*)k, smem_limit)) return MOE_ERR_CUDA;  // (one limit per kernel)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 0) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  if (cudaLaunchKernelEx(&cfg, k, static_cast<A>(args)...) != cudaSuccess) return MOE_ERR_CUDA;
  count_launch();
  return launch_status();
}

using bf = __nv_bfloat16;
const bf* in(const moe_bf16* p) { return reinterpret_cast<const bf*>(p); }
bf* out(moe_bf16* p) { return reinterpret_cast<bf*>(p); }

int pad16(int r) { return (r + 15) & ~15; }

moe_status_t group(const int32_t* idx, int T, int G, const Plan& p, cudaStream_t s) {
  const int most = GROUP_SMEM / 4 / (G + 1), warps = most < 32 ? most : 32;
  return launch(k_group, 1, 0, GROUP_THREADS, warps * (G + 1) * 4, GROUP_SMEM, false, s, idx, T, G, warps, p);
}

// CTAs per cluster that share a contraction of `blocks` stages: enough to
// occupy the SMs with `clusters` of them, and two stages each at least.
int split_of(int clusters, int blocks) {
  int s = 1;
  while (s < 8 && clusters * s < 2 * 152 && blocks >= 4 * s) s *= 2;
  return s;
}

moe_status_t shrink(const moe_bf16* x, const moe_bf16* P, const float* scale, int T, int K, int r, int G, const Plan& p,
                    moe_bf16* h, int32_t* st, cudaStream_t s) {
  const int rp = pad16(r), tiles = max_tiles(T, G), split = split_of((T + TILE - 1) / TILE, (K + KB - 1) / KB);
  const uint64_t lim = g_wait_limit_ns.load();
  return rp <= 64 ? launch(k_shrink<64>, tiles * split, split, THREADS, Ring<64>::BYTES, Ring<64>::BYTES, true, s, in(x), in(P), scale, K, r,
                           rp, p, out(h), lim, st)
                  : launch(k_shrink<128>, tiles * split, split, THREADS, Ring<128>::BYTES, Ring<128>::BYTES, true, s, in(x), in(P), scale, K,
                           r, rp, p, out(h), lim, st);
}

moe_status_t wgrad(const moe_bf16* x, const moe_bf16* u, int T, int C, int r, int G, const Plan& p, moe_bf16* dP,
                   int32_t* st, cudaStream_t s) {
  const int rp = pad16(r), units = G * ((C + TILE - 1) / TILE), split = split_of(units, (T + KB - 1) / KB);
  const uint64_t lim = g_wait_limit_ns.load();
  return rp <= 64 ? launch(k_wgrad<64>, units * split, split, THREADS, Ring<64>::BYTES, Ring<64>::BYTES, true, s, in(x), in(u), C, r, rp, p,
                           out(dP), lim, st)
                  : launch(k_wgrad<128>, units * split, split, THREADS, Ring<128>::BYTES, Ring<128>::BYTES, true, s, in(x), in(u), C, r, rp, p,
                           out(dP), lim, st);
}

moe_status_t expand(const moe_bf16* h, const moe_bf16* Q, const moe_bf16* base, int T, int N, int r, int G, const Plan& p,
                    moe_bf16* y, int32_t* st, cudaStream_t s) {
  const int rp = pad16(r), sms = sm_count();
  if (sms < 1) return MOE_ERR_CUDA;
  const int64_t units = (int64_t)max_tiles(T, G) * ((N + TILE - 1) / TILE);
  const int grid = units < sms ? (int)units : sms;
  const uint64_t lim = g_wait_limit_ns.load();
  auto go = [&](auto k, int bytes) {
    return launch(k, grid, 0, WIDE_THREADS, bytes, bytes, true, s, in(h), in(Q), in(base), N, r, rp, p, out(y), lim, st);
  };
  return rp <= 32   ? go(k_expand<32>, Wide<32>::BYTES)
         : rp <= 64 ? go(k_expand<64>, Wide<64>::BYTES)
                    : go(k_expand<128>, Wide<128>::BYTES);
}

bool sizes_ok(int T, int K, int N, int r, int G) {
  return T >= 0 && T <= (1 << 27) && K > 0 && N > 0 && K % 8 == 0 && N % 8 == 0 && K <= (1 << 20) && N <= (1 << 20) && r > 0 &&
         r % 8 == 0 && G > 0;
}

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + bn && y < x + an;
}

}  // namespace lora
}  // namespace moeglu

using namespace moeglu;
using namespace moeglu::lora;

extern "C" size_t moe_lora_workspace_size(int T, int r, int G) {
  if (T < 0 || r <= 0 || G <= 0) return 0;
  return plan_bytes(T, G) + up256((size_t)T * r * 2);
}

extern "C" moe_status_t moe_lora_fwd(const moe_bf16* x, const moe_bf16* A, const moe_bf16* B, const int32_t* idx,
                                     const float* scale, const moe_bf16* base, int T, int K, int N, int r, int G,
                                     moe_bf16* y, moe_bf16* h, void* ws, size_t ws_bytes, int32_t* status,
                                     moe_stream_t stream) {
  if (!sizes_ok(T, K, N, r, G)) return MOE_ERR_ARG;
  if (r > MAX_R || G > MAX_G) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !A || !B || !idx || !scale || !y || !ws || ws_bytes < moe_lora_workspace_size(T, r, G)) return MOE_ERR_ARG;
  if (!aligned16(x) || !aligned16(A) || !aligned16(B) || !aligned16(base) || !aligned16(y) || !aligned16(h) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u))
    return MOE_ERR_ARG;
  const size_t yn = (size_t)T * N * 2;
  if ((base != y && overlap(y, yn, base, yn)) || overlap(y, yn, x, (size_t)T * K * 2) ||
      overlap(y, yn, A, (size_t)G * r * K * 2) || overlap(y, yn, B, (size_t)G * r * N * 2))
    return MOE_ERR_ARG;
  const cudaStream_t s = as_stream(stream);
  if (T <= FEW_ROWS)
    return launch(k_rows, T * ROW_CTAS, ROW_CTAS, ROW_THREADS, 0, 0, false, s, in(x), in(A), in(B), idx, scale, in(base), K, N,
                  r, G, out(y), out(h));
  const Plan p = plan_at(ws, T, G);
  if (!h) h = reinterpret_cast<moe_bf16*>(static_cast<char*>(ws) + plan_bytes(T, G));
  if (const moe_status_t e = group(idx, T, G, p, s)) return e;
  if (const moe_status_t e = shrink(x, A, scale, T, K, r, G, p, h, status, s)) return e;
  return expand(h, B, base, T, N, r, G, p, y, status, s);
}

extern "C" moe_status_t moe_lora_bwd(const moe_bf16* dy, const moe_bf16* x, const moe_bf16* h, const moe_bf16* A,
                                     const moe_bf16* B, const int32_t* idx, const float* scale, const moe_bf16* base, int T,
                                     int K, int N, int r, int G, moe_bf16* dx, moe_bf16* dA, moe_bf16* dB, void* ws,
                                     size_t ws_bytes, int32_t* status, moe_stream_t stream) {
  if (!sizes_ok(T, K, N, r, G)) return MOE_ERR_ARG;
  if (r > MAX_R || G > MAX_G) return MOE_ERR_UNSUPPORTED;
  if (!dA || !dB || !aligned16(dA) || !aligned16(dB)) return MOE_ERR_ARG;
  const cudaStream_t s = as_stream(stream);
  if (T == 0) {
    if (cudaMemsetAsync(dA, 0, (size_t)G * r * K * 2, s) != cudaSuccess ||
        cudaMemsetAsync(dB, 0, (size_t)G * r * N * 2, s) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!dy || !x || !h || !A || !B || !idx || !scale || !dx || !ws || ws_bytes < moe_lora_workspace_size(T, r, G))
    return MOE_ERR_ARG;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(h) || !aligned16(A) || !aligned16(B) || !aligned16(base) ||
      !aligned16(dx) || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return MOE_ERR_ARG;
  const size_t xn = (size_t)T * K * 2, an = (size_t)G * r * K * 2, bn = (size_t)G * r * N * 2;
  if ((base != dx && overlap(dx, xn, base, xn)) || overlap(dx, xn, x, xn) || overlap(dx, xn, dy, (size_t)T * N * 2) ||
      overlap(dx, xn, h, (size_t)T * r * 2) || overlap(dx, xn, A, an) || overlap(dA, an, A, an) || overlap(dB, bn, B, bn))
    return MOE_ERR_ARG;
  const Plan p = plan_at(ws, T, G);
  auto* u = reinterpret_cast<moe_bf16*>(static_cast<char*>(ws) + plan_bytes(T, G));
  if (const moe_status_t e = group(idx, T, G, p, s)) return e;
  if (const moe_status_t e = shrink(dy, B, scale, T, N, r, G, p, u, status, s)) return e;
  if (const moe_status_t e = expand(u, A, base, T, K, r, G, p, dx, status, s)) return e;
  if (const moe_status_t e = wgrad(x, u, T, K, r, G, p, dA, status, s)) return e;
  return wgrad(dy, h, T, N, r, G, p, dB, status, s);
}
