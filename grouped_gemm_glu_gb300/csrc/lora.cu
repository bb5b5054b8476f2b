// Low-rank adapters of many requests beside a projection that they share.
//
//   h_t = s_a P_a x_t,  y_t = base_t + Q_a^T h_t   for row t with adapter a
//   (P [G][r][K], Q [G][r][N]; rows without one: h = 0, y = base)
//
// The forward has P = A, Q = B.  The backward is the same pair with the roles
// turned (u = s_a B_a dy, dx = base + A_a^T u), and the adapters' gradients are
// sums over an adapter's rows, dA_a = sum u x^T, dB_a = sum h dy^T.  Sums are
// fp32, outputs are rounded once.  Where h and u are tensor-core operands of the
// products behind them they are two bf16 numbers, the value's rounding and what
// that drops (16 bits and more: one bf16 number made y's and dA's errors a third
// larger, and all of y's where base and product cancel); dB takes the bf16 h that
// the caller kept.
//
// Memory bound: with r of 8 to 128 each element of x, base and y takes 2 r
// operations.  Three kernels on tcgen05, all over rows grouped by adapter:
//   k_shrink  D[128 rows][r] = X P^T, contracted over K
//   k_expand  D[128 rows][128 columns] = H Q, contracted over r, plus base
//   k_wgrad   D[128 columns][r] = X^T U, contracted over an adapter's rows
// A first kernel (k_group) sorts the row indexes by adapter, stably, and cuts
// each adapter's rows into tiles of 128; the rows themselves stay where they
// are.  Each warp that loads or stores looks at its 32 rows: neighbours in
// memory (a request's tokens, mostly) move as one box by TMA, others row by row
// (16-byte asynchronous copies into the same swizzled layout), so that every
// order of rows is served, no tile mixes adapters and no work is done for
// absent ones.  h and u are also kept in the grouped order (an adapter's rows
// from a multiple of 16 on, zeros up to the next one), where the products
// behind them read them by TMA.
// k_shrink and k_wgrad produce little from much: the CTAs of a cluster share
// a contraction and add their sums through distributed shared memory, always
// in the same order, so equal inputs give equal bits.
// Few rows (decoding) take k_rows instead: one cluster per row, one launch; in
// the backward k_row_grads behind it.
//
// Measured, calls that follow one another: 8192 x 7168 with 32 adapters of rank
// 16, forward 72 us (grouping 6; k_shrink 24, 117 MB at 4.9 TB/s, where a kernel
// that only loads them takes 21; k_expand 43, 235 MB at 5.5 TB/s, where a plain
// copy takes 38 to 40); with 8 of rank 32, backward 123 us (k_wgrad 48 for both
// gradients, 4.9 TB/s); one row of 2880 4 us, 64 rows of 7168 with 64 adapters 8.2.
#include "common.cuh"
#include "host_common.h"

#include <initializer_list>

namespace moeglu {
namespace lora {

constexpr int TILE = 128;  // rows of one adapter per tile, columns per unit
constexpr int SLAB = 32;   // rows that a warp moves
constexpr int MAX_R = 128;
constexpr int KB = 64;     // contraction per stage (128-byte operand rows)
constexpr int ALIGN = 16;  // an adapter's first place in the grouped order: the MMA's contraction
constexpr int MIN_BOX = 8; // fewer neighbours than this are copied row by row

struct Tile {
  int adapter, start, count, pad;  // -1: rows without an adapter; first place in the grouped order
};
// Workspace: the grouped order.
struct Plan {
  int* sums;    // tiles with an adapter, all tiles, k_expand's jobs taken
  int* first;   // [G + 2]: each adapter's first place; the rows without one; the end
  Tile* tiles;
  int* rows;    // row of each place, -1 where there is none
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
// Arrives on the barrier when the thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// The arrivals of a warp's 32 threads by one of them (they are served one after the other).
__device__ __forceinline__ void mbar_arrive_warp(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 32;" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* m, uint64_t* bar, int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
// (of data that nothing reads again soon: they leave L2 before others)
__device__ __forceinline__ void tma_2d_once(uint32_t dst, const CUtensorMap* m, uint64_t* bar, int32_t c0, int32_t c1) {
  uint64_t first;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::
          "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "l"(first)
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, uint64_t* bar, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// 16-byte piece c of 128-byte row `row` of a tile in the 128-byte swizzle
__device__ __forceinline__ uint32_t piece(uint32_t tile, int row, int c) {
  return tile + row * 128 + ((c ^ (row & 7)) << 4);
}

// The rank's operands (rows of r elements in the grouped order) have rows of
// 32, 64 or 128 bytes, by the rank: 16, 32 or blocks of 64 elements, each
// swizzled over its row's length.
__host__ __device__ constexpr int rank_cols(int rp) { return rp <= 16 ? 16 : rp <= 32 ? 32 : 64; }
__host__ __device__ constexpr int rank_bytes(int rp) { return rp <= 64 ? rank_cols(rp) * 2 : 256; }
__device__ __forceinline__ uint64_t swizzle_bits(uint32_t row_bytes) {
  return (uint64_t)(row_bytes == 128 ? 2u : row_bytes == 64 ? 4u : 6u) << 61;
}
// Operand tiles: rows of row_bytes along the contraction (kmajor) or across it
// (mnmajor: the rows are steps of the contraction, `block` bytes between
// blocks of the kept dimension).
__device__ __forceinline__ uint64_t sdesc_kmajor(uint32_t saddr, uint32_t row_bytes) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(row_bytes >> 1) << 32) | (1ull << 46) | swizzle_bits(row_bytes);
}
__device__ __forceinline__ uint64_t sdesc_mnmajor(uint32_t saddr, uint32_t row_bytes, uint32_t block) {
  return sdesc_kmajor(saddr, row_bytes) | ((uint64_t)(block >> 4) << 16);
}
constexpr uint32_t A_MN = 1u << 15, B_MN = 1u << 16;  // instruction descriptor: that operand lies across the contraction

// 32 columns of the thread's lane of tensor memory, written; and the MMA whose
// left operand lies there (a row per lane, two elements per column).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void umma_bf16_from_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, 1, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc)
      : "memory");
}

// The sum of twice 32 columns of the thread's lane.
__device__ __forceinline__ void tmem_ld32_sum(uint32_t at, uint32_t other, float* v) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, [%64];\n tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
      "}, [%65];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(at), "r"(other)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) + __uint_as_float(r[32 + i]);
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ int ld_cluster_int(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
// The dynamic shared memory from its first multiple of 1024 bytes on (the
// swizzle's period; 1024 bytes more are asked for).
__device__ __forceinline__ unsigned char* aligned_smem(unsigned char* p) { return p + ((0u - smem_u32(p)) & 1023u); }

// A look at a barrier that does not hold the thread back; not ready gives up.
__device__ __noinline__ bool no_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  if (ok) return true;
  *abort = 1;
  set_status(status, MOE_ERR_TIMEOUT);
  return false;
}
// mbar_wait for waits that mostly last a few hundred cycles: the clock and the
// abort flag are read at every 256th look only, the first time included.  (A look
// lasts until the barrier is ready or for some microseconds; the least limit,
// 1 ns, therefore does not wait at all.)
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, const WaitGuard& g) {
  if (g.limit_ns < 2) return no_wait(bar, parity, g.abort, g.status);
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_test(bar, parity)) return true;
    if ((it & 255u) == 0) {
      if (*g.abort) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > g.limit_ns) {
        *g.abort = 1;
        set_status(g.status, MOE_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

// The waits at a CTA's end, before it gives up its shared and its tensor memory:
// for copies and MMAs that it has issued, whether or not it has aborted.
constexpr uint64_t LAND_NS = 1000000;
__device__ __forceinline__ bool land(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_test(bar, parity))
    if (globaltimer_ns() - t0 > limit_ns) return false;
  return true;
}
// MMAs: their end is signalled in any case.
__device__ __forceinline__ void land_mma(uint64_t* done, uint32_t parity, const WaitGuard& g) {
  if (land(done, parity, g.limit_ns > LAND_NS ? g.limit_ns : LAND_NS)) return;
  *g.abort = 1;
  set_status(g.status, MOE_ERR_TIMEOUT);
}
// Copies of the last steps issued, after an abort: a stage on which another warp
// has not arrived stays open, but a millisecond is enough for the copies.
__device__ __forceinline__ void settle(uint64_t* full, int stages, int issued) {
  for (int k = max(0, issued - stages); k < issued; ++k) land(&full[k % stages], (k / stages) & 1, LAND_NS);
}

// The operands of TMA and tcgen05 instructions are uniform registers.  Loops
// that issue them are run by whole warps with one elected lane, on values made
// uniform here: where a single lane runs the loop, each operand is moved there
// on its own (k_wgrad's four MMAs and a commit took 1190 cycles a step).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
template <class T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xFFFFFFFFu, v, 0);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitGuard& g) {
  return __all_sync(0xFFFFFFFFu, wait_on(bar, parity, g));
}

// A warp's 32 places: the row of each lane (-1: none), and whether they are
// neighbours in memory, as far as there are any (the first lanes').
struct Slab {
  int row, first, count;
  bool box;
  // bit l: lane l's group of eight lanes has neighbours too, as far as it has rows / has eight of them
  uint32_t near, whole;
};
__device__ __forceinline__ Slab slab_of(int row) {
  Slab s;
  s.row = row;
  s.count = __popc(__ballot_sync(0xFFFFFFFFu, row >= 0));
  s.first = __shfl_sync(0xFFFFFFFFu, row, 0);
  s.box = __all_sync(0xFFFFFFFFu, row < 0 || row == s.first + (int)(threadIdx.x & 31));
  const int head = __shfl_sync(0xFFFFFFFFu, row, threadIdx.x & 24);
  const uint32_t next = __ballot_sync(0xFFFFFFFFu, row < 0 || row == head + (int)(threadIdx.x & 7));
  const uint32_t some = __ballot_sync(0xFFFFFFFFu, row >= 0);
  auto all8 = [](uint32_t m) { return m & (m >> 1) & (m >> 2) & (m >> 3) & (m >> 4) & (m >> 5) & (m >> 6) & (m >> 7) & 0x01010101u; };
  s.near = all8(next) * 0xFFu;
  s.whole = all8(next & some) * 0xFFu;
  return s;
}

// ---------------------------------------------------------------------------
// Grouping: one CTA; warp w counts and places its stretch of rows
// ---------------------------------------------------------------------------
constexpr int GROUP_THREADS = 1024, GROUP_SMEM = 128 * 1024, MAX_G = GROUP_SMEM / 4 - 1;
constexpr int HELD = 8;  // indexes that a lane keeps between the two passes

__device__ __forceinline__ int warp_scan(int v) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if ((int)(threadIdx.x & 31) >= d) v += o;
  }
  return v;
}

__global__ void __launch_bounds__(GROUP_THREADS) k_group(const int32_t* __restrict__ idx, int T, int G, int warps, Plan p) {
  launch_dependents();
  extern __shared__ int hist[];  // [G + 1][warps]
  __shared__ int part[2][32], count[GROUP_THREADS], begin[GROUP_THREADS], tile_at[GROUP_THREADS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, groups = G + 1;
  const int per = ((T + warps - 1) / warps + 31) & ~31;
  const int lo = min(T, warp * per), hi = warp < warps ? min(T, lo + per) : lo;
  int held[HELD];
#pragma unroll
  for (int i = 0; i < HELD; ++i) held[i] = lo + 32 * i + lane < hi ? idx[lo + 32 * i + lane] : 0;
  for (int i = tid; i < warps * groups; i += GROUP_THREADS) hist[i] = 0;
  __syncthreads();
  // f(row, group, lanes of the same group) for the warp's rows, 32 at a time
  auto each = [&](auto f) {
    auto one = [&](int b, int a) {
      const bool ok = b + lane < hi;
      a = !ok ? -1 : (unsigned)a < (unsigned)G ? a : G;  // (-1: a group of its own, not counted)
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, a);
      f(b + lane, a, same);
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (lo + 32 * i < hi) one(lo + 32 * i, held[i]);
    for (int b = lo + 32 * HELD; b < hi; b += 32) one(b, b + lane < hi ? idx[b + lane] : 0);
  };
  const uint32_t below = (1u << lane) - 1;
  each([&](int, int a, uint32_t same) {
    if (a >= 0 && (same & below) == 0) hist[a * warps + warp] += __popc(same);
    __syncwarp();
  });
  __syncthreads();
  // 1024 groups at a time: the rows of each before each warp's, and the sums over the groups before it (rows up to
  // whole ALIGNs, tiles)
  int rows0 = 0, tiles0 = 0;
  const bool few = groups <= GROUP_THREADS;  // (then `begin` still holds every group's first place in the end)
  for (int g0 = 0; g0 < groups; g0 += GROUP_THREADS) {
    for (int g = g0 + warp; g < min(groups, g0 + GROUP_THREADS); g += GROUP_THREADS / 32) {
      const int n = lane < warps ? hist[g * warps + lane] : 0, s = warp_scan(n);
      if (lane < warps) hist[g * warps + lane] = s - n;
      if (lane == 31) count[g - g0] = s;
    }
    __syncthreads();
    const int g = g0 + tid, n = g < groups ? count[tid] : 0;
    const int up = (n + ALIGN - 1) / ALIGN * ALIGN, tiles = (n + TILE - 1) / TILE;
    int rs = warp_scan(up), ts = warp_scan(tiles);
    if (lane == 31) part[0][warp] = rs, part[1][warp] = ts;
    __syncthreads();
    if (warp < 2) part[warp][lane] = warp_scan(part[warp][lane]);
    __syncthreads();
    if (warp) rs += part[0][warp - 1], ts += part[1][warp - 1];
    begin[tid] = rows0 + rs - up;
    tile_at[tid] = tiles0 + ts - tiles;
    if (g < groups) p.first[g] = begin[tid];
    if (g == G) {
      p.first[groups] = begin[tid] + up;
      p.sums[0] = tile_at[tid];
      p.sums[1] = tile_at[tid] + tiles;
      p.sums[2] = 0;
    }
    rows0 += part[0][31];
    tiles0 += part[1][31];
    __syncthreads();
    for (int k = warp; k < min(groups - g0, GROUP_THREADS); k += GROUP_THREADS / 32) {
      const int c = count[k], r0 = begin[k], a = g0 + k;
      for (int i = lane; i * TILE < c; i += 32)
        p.tiles[tile_at[k] + i] = {a < G ? a : -1, r0 + i * TILE, min(TILE, c - i * TILE), 0};
      if (c + lane < (c + ALIGN - 1) / ALIGN * ALIGN) p.rows[r0 + c + lane] = -1;
      if (!few && lane < warps) hist[a * warps + lane] += r0;
    }
    __syncthreads();
  }
  each([&](int row, int a, uint32_t same) {
    int at = 0;
    if (a >= 0) {
      at = hist[a * warps + warp];
      p.rows[at + (few ? begin[a] : 0) + __popc(same & below)] = row;
    }
    __syncwarp();
    if (a >= 0 && (same & below) == 0) hist[a * warps + warp] = at + __popc(same);
    __syncwarp();
  });
}

// ---------------------------------------------------------------------------
// k_shrink: cluster (tile), its CTAs share K.  Warps 0 to 3 load 32 rows each
// and write out, warp 4 issues the MMAs.
// ---------------------------------------------------------------------------
constexpr int SHRINK_THREADS = 160;
// (4500 x 2880 x 5760 with rank 64 40.7 us, with three stages 41.2; 512 rows of 64 adapters of rank 16 39.0 and 41.0; ranks
// 16 and 32 at 8192 x 7168 within 1%; rank 128, whose stages are larger, 100.0 and 95.9)
__host__ __device__ constexpr int shrink_stages(int rp) { return rp <= 64 ? 4 : 3; }
__host__ __device__ constexpr int shrink_stage(int rp) { return TILE * 128 + rp * 128; }
constexpr int shrink_bytes(int rp) {  // (the ring holds the sums in the end: 512 rp bytes)
  return (shrink_stages(rp) * shrink_stage(rp) > 512 * rp ? shrink_stages(rp) * shrink_stage(rp) : 512 * rp) + 1024;
}
struct Bars {
  uint64_t full[4], empty[4], done;
  int abort;
  uint32_t tmem;
};
// Columns of tensor memory for an accumulator of rp columns (a power of two, at
// least 32).  An allocation may wait for another CTA to give some up, and a CTA of
// a dependent kernel (of this file or of any other) keeps what it has until the
// kernel in front of it has ended.  So each of these kernels allocates once, and
// lets its dependents start only behind that, in every CTA that works: whoever holds
// tensor memory and waits does so for CTAs that have theirs.
__device__ __forceinline__ uint32_t tmem_cols(int rp) { return rp <= 32 ? 32 : rp <= 64 ? 64 : 128; }

// Eight values times f as bf16, and what that drops as bf16 (nothing of an
// infinity): together 16 bits and more.
struct Parts {
  uint4 hi, lo;
};
__device__ __forceinline__ uint32_t dropped(float x, float y, uint32_t hi) {
  const float a = x - bf16_lo(hi), b = y - bf16_hi(hi), most = 3.3e38f;
  return pack_bf16x2(fabsf(a) < most ? a : 0.0f, fabsf(b) < most ? b : 0.0f);
}
__device__ __forceinline__ Parts split8(float4 s, float4 t, float f) {
  s = make_float4(s.x * f, s.y * f, s.z * f, s.w * f);
  t = make_float4(t.x * f, t.y * f, t.z * f, t.w * f);
  Parts p;
  p.hi = make_uint4(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w), pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
  p.lo = make_uint4(dropped(s.x, s.y, p.hi.x), dropped(s.z, s.w, p.hi.y), dropped(t.x, t.y, p.hi.z), dropped(t.z, t.w, p.hi.w));
  return p;
}

// X [T][K] (and as a tensor map, boxes of 64 columns x 32 rows), P as a map
// of boxes 64 x rp.  h [T][r] (nullable) by row, hs [2][places][r] in the
// grouped order, in two parts (split4); also (other, nullable [T][r]) copied into
// that order as others [places][r].
__global__ void __launch_bounds__(SHRINK_THREADS) k_shrink(const __grid_constant__ CUtensorMap mx,
                                                           const __grid_constant__ CUtensorMap mp,
                                                           const __nv_bfloat16* __restrict__ X,
                                                           const float* __restrict__ scale, int K, int r, int rp, Plan plan,
                                                           int places, __nv_bfloat16* __restrict__ h, __nv_bfloat16* __restrict__ hs,
                                                           const __nv_bfloat16* __restrict__ other,
                                                           __nv_bfloat16* __restrict__ others, uint64_t limit_ns,
                                                           int32_t* status) {
  extern __shared__ unsigned char smem_[];
  unsigned char* smem = aligned_smem(smem_);
  __shared__ Bars b;
  __shared__ int rows[TILE];
  const uint32_t size = cluster_size(), rank = cluster_ctarank();
  const int tile = blockIdx.x / size, warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31, stages = shrink_stages(rp);
  wait_for_primary();
  if (tile >= plan.sums[1]) return;  // (the whole cluster)
  // backwards: k_wgrad, next in the backward, begins with the first tiles and finds dy's last read rows in L2
  const Tile t = plan.tiles[plan.sums[1] - 1 - tile];
  const int up = (t.count + ALIGN - 1) / ALIGN * ALIGN;
  if (threadIdx.x < TILE) rows[threadIdx.x] = threadIdx.x < up ? plan.rows[t.start + threadIdx.x] : -1;
  if (t.adapter < 0) {  // rows without an adapter
    __syncthreads();
    if (h)
      for (int i = threadIdx.x + rank * SHRINK_THREADS; i < t.count * (r / 8); i += SHRINK_THREADS * size)
        *reinterpret_cast<uint4*>(h + (size_t)rows[i / (r / 8)] * r + (i % (r / 8)) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&b.full[i], 4);
      mbar_init(&b.empty[i], 1);
    }
    mbar_init(&b.done, 1);
    b.abort = 0;
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(&b.tmem, tmem_cols(rp));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();  // (with tensor memory in hand: tmem_cols)
  const WaitGuard g{&b.abort, status, limit_ns};
  const uint32_t ring = smem_u32(smem), stage = shrink_stage(rp);
  const int blocks = (K + KB - 1) / KB;
  const int k0 = (int)((int64_t)blocks * rank / size), steps = (int)((int64_t)blocks * (rank + 1) / size) - k0;
  int st = 0, issued = 0;  // a step's stage, and its turn of the ring; steps whose copies this warp has issued
  uint32_t turn = 0;
  auto next_stage = [&] {
    if (++st == stages) st = 0, ++turn;
  };
  if (warp < 4) {
    const Slab s = slab_of(rows[threadIdx.x]);
    const uint32_t slab = warp * SLAB * 128;
    const int adapter = uniform(t.adapter), first = uniform(s.first), count = uniform(s.count);
    if (count == 0 || (s.box && count >= MIN_BOX)) {
      for (int i = 0; i < steps; ++i, next_stage()) {
        if (turn > 0 && !warp_wait(&b.empty[st], (turn - 1) & 1, g)) break;
        const uint32_t at = ring + st * stage;
        if (elect_one()) {
          mbar_arrive_expect_tx(&b.full[st], (count ? SLAB * 128 : 0) + (warp == 0 ? rp * 128 : 0));
          if (count) tma_2d(at + slab, &mx, &b.full[st], (k0 + i) * KB, first);
          if (warp == 0) tma_3d(at + TILE * 128, &mp, &b.full[st], (k0 + i) * KB, 0, adapter);
        }
        __syncwarp();
        ++issued;
      }
    } else {
      // row by row: eight lanes copy a row's 128 bytes, and arrive two steps later, when they have landed
      const int c = lane & 7;
      const __nv_bfloat16* src[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = __shfl_sync(0xFFFFFFFFu, s.row, (lane >> 3) + 4 * j);
        src[j] = row >= 0 ? X + (size_t)row * K + c * 8 : nullptr;
      }
      constexpr int LAG = 2;
      int i = 0, landed = 0;  // the stage of the step before the last LAG ones
      auto arrive = [&] {
        if (lane == 0) mbar_arrive(&b.full[landed]);
        if (++landed == stages) landed = 0;
      };
      for (; i < steps; ++i, next_stage()) {
        if (turn > 0 && !warp_wait(&b.empty[st], (turn - 1) & 1, g)) break;
        const uint32_t at = ring + st * stage;
        const int k = (k0 + i) * KB;
        if (warp == 0 && elect_one()) {
          mbar_expect_tx(&b.full[st], rp * 128);
          tma_3d(at + TILE * 128, &mp, &b.full[st], k, 0, adapter);
        }
        __syncwarp();
        ++issued;
        const bool in = k + c * 8 < K;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (src[j]) cp16(piece(at + slab, (lane >> 3) + 4 * j, c), in ? src[j] + k : X, in);
        cp_commit();
        if (i >= LAG) {
          cp_wait<LAG>();
          fence_async_shared();
          __syncwarp();
          arrive();
        }
      }
      cp_wait<0>();
      fence_async_shared();
      __syncwarp();
      if (i == steps)
        for (int k = max(0, steps - LAG); k < steps; ++k) arrive();
    }
  } else {
    const uint32_t idesc = idesc_bf16_f32(TILE, rp), tmem = uniform(b.tmem);
    for (int i = 0; i < steps; ++i, next_stage()) {
      if (!warp_wait(&b.full[st], turn & 1, g)) break;
      tc_fence_after();
      const uint64_t a = sdesc_kmajor(ring + st * stage, 128), w = sdesc_kmajor(ring + st * stage + TILE * 128, 128);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < KB / 16; ++k) umma_bf16(tmem, a + 2 * k, w + 2 * k, idesc, (i | k) != 0);
        tc_commit(&b.empty[st]);
      }
      __syncwarp();
    }
    if (elect_one()) tc_commit(&b.done);
    __syncwarp();
  }
  if (warp == 4) land_mma(&b.done, 0, g);
  tc_fence_before();
  __syncthreads();  // (every copy has landed and every MMA has read: the ring is free, unless a wait gave up)
  tc_fence_after();
  if (b.abort && lane == 0) settle(b.full, stages, issued);
  __syncwarp();
  // the sums to shared memory, as float4 [rp / 4][128]
  if (warp < 4 && !b.abort) {
    for (int c = 0; c < rp; c += 32) {
      float v[32];
      if (steps > 0) {
        tmem_ld32(b.tmem + ((uint32_t)(32 * warp) << 16) + c, v);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + 4 * i < rp)
          *reinterpret_cast<float4*>(smem + (((c >> 2) + i) * TILE + threadIdx.x) * 16) =
              make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  }
  tc_fence_before();
  cluster_sync();
  if (!b.abort) {
    const float f = scale[t.adapter];
    const int items = up * (r / 8);
    for (int i = threadIdx.x + rank * SHRINK_THREADS; i < items; i += SHRINK_THREADS * size) {
      const int q = i / up, l = i - q * up;  // (eight columns of a row)
      const bool mine = l < t.count;
      float4 sum[2], v[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        sum[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c)
          v[k][c] = c < size && mine ? ld_cluster(mapa_shared(ring + ((2 * q + k) * TILE + l) * 16, c)) : sum[k];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c) {
          sum[k].x += v[k][c].x, sum[k].y += v[k][c].y;
          sum[k].z += v[k][c].z, sum[k].w += v[k][c].w;
        }
      Parts o{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (mine) o = split8(sum[0], sum[1], f);
      const size_t to = (size_t)(t.start + l) * r + q * 8;
      if (h && mine) *reinterpret_cast<uint4*>(h + (size_t)rows[l] * r + q * 8) = o.hi;
      *reinterpret_cast<uint4*>(hs + to) = o.hi;
      *reinterpret_cast<uint4*>(hs + (size_t)places * r + to) = o.lo;
      if (other)
        *reinterpret_cast<uint4*>(others + to) =
            mine ? *reinterpret_cast<const uint4*>(other + (size_t)rows[l] * r + q * 8) : make_uint4(0, 0, 0, 0);
    }
  }
  cluster_sync();  // (the other CTAs have read this one's sums)
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(b.tmem, tmem_cols(rp));
  }
}

// ---------------------------------------------------------------------------
// k_wgrad: cluster (128 columns of x or dy, X [T][C]), its CTAs share the tiles of all
// adapters: dP [G][r][C] = U^T X over each adapter's rows, U in the grouped
// order, u in two parts (h, which the caller gives in bf16, in one).  An adapter's
// tiles that cross from one CTA's share into the next ones' are summed by the
// whole cluster in the end.  A step of the ring is one tile, or neighbouring small
// ones together (they lie side by side in the grouped order), whose rows are under
// way at once.
// BESIDE: u's parts are one operand of twice the columns, whose sums meet when
// they are written out, so that an MMA reads x once for both; else two MMAs into
// one accumulator, for runs of few rows, which writing out bounds (host rule at
// wgrad).
// Warps 0 to 3 load 32 rows each, 4 issues the MMAs, 5 to 8 write out; two
// accumulators, and one for the run from before, which stays there to the end.
// ---------------------------------------------------------------------------
constexpr int WGRAD_THREADS = 288, BATCH = 32, STEPS = 16;  // tiles looked up together, in so many steps
constexpr int SMALL = 64;  // places: tiles of at most so many that begin in the same SMALL places share a step
__host__ __device__ constexpr int wgrad_stages(int rp) { return rp <= 32 ? 2 : rp <= 64 ? 3 : 2; }
__host__ __device__ constexpr int wgrad_stage(int rp) { return TILE * 256 + 2 * TILE * rank_bytes(rp); }
constexpr int wgrad_bytes(int rp) { return wgrad_stages(rp) * wgrad_stage(rp) + 1024; }
static_assert(wgrad_stages(16) * wgrad_stage(16) >= 2 * 512 * 16 && wgrad_stages(128) * wgrad_stage(128) >= 2 * 512 * 128,
              "two runs' sums");

// of a tile in this CTA: the first / last of its run of one adapter; the run began before / goes on behind it; the first /
// last of its step
enum { RUN_BEGINS = 1, RUN_ENDS = 2, FROM_BEFORE = 4, GOES_ON = 8, STEP_BEGINS = 16, STEP_ENDS = 32 };

// One of the two gradients, which share a launch: dA (x and u) and dB (dy and h).
struct Side {
  CUtensorMap mx, mu;
  const __nv_bfloat16* X;
  __nv_bfloat16* dP;
  int C, units;  // units: 128 columns each
};
struct Sides {
  Side of[2];
};

template <bool BESIDE>
__global__ void __launch_bounds__(WGRAD_THREADS) k_wgrad(const __grid_constant__ Sides sides, int r, int rp, int G, Plan plan,
                                                         int places, uint64_t limit_ns, int32_t* status) {
  extern __shared__ unsigned char smem_[];
  unsigned char* smem = aligned_smem(smem_);
  __shared__ uint64_t full[3], empty[3], acc_full[2], acc_empty[2], done;  // (the head's accumulator has none: `done`)
  __shared__ int abort_, head_through, tail_adapter;
  __shared__ uint32_t tmem_;
  __shared__ int4 part[BATCH];                           // of each tile: first place, places, adapter, flags
  __shared__ int2 step_of[STEPS];                        // first place, places
  __shared__ int row_of[STEPS][TILE], box_of[STEPS][4];  // rows of each step; the first one of 32 neighbours, or -1
  const uint32_t size = cluster_size(), rank = cluster_ctarank();
  const int unit = (int)(blockIdx.x / size), second = unit >= sides.of[0].units ? 1 : 0;
  const Side& side = sides.of[second];
  const CUtensorMap &mx = side.mx, &mu = side.mu;
  const __nv_bfloat16* const X = side.X;
  __nv_bfloat16* const dP = side.dP;
  const int C = side.C, c0 = (unit - (second ? sides.of[0].units : 0)) * TILE;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int stages = wgrad_stages(rp);
  const uint32_t ring = smem_u32(smem), stage = wgrad_stage(rp);
  const bool beside = BESIDE && !second;
  const uint32_t acc_cols = BESIDE ? 2 * rank_cols(rp) : tmem_cols(rp);
  // in the end, behind the last step, the ring holds what the cluster sums, as float4 [rp / 4][128] each: the run that goes
  // on behind this share, and the one from before it
  unsigned char *const tail = smem, *const head = smem + 512 * rp;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(&done, 1);
    abort_ = head_through = 0;
    tail_adapter = -1;
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(&tmem_, 4 * acc_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();
  wait_for_primary();
  const WaitGuard g{&abort_, status, limit_ns};
  const uint32_t tmem = uniform(tmem_);
  const int tiles = plan.sums[0];
  auto share = [&](int c) { return (int)((int64_t)tiles * c / (int)size); };  // tiles before CTA c's
  const int lo = share(rank), hi = share(rank + 1);
  // steps and runs so far, counted by every role for itself; the step's stage, and its turn of the ring (counted on:
  // a division by the number of stages cost more than the rest of a step)
  int i = 0, run = 0, st = 0;
  uint32_t turn = 0;
  auto next_stage = [&] {
    ++i;
    if (++st == stages) st = 0, ++turn;
  };
  bool before = false, has_head = false, alive = true;
  const int quad = warp & 3, l = 32 * quad + lane;  // (a warp reads the tensor-memory lanes of its number modulo 4)
  auto sums = [&](int acc, int cc, float* v) {  // 32 columns of an accumulator
    const uint32_t at = tmem + acc * acc_cols + ((uint32_t)(32 * quad) << 16) + cc;
    if (beside && rp > 16) {
      tmem_ld32_sum(at, at + rank_cols(rp), v);
    } else {
      tmem_ld32(at, v);
      if (beside) {
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] += v[16 + k];
      }
    }
  };
  auto keep = [&](int acc, unsigned char* to) {
    for (int cc = 0; cc < rp; cc += 32) {
      float v[32];
      sums(acc, cc, v);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (cc + 4 * k < rp)
          *reinterpret_cast<float4*>(to + (((cc >> 2) + k) * TILE + l) * 16) =
              make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
  };
  const uint32_t lower = TILE * 256 + TILE * rank_bytes(rp);  // u's second part in a stage
  for (int b0 = lo, m = 0; b0 < hi; b0 += m) {
    if (b0 > lo) __syncthreads();
    int steps;
    {
      const int ti = b0 + lane;
      Tile t{-1, 0, 0, 0};
      if (ti < tiles) t = plan.tiles[ti];
      int before_it = __shfl_up_sync(0xFFFFFFFFu, t.adapter, 1), behind_it = __shfl_down_sync(0xFFFFFFFFu, t.adapter, 1);
      if (lane == 0) before_it = ti > 0 ? plan.tiles[ti - 1].adapter : -1;
      if (lane == 31) behind_it = ti + 1 < tiles ? plan.tiles[ti + 1].adapter : -1;
      const int up = (t.count + ALIGN - 1) / ALIGN * ALIGN;
      // (tiles that share a step have the same number here: together they end before TILE places from the step's first)
      const int with = up <= SMALL ? t.start / SMALL : -1, with_last = __shfl_up_sync(0xFFFFFFFFu, with, 1);
      const bool opens = lane == 0 || with < 0 || with != with_last;
      uint32_t first = __ballot_sync(0xFFFFFFFFu, ti < hi && opens);
      m = min(BATCH, hi - b0);
      steps = __popc(first);
      if (steps > STEPS) {  // the tiles before the step behind the last
        uint32_t more = first;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) more &= more - 1;
        m = __ffs(more) - 1;
        first ^= more;
        steps = STEPS;
      }
      if (warp == 0 && lane < m) {
        const bool begins = before_it != t.adapter, ends = behind_it != t.adapter;
        const uint32_t behind = first >> lane >> 1;
        part[lane] = make_int4(t.start, up, t.adapter,
                               (begins || ti == lo ? RUN_BEGINS : 0) | (ends || ti + 1 == hi ? RUN_ENDS : 0) |
                                   (!begins && ti == lo ? FROM_BEFORE : 0) | (!ends && ti + 1 == hi ? GOES_ON : 0) |
                                   (opens ? STEP_BEGINS : 0) | (lane + 1 == m || (behind & 1) ? STEP_ENDS : 0));
      }
      constexpr int WARPS = WGRAD_THREADS / 32, MORE = (STEPS + WARPS - 1) / WARPS;
      int from[MORE], n[MORE], row[MORE][4];
#pragma unroll
      for (int q = 0; q < MORE; ++q) {
        uint32_t rest = first;
        for (int k = warp + q * WARPS; k > 0; --k) rest &= rest - 1;
        const int a = rest ? __ffs(rest) - 1 : 0, next = rest & (rest - 1), b = next ? __ffs(next) - 2 : m - 1;
        from[q] = __shfl_sync(0xFFFFFFFFu, t.start, a);
        const int end = __shfl_sync(0xFFFFFFFFu, t.start + up, b);
        n[q] = rest ? end - from[q] : 0;
      }
#pragma unroll
      for (int q = 0; q < MORE; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // (all loads before the first use)
          const int l = SLAB * k + lane;
          row[q][k] = l < n[q] ? plan.rows[from[q] + l] : -1;
        }
#pragma unroll
      for (int q = 0; q < MORE; ++q) {
        const int j = warp + q * WARPS;
        if (j >= steps) break;
        if (lane == 0) step_of[j] = make_int2(from[q], n[q]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int first_row = __shfl_sync(0xFFFFFFFFu, row[q][k], 0);
          const bool box = __all_sync(0xFFFFFFFFu, row[q][k] >= 0 && row[q][k] == first_row + lane);
          row_of[j][SLAB * k + lane] = row[q][k];
          if (lane == 0) box_of[j][k] = box ? first_row : -1;
        }
      }
    }
    __syncthreads();
    if (warp < 4) {
      const int c = lane & 7;
      const bool two = c0 + 64 < C;  // (the second block of 64 columns has some)
      // row by row: the lane's eight columns in either block, and their place in rows 0 to 3 and 4 to 7 of eight
      const bool left = c0 + c * 8 < C, right = c0 + 64 + c * 8 < C;
      const __nv_bfloat16* mine = X + (left ? c0 + c * 8 : 0);
      const uint32_t even = piece(0, lane >> 3, c), odd = piece(0, 4 + (lane >> 3), c) - 512;
      int landing = -1;              // the stage of a step whose rows are still being copied one by one
      auto landed = [&](bool behind) {  // (behind: another step's copies have been issued since)
        if (behind)
          cp_wait<1>();
        else
          cp_wait<0>();
        fence_async_shared();
        __syncwarp();
        if (elect_one()) mbar_arrive(&full[landing]);
        __syncwarp();
        landing = -1;
      };
      int start = uniform(step_of[0].x), count = uniform(step_of[0].y), box = uniform(box_of[0][warp]);
      for (int j = 0; j < steps; ++j) {
        const int from = start, now = count, first = box;
        if (j + 1 < steps) start = uniform(step_of[j + 1].x), count = uniform(step_of[j + 1].y), box = uniform(box_of[j + 1][warp]);
        const uint32_t at = ring + st * stage, dst = at + warp * (SLAB * 128);
        if (turn > 0) alive = alive && warp_wait(&empty[st], (turn - 1) & 1, g);
        if (!alive) break;
        const uint32_t extra = warp == 0 ? TILE * rank_bytes(rp) * (second ? 1 : 2) : 0;
        if (first >= 0) {
          if (elect_one()) {
            mbar_arrive_expect_tx(&full[st], SLAB * 128 * (two ? 2 : 1) + extra);
            if (second) {
              tma_2d(dst, &mx, &full[st], c0, first);
              if (two) tma_2d(dst + TILE * 128, &mx, &full[st], c0 + 64, first);
            } else {  // (x makes room for dy, which is in L2 in part)
              tma_2d_once(dst, &mx, &full[st], c0, first);
              if (two) tma_2d_once(dst + TILE * 128, &mx, &full[st], c0 + 64, first);
            }
          }
        } else if (extra) {
          if (elect_one()) mbar_expect_tx(&full[st], extra);
        }
        if (extra) {
          if (elect_one()) {
            tma_2d(at + TILE * 256, &mu, &full[st], 0, from);
            if (rp > 64) tma_2d(at + TILE * 256 + TILE * 128, &mu, &full[st], 64, from);
            if (!second) {
              tma_2d(at + lower, &mu, &full[st], 0, places + from);
              if (rp > 64) tma_2d(at + lower + TILE * 128, &mu, &full[st], 64, places + from);
            }
          }
        }
        __syncwarp();
        if (first < 0) {
          // row by row, with zeros where there is no row (columns past the last are products that nobody reads)
          const int up = now - SLAB * warp;  // rows of the slab that the MMAs read (a multiple of 16)
          int id[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) id[q] = row_of[j][SLAB * warp + 4 * q + (lane >> 3)];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            if (4 * q >= up) break;
            const __nv_bfloat16* src = mine + (size_t)max(id[q], 0) * C;
            const uint32_t to = dst + (q & 1 ? odd : even) + 512 * q;
            cp16(to, src, id[q] >= 0 && left);
            cp16(to + TILE * 128, right ? src + 64 : src, id[q] >= 0 && right);
          }
          cp_commit();
        }
        if (landing >= 0) landed(first < 0);
        if (first < 0) landing = st;
        next_stage();
      }
      if (landing >= 0) landed(false);
    } else if (warp == 4) {
      const uint32_t urow = rp > 64 ? 128 : rank_bytes(rp);
      const uint32_t idesc = idesc_bf16_f32(TILE, beside ? rank_cols(rp) + rp : rp) | A_MN | B_MN;
      int from = 0;
      for (int j = 0; j < m; ++j) {
        const int start = uniform(part[j].x), up = uniform(part[j].y), flags = uniform(part[j].w);
        if (flags & STEP_BEGINS) {
          from = start;
          alive = alive && warp_wait(&full[st], turn & 1, g);
        }
        if (flags & RUN_BEGINS) before = (flags & FROM_BEFORE) != 0;
        const int acc = before ? 2 : run & 1;
        if (alive && (flags & RUN_BEGINS) && !before && run >= 2) alive = warp_wait(&acc_empty[acc], (run / 2 - 1) & 1, g);
        if (!alive) break;
        tc_fence_after();
        const uint32_t k0 = (start - from) / ALIGN;
        const uint64_t x = sdesc_mnmajor(ring + st * stage, 128, TILE * 128) + (2048 >> 4) * k0;
        const uint64_t u = sdesc_mnmajor(ring + st * stage + TILE * 256, urow, TILE * urow) + urow * k0;
        const uint32_t keep = (flags & RUN_BEGINS) ? 0u : 1u;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < TILE / ALIGN; ++k)
            if (k * ALIGN < up)
              umma_bf16(tmem + acc * acc_cols, x + (2048 >> 4) * k, u + urow * k, idesc, k > 0 ? 1u : keep);
          if (!BESIDE && !second)
#pragma unroll
            for (int k = 0; k < TILE / ALIGN; ++k)
              if (k * ALIGN < up)
                umma_bf16(tmem + acc * acc_cols, x + (2048 >> 4) * k, u + (lower - TILE * 256) / 16 + urow * k, idesc, 1u);
          if (flags & STEP_ENDS) tc_commit(&empty[st]);
          if ((flags & RUN_ENDS) && !before) tc_commit(&acc_full[acc]);
        }
        __syncwarp();
        if ((flags & RUN_ENDS) && !before) ++run;
        if (flags & STEP_ENDS) next_stage();
      }
    } else {
      for (int j = 0; j < m && alive; ++j) {
        const int adapter = part[j].z, flags = part[j].w;
        if (flags & RUN_BEGINS) before = (flags & FROM_BEFORE) != 0;
        if (!(flags & RUN_ENDS)) continue;
        const bool goes_on = (flags & GOES_ON) != 0;
        if (before) {  // (kept in tensor memory)
          has_head = true;
          if (l == 0) head_through = goes_on;
          continue;
        }
        const int acc = run & 1;
        alive = warp_wait(&acc_full[acc], (run / 2) & 1, g);
        if (!alive) break;
        tc_fence_after();
        // to the gradient, or, a run that goes on, to shared memory for the cluster
        if (goes_on) {
          keep(acc, tail);
          if (l == 0) tail_adapter = adapter;
        }
        for (int cc = 0; cc < rp && !goes_on; cc += 32) {
          float v[32];
          sums(acc, cc, v);
          if (c0 + l < C) {
            __nv_bfloat16* out = dP + ((size_t)adapter * r + cc) * C + c0 + l;
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              if (cc + k < r) {
#pragma unroll
                for (int q = 0; q < 8; ++q, out += C) *out = __float2bfloat16_rn(v[k + q]);
              }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[acc]);
        ++run;
      }
    }
  }
  if (warp >= 5 && c0 + 4 * lane < C)  // adapters without rows
    for (int a = rank + size * (warp - 5); a < G; a += 4 * size)
      if (plan.first[a] == plan.first[a + 1])
        for (int j = 0; j < r; ++j) *reinterpret_cast<uint2*>(dP + ((size_t)a * r + j) * C + c0 + 4 * lane) = make_uint2(0, 0);
  if (warp == 4) {
    if (elect_one()) tc_commit(&done);  // (the same lane is elected throughout: its commit covers all that was issued)
    __syncwarp();
    land_mma(&done, 0, g);
  } else if (has_head) {
    land_mma(&done, 0, g);
    tc_fence_after();
    keep(2, head);
  }
  __syncwarp();
  cluster_sync();
  if (warp < 4 && lane == 0 && abort_) settle(full, stages, i);
  __syncwarp();
  if (size > 1 && !abort_) {
    // the runs that cross shares: the one that begins in CTA c, its heads in the next ones up to where it ends
    int adapter[8], through[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < (int)size) {
        adapter[c] = ld_cluster_int(mapa_shared(smem_u32(&tail_adapter), c));
        through[c] = ld_cluster_int(mapa_shared(smem_u32(&head_through), c));
      }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c >= (int)size || adapter[c] < 0) continue;
      uint32_t parts = 0;  // bit d: CTA d holds a head of the run
      bool open = true;
#pragma unroll
      for (int d = 0; d < 8; ++d)
        if (d > c && d < (int)size && open && share(d) < share(d + 1)) {
          parts |= 1u << d;
          open = through[d] != 0;
        }
      const int items = TILE * (r / 4);
      for (int k = threadIdx.x + rank * WGRAD_THREADS; k < items; k += WGRAD_THREADS * size) {
        const int column = k % TILE, q = k / TILE;
        const uint32_t at = (q * TILE + column) * 16;
        float4 s = ld_cluster(mapa_shared(ring + at, c)), v[8];
#pragma unroll
        for (int d = 1; d < 8; ++d)
          v[d] = (parts >> d) & 1 ? ld_cluster(mapa_shared(smem_u32(head) + at, d)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int d = 1; d < 8; ++d) s.x += v[d].x, s.y += v[d].y, s.z += v[d].z, s.w += v[d].w;
        if (c0 + column < C) {
          __nv_bfloat16* out = dP + ((size_t)adapter[c] * r + 4 * q) * C + c0 + column;
          out[0] = __float2bfloat16_rn(s.x);
          out[(size_t)C] = __float2bfloat16_rn(s.y);
          out[(size_t)2 * C] = __float2bfloat16_rn(s.z);
          out[(size_t)3 * C] = __float2bfloat16_rn(s.w);
        }
      }
    }
  }
  tc_fence_before();
  cluster_sync();  // (the others have read this CTA's sums)
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 4 * acc_cols);
  }
}

// ---------------------------------------------------------------------------
// k_expand: y = base + h Q over units of (tile, 128 columns).  Several CTAs per
// SM take jobs of one or two neighbouring units from a counter (a unit whose rows are
// no neighbours takes twice as long as others, one with few rows little less:
// fixed shares by any count left some CTAs working for twice as long as most).
// A CTA multiplies, adds and stores one unit at a time while the next one's
// rows of base are on their way (where shared memory has room for them), and
// the SM's other CTAs fill its waits.
// Warps 0 to 3 load 32 rows each, warp 4 issues the MMAs, all eight add and
// store 32 rows x 64 columns each.
// ---------------------------------------------------------------------------
// two bf16 values and two fp32 ones, added and rounded
__device__ __forceinline__ uint32_t plus(uint32_t b, float x, float y) {
  const float2 s = __fadd2_rn(make_float2(bf16_lo(b), bf16_hi(b)), make_float2(x, y));
  return pack_bf16x2(s.x, s.y);
}
constexpr int EXPAND_THREADS = 256;
// Units in a job: two share the tile's h and its rows' numbers; forward of 8192 x 7168 with rank 16 73.8 us, one by one
// 75.8, threes 74.6; rank 128 95.9, 108.7, 96.3; 4500 x 2880 x 5760 with rank 64 40.7, 43.5, 39.8; 512 rows of 64 adapters
// of rank 16 39.0, 45.8, 38.2 (rank 16 without base ahead).  Ones while every unit has a CTA of its own (300 x 512: 14.2 us,
// twos 15.6).
constexpr int expand_job(int64_t units, int ctas) { return units > ctas ? 2 : 1; }
__host__ __device__ constexpr int expand_q(int rp) { return rp * 256; }
// h's second part: beside the first in shared memory up to rank 32, where three CTAs per SM have room for both; in tensor
// memory above, from where the MMA takes it (two CTAs per SM; in shared memory two and one: 4500 x 2880 x 5760 with rank 64
// 43.5 us, so 40.7; 8192 x 7168 with rank 128 111.6 and 95.9; rank 32 in tensor memory 74.2, so 75.1, but 512 rows of 64
// adapters 45.2 and 39.1).
__host__ __device__ constexpr bool expand_lo_in_tmem(int rp) { return rp > 32; }
// Units of base loaded ahead: where it costs no CTA of an SM (rank 64 at 8192 x 7168 80.8 us, 85.6 without), and up to rank
// 16, where it costs the third one, for adapters with many rows (8192 x 7168 72.4, 73.6 without; 512 rows of 64 adapters
// 43.0 and 38.9).
int expand_ahead(int rp, bool many) { return rp <= 16 ? many : rp > 32 && rp <= 64; }
constexpr int expand_bytes(int rp, int ahead) {
  return (1 + ahead) * TILE * 256 + expand_q(rp) + (expand_lo_in_tmem(rp) ? 1 : 2) * TILE * rank_bytes(rp) + 1024;
}
constexpr int EXPAND_MOST = expand_bytes(64, 1) > expand_bytes(MAX_R, 0) ? expand_bytes(64, 1) : expand_bytes(MAX_R, 0);

template <bool LO_TMEM>
__global__ void __launch_bounds__(EXPAND_THREADS, LO_TMEM ? 2 : 3) k_expand(const __grid_constant__ CUtensorMap mh,
                                                              const __grid_constant__ CUtensorMap mq,
                                                              const __grid_constant__ CUtensorMap mb,
                                                              const __grid_constant__ CUtensorMap my,
                                                              const __grid_constant__ CUtensorMap mb8,
                                                              const __grid_constant__ CUtensorMap my8,
                                                              const __nv_bfloat16* hs, const __nv_bfloat16* base, int N, int r,
                                                              int rp, int ahead, int job, Plan plan, int places,
                                                              __nv_bfloat16* y, uint64_t limit_ns, int32_t* status) {
  extern __shared__ unsigned char smem_[];
  unsigned char* smem = aligned_smem(smem_);
  __shared__ uint64_t rows_in[2], product_in, lo_in, product_out;  // base's rows, h and Q in place; the MMAs' end
  __shared__ int abort_, taken[2];  // (the numbers of the jobs behind the next one, by turns)
  __shared__ uint32_t tmem_;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31, slab = warp & 3, block = warp >> 2;
  constexpr uint32_t tmem_columns = LO_TMEM ? 2 * TILE : TILE;
  const uint32_t at = smem_u32(smem), q_at = at + (1 + ahead) * (TILE * 256), h_at = q_at + expand_q(rp);
  if (threadIdx.x == 0) {
    mbar_init(&rows_in[0], 4 * 32);
    mbar_init(&rows_in[1], 4 * 32);
    mbar_init(&product_in, 1);
    mbar_init(&lo_in, 4);
    mbar_init(&product_out, 1);
    abort_ = 0;
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(&tmem_, tmem_columns);
    tmem_relinquish();
  }
  wait_for_primary();
  const int chunks = (N + TILE - 1) / TILE, per_tile = (chunks + job - 1) / job;
  const int64_t jobs = (int64_t)plan.sums[1] * per_tile;  // in the order (tile, columns); the first are the CTAs' numbers
  auto take = [&] { return (int)gridDim.x + atomicAdd(plan.sums + 2, 1); };
  if (threadIdx.x == 0) taken[1] = take();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();
  const WaitGuard g{&abort_, status, limit_ns};
  const uint32_t tmem = uniform(tmem_);
  const uint32_t idesc = idesc_bf16_f32(TILE, TILE) | B_MN, hrow = rp > 64 ? 128 : rank_bytes(rp);

  // a job: its tile's adapter and place, its chunks (end 0: none), and the warp's slab of the tile
  struct Part {
    int adapter, start, chunk, end;
    Slab s;
  };
  // found in three steps, each with the loads of the one before
  struct Find {
    Tile t;
    int chunk, row;
  };
  auto find_tile = [&](Find& f, int number) {
    f.t = Tile{-1, 0, 0, 0};
    f.chunk = -1;
    if (number < jobs) {
      const int tile = number / per_tile;
      f.t = plan.tiles[tile];
      f.chunk = (number - tile * per_tile) * job;
    }
  };
  auto find_row = [&](Find& f) {
    const int place = SLAB * slab + lane;
    f.row = place < f.t.count ? plan.rows[f.t.start + place] : -1;
  };
  auto part_of = [&](const Find& f) {
    Part p{uniform(f.t.adapter), uniform(f.t.start), uniform(f.chunk), 0, slab_of(f.row)};
    if (p.chunk >= 0) p.end = min(p.chunk + job, chunks);
    p.s.first = uniform(p.s.first);
    p.s.count = uniform(p.s.count);
    return p;
  };
  // the rows of base of one unit; every lane of warps 0 to 3 arrives once
  auto load_rows = [&](const Part& p, int chunk, int buf) {
    const int c0 = chunk * TILE;
    const uint32_t to = at + buf * (TILE * 256) + warp * (SLAB * 128);
    const bool two = c0 + 64 < N;
    uint64_t* bar = &rows_in[buf];
    if (!base || p.s.count == 0) {
      if (elect_one()) mbar_arrive_warp(bar);
    } else if (p.s.box && p.s.count > SLAB / 2) {
      if (elect_one()) {
        mbar_expect_tx(bar, SLAB * 128 * (two ? 2 : 1));
        tma_2d(to, &mb, bar, c0, p.s.first);
        if (two) tma_2d(to + TILE * 128, &mb, bar, c0 + 64, p.s.first);
        mbar_arrive_warp(bar);
      }
    } else {
      // neighbours by eights as boxes, by the first lane of each eight
      const bool near = (p.s.near >> lane) & 1;
      if ((lane & 7) == 0 && near && p.s.row >= 0) {
        mbar_expect_tx(bar, 8 * 128 * (two ? 2 : 1));
        tma_2d(to + lane * 128, &mb8, bar, c0, p.s.row);
        if (two) tma_2d(to + TILE * 128 + lane * 128, &mb8, bar, c0 + 64, p.s.row);
      }
      __syncwarp();
      if (p.s.near == 0xFFFFFFFFu) {
        if (lane == 0) mbar_arrive_warp(bar);
      } else {
        const int c = lane & 15;
        for (uint32_t m = ~p.s.near & 0x01010101u; m; m &= m - 1) {
          const int l0 = __ffs(m) - 1 + (lane >> 4);
#pragma unroll
          for (int l = l0; l < l0 + 8; l += 2) {
            const int id = __shfl_sync(0xFFFFFFFFu, p.s.row, l);
            if (id >= 0 && c0 + c * 8 < N)
              cp16(piece(to + (c >> 3) * (TILE * 128), l, c & 7), base + (size_t)id * N + c0 + c * 8, true);
          }
        }
        cp_arrive(bar);
      }
    }
    __syncwarp();
  };
  auto load_product = [&](const Part& p, int chunk, bool fresh) {  // warp 6, which loads no rows
    if (!elect_one()) return;
    const int c0 = chunk * TILE;
    const bool two = c0 + 64 < N;  // (the second block of 64 columns has some)
    const uint32_t h_bytes = fresh ? (LO_TMEM ? 1 : 2) * TILE * rank_bytes(rp) : 0;
    mbar_arrive_expect_tx(&product_in, rp * 128 * (two ? 2 : 1) + h_bytes);
    if (fresh) {
      tma_2d(h_at, &mh, &product_in, 0, p.start);
      if (rp > 64) tma_2d(h_at + TILE * 128, &mh, &product_in, 64, p.start);
      if (!LO_TMEM) tma_2d(h_at + TILE * rank_bytes(rp), &mh, &product_in, 0, places + p.start);
    }
    tma_3d(q_at, &mq, &product_in, c0, 0, p.adapter);
    if (two) tma_3d(q_at + rp * 128, &mq, &product_in, c0 + 64, 0, p.adapter);
  };

  // h's second part to tensor memory, by warps 0 to 3, 64 elements at a time: read while another product is under way,
  // stored when that is done (zeros past the rank, whose columns the product reads up to rp, and in places without a row)
  uint4 lo[8];
  auto read_lo = [&](const Part& p, int piece0) {
    const uint4* src = reinterpret_cast<const uint4*>(hs + (size_t)(places + p.start + SLAB * slab + lane) * r);
    const int pieces = p.s.row >= 0 ? r / 8 : 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) lo[k] = piece0 + k < pieces ? src[piece0 + k] : make_uint4(0, 0, 0, 0);
  };
  auto store_lo = [&](int piece0) { tmem_st32(tmem + TILE + ((uint32_t)(SLAB * slab) << 16) + 4 * piece0, &lo[0].x); };
  auto rest_of_lo = [&](const Part& p) {
    if (rp > 64) {
      read_lo(p, 8);
      store_lo(8);
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (elect_one()) mbar_arrive(&lo_in);
    __syncwarp();
  };

  Find found, behind;
  find_tile(behind, blockIdx.x);
  find_tile(found, taken[1]);
  find_row(behind);
  find_row(found);
  Part now = part_of(behind), next = part_of(found);
  int chunk = now.chunk, done = 0;  // jobs done
  bool more = now.end > 0;
  int products = 0, buf = 0;
  // the parities of what has been waited for, and of what has been issued: rows by buffer, a bit each (issued by warps 0
  // to 3); products (warp 6) and MMAs (warp 4)
  uint32_t rows_waited = 0, rows_issued = 0, issued = 0, los = 0;  // (los: second parts that warp 4 has waited for)
  if (more) {
    if (warp < 4) load_rows(now, chunk, 0), rows_issued = 1;
    if (warp == 6 && now.adapter >= 0) load_product(now, chunk, true), issued = 1;
    __syncwarp();
    if (LO_TMEM && warp < 4 && now.adapter >= 0) {
      read_lo(now, 0);
      store_lo(0);
      rest_of_lo(now);
    }
  }
  while (more) {
    const bool last = chunk + 1 == now.end;  // of this job
    const bool product = now.adapter >= 0, another = !last || next.end > 0;
    const int c0 = chunk * TILE, next_chunk = last ? next.chunk : chunk + 1;
    const bool first = chunk == now.chunk;
    if (warp == 7 && lane == 0 && first && next.end > 0) taken[done & 1] = take();
    if (last && !first) find_tile(found, next.end > 0 ? taken[done & 1] : 0x7FFFFFFF);
    if (ahead && another && warp < 4) load_rows(last ? next : now, next_chunk, buf ^ 1), rows_issued ^= 2 >> buf;
    const bool fresh_lo = LO_TMEM && last && another && warp < 4 && next.adapter >= 0;
    if (fresh_lo) read_lo(next, 0);
    bool ok = true;
    if (product) {
      if (warp == 4) {
        bool in = warp_wait(&product_in, products & 1, g);
        if (LO_TMEM && first) in = warp_wait(&lo_in, los++ & 1, g) && in;
        tc_fence_after();
        const uint64_t h = sdesc_kmajor(h_at, hrow), q = sdesc_mnmajor(q_at, 128, rp * 128);
        if (in && elect_one()) {  // (if not, the others' wait for the product ends by the abort flag)
#pragma unroll
          for (int k = 0; k < MAX_R / 16; ++k)
            if (16 * k < rp) {
              const uint64_t a = h + ((k >> 2) * (TILE * 128) + 32 * (k & 3)) / 16;
              umma_bf16(tmem, a, q + (2048 >> 4) * k, idesc, k > 0);
              if (LO_TMEM)
                umma_bf16_from_tmem(tmem, tmem + TILE + 8 * k, q + (2048 >> 4) * k, idesc);
              else
                umma_bf16(tmem, a + TILE * rank_bytes(rp) / 16, q + (2048 >> 4) * k, idesc, 1u);
            }
          tc_commit(&product_out);
        }
        issued ^= in;
      }
      __syncwarp();
      ok = wait_on(&product_out, products & 1, g);
      ++products;
    }
    // (h and Q have been read: the next unit's may come)
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (warp == 6 && ok && another && (last ? next : now).adapter >= 0) {
      load_product(last ? next : now, next_chunk, last);
      issued ^= 1;
    }
    __syncwarp();
    if (fresh_lo) {
      tc_fence_after();
      store_lo(0);
    }
    if (last && !first) find_row(found);
    ok &= wait_on(&rows_in[buf], (rows_waited >> buf) & 1, g);
    rows_waited ^= 1 << buf;
    tc_fence_after();
    const int col = c0 + 64 * block;
    const uint32_t mine = at + buf * (TILE * 256) + block * (TILE * 128) + slab * (SLAB * 128);
    const Slab& s = now.s;
    if (__all_sync(0xFFFFFFFFu, ok) && s.count > 0 && col < N) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint4 o[4];
        float v[32];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          o[k] = base ? *reinterpret_cast<const uint4*>(smem + (piece(mine, lane, 4 * half + k) - at)) : make_uint4(0, 0, 0, 0);
        if (product) {  // (base's bits otherwise: a sum would make -0 a 0 and every NaN the same)
          tmem_ld32(tmem + ((uint32_t)(32 * slab) << 16) + 64 * block + 32 * half, v);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float* a = v + 8 * k;
            o[k] = make_uint4(plus(o[k].x, a[0], a[1]), plus(o[k].y, a[2], a[3]), plus(o[k].z, a[4], a[5]), plus(o[k].w, a[6], a[7]));
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(smem + (piece(mine, lane, 4 * half + k) - at)) = o[k];
      }
      fence_async_shared();
      __syncwarp();
      if (s.whole == 0xFFFFFFFFu && s.box) {
        if (elect_one()) {
          tma_store_2d(&my, mine, col, s.first);
          bulk_commit();
        }
      } else if ((lane & 7) == 0 && ((s.whole >> lane) & 1)) {
        tma_store_2d(&my8, mine + lane * 128, col, s.row);
        bulk_commit();
      }
      // (eights that have rows and did not go as boxes)
      for (uint32_t m = ~s.whole & 0x01010101u & (0xFFFFFFFFu >> (32 - s.count)); m; m &= m - 1) {
        const int l0 = __ffs(m) - 1 + (lane >> 3), c = lane & 7;
#pragma unroll
        for (int l = l0; l < l0 + 8; l += 4) {
          const int id = __shfl_sync(0xFFFFFFFFu, s.row, l);
          if (id >= 0 && col + c * 8 < N)
            *reinterpret_cast<uint4*>(y + (size_t)id * N + col + c * 8) =
                *reinterpret_cast<const uint4*>(smem + (piece(mine, l, c) - at));
        }
      }
      bulk_wait_read_all();
    }
    tc_fence_before();
    ok = __syncthreads_and(ok);  // (the unit's rows and its accumulator are free)
    tc_fence_after();
    if (!ok) break;
    chunk = next_chunk;
    if (last) {
      if (first) {
        find_tile(found, next.end > 0 ? taken[done & 1] : 0x7FFFFFFF);
        find_row(found);
      }
      now = next;
      next = part_of(found);
      ++done;
    }
    more = another;
    if (!ahead && another && warp < 4) load_rows(now, chunk, 0), rows_issued ^= 1;
    if (fresh_lo) rest_of_lo(now);
    if (ahead) buf ^= 1;
  }
  cp_wait<0>();
  if (LO_TMEM) tmem_wait_st();
  // (the last phase issued; that of a barrier without one counts as over)
  if (abort_ && lane == 0) {
    if (warp == 0)
      for (int k = 0; k < 2; ++k) land(&rows_in[k], ~(rows_issued >> k) & 1, LAND_NS);
    if (warp == 6) land(&product_in, ~issued & 1, LAND_NS);
  }
  __syncwarp();
  if (warp == 4) land_mma(&product_out, ~issued & 1, g);
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_columns);
  }
}

// ---------------------------------------------------------------------------
// k_rows: few rows, one cluster per row, on the CUDA cores
// ---------------------------------------------------------------------------
constexpr int ROW_THREADS = 256, ROW_COLS = ROW_THREADS / 2;

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

// Every CTA of a row's cluster takes its share of K for h and of the columns
// for y.  A warp computes JB elements of h at a time; for y one half of the
// threads takes the first half of the rank, the other the second, each with the
// first AHEAD rows of Q loaded before h is known.  OCC CTAs per SM.  What bounds
// it are the loads that few CTAs have under way, so the fewer rows, the more
// CTAs per row and loads per thread (rows_kernel).
template <int CTAS, int AHEAD, int JB, int OCC>
__global__ void __launch_bounds__(ROW_THREADS, OCC) k_rows(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ P,
                                                      const __nv_bfloat16* __restrict__ Q, const int32_t* __restrict__ idx,
                                                      const float* __restrict__ scale, const __nv_bfloat16* base, int K,
                                                      int N, int r, int G, __nv_bfloat16* y, __nv_bfloat16* __restrict__ h,
                                                      float* __restrict__ full) {
  __shared__ float sums[CTAS][MAX_R];  // every CTA's sums over its part of K, from all of them
  __shared__ float hid[MAX_R];
  __shared__ float4 other[2][ROW_COLS];
  const int row = blockIdx.x / CTAS, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int a = idx[row];
  const bool has = (unsigned)a < (unsigned)G;  // (of the whole cluster)
  const int K8 = K / 8, k0 = (int)((int64_t)K8 * rank / CTAS), k1 = (int)((int64_t)K8 * (rank + 1) / CTAS);
  const int N8 = N / 8, n0 = (int)((int64_t)N8 * rank / CTAS), n1 = (int)((int64_t)N8 * (rank + 1) / CTAS);
  const int half = threadIdx.x / ROW_COLS, t = threadIdx.x % ROW_COLS;
  const int j0 = half ? r / 2 : 0, j1 = half ? r : r / 2;
  const uint4* q = reinterpret_cast<const uint4*>(Q + (has ? (size_t)a * r * N : 0));
  uint4 qa[AHEAD];
  if (has) {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const uint4* x = reinterpret_cast<const uint4*>(X + (size_t)row * K);
    const uint4* p = reinterpret_cast<const uint4*>(P + (size_t)a * r * K);
    constexpr int WARPS = ROW_THREADS / 32;
    bool begun = false;  // (the other CTAs: their shared memory may be written from then on)
    for (int jb = warp; jb < r; jb += JB * WARPS) {
      float s[JB];
#pragma unroll
      for (int i = 0; i < JB; ++i) s[i] = 0.0f;
#pragma unroll 2
      for (int k = k0 + lane; k < k1; k += 32) {
        const uint4 xv = x[k];
        uint4 pv[JB];
#pragma unroll
        for (int i = 0; i < JB; ++i) pv[i] = jb + i * WARPS < r ? p[(size_t)(jb + i * WARPS) * K8 + k] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < JB; ++i)
          if (jb + i * WARPS < r) s[i] = dot8(xv, pv[i], s[i]);
      }
      if (!begun) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) qa[i] = n0 + t < n1 && j0 + i < j1 ? q[(size_t)(j0 + i) * N8 + n0 + t] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < JB; ++i)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], d);
      if (!begun) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      begun = true;
#pragma unroll
      for (int i = 0; i < JB; ++i)
        if (lane < CTAS && jb + i * WARPS < r)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&sums[rank][jb + i * WARPS]), lane)),
                       "f"(s[i])
                       : "memory");
    }
    // (r >= 8: every warp has had an element)
    cluster_sync();
    if (threadIdx.x < r) {
      float s = 0.0f;
#pragma unroll
      for (int c = 0; c < CTAS; ++c) s += sums[c][threadIdx.x];
      s *= scale[a];
      hid[threadIdx.x] = s;  // (no operand of a tensor core here: not rounded)
      if (h && rank == 0) h[(size_t)row * r + threadIdx.x] = __float2bfloat16_rn(s);
      if (full && rank == 0) full[(size_t)row * r + threadIdx.x] = s;
    }
    __syncthreads();
  } else if (h && rank == 0 && threadIdx.x < r) {
    h[(size_t)row * r + threadIdx.x] = __float2bfloat16_rn(0.0f);
  }
  for (int nb = n0; nb < n1; nb += ROW_COLS) {
    const int n = nb + t;
    const bool mine = n < n1;
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    if (has && mine) {
      if (nb == n0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (j0 + i < j1) add8(s, hid[j0 + i], qa[i]);
      }
#pragma unroll 8
      for (int j = nb == n0 ? j0 + AHEAD : j0; j < j1; ++j) add8(s, hid[j], q[(size_t)j * N8 + n]);
    }
    if (has) {
      if (half) {
        other[0][t] = make_float4(s[0], s[1], s[2], s[3]);
        other[1][t] = make_float4(s[4], s[5], s[6], s[7]);
      }
      __syncthreads();
    }
    if (!half && mine) {
      const uint4 o = base ? reinterpret_cast<const uint4*>(base + (size_t)row * N)[n] : make_uint4(0, 0, 0, 0);
      const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
      if (has) {
        const float4 u = other[0][t], v = other[1][t];
        s[0] += u.x, s[1] += u.y, s[2] += u.z, s[3] += u.w;
        s[4] += v.x, s[5] += v.y, s[6] += v.z, s[7] += v.w;
      }
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = has ? pack_bf16x2(bf16_lo(ow[i]) + s[2 * i], bf16_hi(ow[i]) + s[2 * i + 1]) : ow[i];
      reinterpret_cast<uint4*>(y + (size_t)row * N)[n] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (has) __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// k_row_grads: the adapters' gradients from few rows, on the CUDA cores.  CTA
// (256 columns of x or dy, adapter); its warps take four rows of dP at a time,
// lanes eight columns each, and go over the adapter's rows in their order.  u
// (of k_rows) in fp32.  Bound by the writing of dA and dB, most of them zeros
// as a rule.
// ---------------------------------------------------------------------------
constexpr int GRAD_THREADS = 128, GRAD_COLS = 256, GRAD_ROWS = 64, FEW_ROWS = 4096;

__global__ void __launch_bounds__(GRAD_THREADS, 8) k_row_grads(const __nv_bfloat16* __restrict__ x, const float* __restrict__ u,
                                                               const __nv_bfloat16* __restrict__ dy,
                                                               const __nv_bfloat16* __restrict__ h,
                                                               const int32_t* __restrict__ idx, int T, int K, int N, int r,
                                                               __nv_bfloat16* __restrict__ dA, __nv_bfloat16* __restrict__ dB) {
  __shared__ int rows[GRAD_ROWS], n_;
  __shared__ float us[FEW_ROWS];  // of the adapter's rows, [n][r]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, a = blockIdx.y, units = (K + GRAD_COLS - 1) / GRAD_COLS;
  const bool second = (int)blockIdx.x >= units;
  const __nv_bfloat16* X = second ? dy : x;
  __nv_bfloat16* dP = second ? dB : dA;
  const int C = second ? N : K, col = ((int)blockIdx.x - (second ? units : 0)) * GRAD_COLS + 8 * lane;
  if (warp == 0) {
    int n = 0;
    for (int b = 0; b < T; b += 32) {
      const bool mine = b + lane < T && idx[b + lane] == a;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine);
      if (mine) rows[n + __popc(m & ((1u << lane) - 1))] = b + lane;
      n += __popc(m);
    }
    if (lane == 0) n_ = n;
  }
  __syncthreads();
  wait_for_primary();
  const int n = n_;
  for (int i = threadIdx.x; i < n * r; i += GRAD_THREADS) {
    const size_t at = (size_t)rows[i / r] * r + i % r;
    us[i] = second ? __bfloat162float(h[at]) : u[at];
  }
  __syncthreads();
  if (col >= C) return;
  for (int j = 4 * warp; j < r; j += GRAD_THREADS / 8) {
    float s[4][8] = {};
    for (int q = 0; q < n; q += 4) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (q + i < n) v[i] = *reinterpret_cast<const uint4*>(X + (size_t)rows[q + i] * C + col);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (q + i < n)
#pragma unroll
          for (int k = 0; k < 4; ++k) add8(s[k], us[(q + i) * r + j + k], v[i]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint4*>(dP + ((size_t)a * r + j + k) * C + col) =
          make_uint4(pack_bf16x2(s[k][0], s[k][1]), pack_bf16x2(s[k][2], s[k][3]), pack_bf16x2(s[k][4], s[k][5]),
                     pack_bf16x2(s[k][6], s[k][7]));
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// k_rows for calls of at most so many rows, and rows times rank.  It reads an adapter for each row (from L2, mostly),
// the tiles each adapter once.  us, the tiles behind the stroke, by width (K = N), rows x rank and adapters:
//              256 x 16, 64   256 x 16, 4   128 x 32, 64   64 x 64, 64   64 x 64, 4   32 x 128, 64   32 x 128, 4
//   256        15 / 15        15 / 14       12 / 15        12 / 15       12 / 14      12 / 16        13 / 15
//   1024       15 / 19        15 / 15       12 / 17        12 / 18       12 / 15      13 / 18        13 / 15
//   2880       18 / 25        18 / 16       15 / 23        16 / 25       16 / 16      18 / 22        18 / 17
//   7168       22 / 36        21 / 19       21 / 35        28 / 38       21 / 18      38 / 37        23 / 21
// Above, single rows of many adapters would still be faster here (300 x 16, 64: 26 / 36 at 7168, 21 / 25 at 2880, but 18 / 15
// at 256; 512 x 8, 64: 28 / 44, 24 / 28, 21 / 16), rows of few adapters not; how many rows an adapter has is not known here.
constexpr int MOST_ROWS = 256;
bool few_rows(int T, int r) { return T <= MOST_ROWS && (int64_t)T * r <= FEW_ROWS; }

// k_rows for T rows of rank r, 7168 x 7168, us by CTAs per row, AHEAD, JB, OCC:
//   rows, rank     1, 16   1, 64   1, 128   8, 64   16, 16   16, 64   32, 64   64, 16   128, 16
//   16, 8, 2, 2    4.5     8.7     14.8     10.0    8.4      18.6     27.8     20.5     -
//   16, 4, 4, 2    5.1     8.0     12.5     9.9     10.0     17.2     27.1     23.9     -
//   8, 8, 4, 2     5.8     11.1    19.6     11.1    6.4      12.9     13.3     11.6     -
//   8, 4, 2, 4     5.9     13.3    24.2     13.5    6.4      15.0     15.0     8.2      15.2
//   8, 1, 1, 8     6.6     14.0    24.2     -       7.2      15.6     15.9     8.8      12.9
// A GPC holds one cluster of 16 with another's CTAs beside it; clusters of 8 leave some SMs with less than two CTAs
// (38 rows of rank 64: 8, 8, 4, 2 takes 22.9, 8, 4, 2, 4 17.2).  A rank of 16 has two elements of h per warp.
decltype(&k_rows<8, 1, 1, 8>) rows_kernel(int T, int r, int& ctas) {
  const int sms = sm_count();
  ctas = T * 16 <= sms ? 16 : 8;
  if (ctas == 16) return r <= 16 ? k_rows<16, 8, 2, 2> : k_rows<16, 4, 4, 2>;
  if (T * 9 <= 2 * sms) return k_rows<8, 8, 4, 2>;
  return T * 8 <= 4 * sms ? k_rows<8, 4, 2, 4> : k_rows<8, 1, 1, 8>;
}

// The backward by k_rows and k_row_grads, for few rows per adapter, which a warp goes over one after the other.  us as
// above, 64 rows:
//              rank 16, 64   rank 16, 8   rank 16, 2   rank 64, 64   rank 64, 8   rank 64, 4 (by tiles)
//   256        9 / 25        10 / 20      15 / 19      17 / 27       21 / 22      27 / 22
//   1024       9 / 29        10 / 21      15 / 19      18 / 41       21 / 22      27 / 22
//   2880       12 / 35       11 / 23      16 / 21      31 / 45       26 / 25      31 / 23
//   7168       16 / 52       13 / 29      17 / 24      56 / 90       32 / 32      37 / 27
bool few_grads(int T, int r, int G) {
  return T <= GRAD_ROWS && (int64_t)T * r <= FEW_ROWS && (int64_t)T * r <= 512 * (int64_t)G;
}

// Adapters with many rows each, on average at least.
bool many_rows(int T, int G) { return T >= 64 * (int64_t)G; }

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
int used_groups(int T, int G) { return G + 1 < T ? G + 1 : T; }             // at most, the rows without one among them
int max_tiles(int T, int G) { return T / TILE + used_groups(T, G); }
int places(int T, int G) { return (T / ALIGN + used_groups(T, G)) * ALIGN; }  // of the grouped order, at most

size_t plan_bytes(int T, int G) {
  return 256 + up256((size_t)(G + 2) * 4) + up256((size_t)max_tiles(T, G) * sizeof(Tile)) + up256((size_t)places(T, G) * 4);
}
size_t sorted_bytes(int T, int r, int G) { return up256((size_t)places(T, G) * r * 2); }

Plan plan_at(void* ws, int T, int G) {
  char* p = static_cast<char*>(ws);
  Plan q;
  q.sums = reinterpret_cast<int*>(p);
  p += 256;
  q.first = reinterpret_cast<int*>(p);
  p += up256((size_t)(G + 2) * 4);
  q.tiles = reinterpret_cast<Tile*>(p);
  p += up256((size_t)max_tiles(T, G) * sizeof(Tile));
  q.rows = reinterpret_cast<int*>(p);
  return q;
}

template <class... A, class... B>
moe_status_t launch(void (*k)(A...), dim3 ctas, int cluster, int threads, int smem, int smem_limit, bool dependent,
                    cudaStream_t stream, const B&... args) {
  // (one limit per kernel)
  if (smem_limit && (!set_smem_limit((const void*)k, smem_limit) || !prefer_shared((const void*)k))) return MOE_ERR_CUDA;
  if (cluster > 8 && !allow_large_clusters((const void*)k)) return MOE_ERR_CUDA;
  return launch_kernel(k, ctas, cluster, threads, smem, dependent, stream, args...);
}

using bf = __nv_bfloat16;
const bf* in(const moe_bf16* p) { return reinterpret_cast<const bf*>(p); }
bf* out(moe_bf16* p) { return reinterpret_cast<bf*>(p); }
int pad16(int r) { return (r + 15) & ~15; }

// Tensor maps of a [rows][cols] bf16 matrix in boxes of box_cols x box_rows,
// swizzled over the box's row, and of an adapters' weight [G][r][C].
bool map_rows(CUtensorMap* m, const void* p, int rows, int cols, int box_cols, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {(uint32_t)box_cols, (uint32_t)box_rows};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, box,
                     box_cols == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                     : box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                      : CU_TENSOR_MAP_SWIZZLE_32B);
}
bool map_weight(CUtensorMap* m, const void* p, int G, int r, int C, int rp) {
  const uint64_t dims[3] = {(uint64_t)C, (uint64_t)r, (uint64_t)G}, strides[2] = {(uint64_t)C * 2, (uint64_t)C * 2 * r};
  const uint32_t box[3] = {64, (uint32_t)rp, 1};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

moe_status_t group(const int32_t* idx, int T, int G, const Plan& p, cudaStream_t s) {
  const int most = GROUP_SMEM / 4 / (G + 1), warps = most < 32 ? most : 32;
  return launch(k_group, 1, 0, GROUP_THREADS, warps * (G + 1) * 4, GROUP_SMEM, false, s, idx, T, G, warps, p);
}

// CTAs per cluster that share a contraction of `blocks` stages: as many as the
// SMs hold at once with `clusters` of them (by their shared memory, static and
// dynamic, of which an SM has 228 KB and each CTA takes 1 KB more than it asks
// for), and two stages each at least.
int split_of(int smem, int clusters, int blocks) {
  const int slots = sm_count() * (228 * 1024 / (smem + 1024));

  int s = slots / (clusters > 0 ? clusters : 1);
  if (s > blocks / 2) s = blocks / 2;
  return s < 1 ? 1 : s > 8 ? 8 : s;
}

int shrink_split(int T, int K, int r, int G) { return split_of(shrink_bytes(pad16(r)) + 1024, max_tiles(T, G), (K + KB - 1) / KB); }

moe_status_t shrink(const moe_bf16* x, const moe_bf16* P, const float* scale, int T, int K, int r, int G, const Plan& p,
                    moe_bf16* h, moe_bf16* hs, const moe_bf16* other, moe_bf16* others, int32_t* st, cudaStream_t s) {
  const int rp = pad16(r), tiles = max_tiles(T, G), bytes = shrink_bytes(rp);
  const int split = shrink_split(T, K, r, G);
  CUtensorMap mx, mp;
  if (!map_rows(&mx, x, T, K, 64, SLAB) || !map_weight(&mp, P, G, r, K, rp)) return MOE_ERR_CUDA;
  return launch(k_shrink, tiles * split, split, SHRINK_THREADS, bytes, shrink_bytes(MAX_R), true, s, mx, mp, in(x), scale, K,
                r, rp, p, places(T, G), out(h), out(hs), in(other), out(others), g_wait_limit_ns.load(), st);
}

moe_status_t wgrad(const moe_bf16* x, const moe_bf16* us, int K, moe_bf16* dA, const moe_bf16* dy, const moe_bf16* hs, int N,
                   moe_bf16* dB, int T, int r, int G, const Plan& p, int32_t* st, cudaStream_t s) {
  const int rp = pad16(r), bytes = wgrad_bytes(rp);
  Sides sides;
  auto fill = [&](Side& d, const moe_bf16* X, const moe_bf16* U, int C, moe_bf16* dP) {
    d.X = in(X);
    d.dP = out(dP);
    d.C = C;
    d.units = (C + TILE - 1) / TILE;
    return map_rows(&d.mx, X, T, C, 64, SLAB) && map_rows(&d.mu, U, (U == us ? 2 : 1) * places(T, G), r, rank_cols(rp), TILE);
  };
  if (!fill(sides.of[0], x, us, K, dA) || !fill(sides.of[1], dy, hs, N, dB)) return MOE_ERR_CUDA;
  const int units = sides.of[0].units + sides.of[1].units;
  // (the zeros of adapters without rows, of which there are G - T at least, take about as long as tiles: one row of 51
  // adapters of rank 128, 2440 to 256, 27 us instead of 51)
  const int zeros = G > T ? (int)((int64_t)(G - T) * r / MAX_R) : 0;
  const int split = split_of(bytes + 10 * 1024, units, max_tiles(T, G) + zeros);
  // (8192 x 7168 with 8 adapters of rank 64 61.8 us with BESIDE, 66.2 without; 512 rows of 64 adapters 69 and 58)
  const bool beside = rp <= 64 && many_rows(T, G);
  return launch(beside ? k_wgrad<true> : k_wgrad<false>, units * split, split, WGRAD_THREADS, bytes, wgrad_bytes(MAX_R),
                true, s, sides, r, rp, G, p, places(T, G), g_wait_limit_ns.load(), st);
}

moe_status_t expand(const moe_bf16* hs, const moe_bf16* Q, const moe_bf16* base, int T, int N, int r, int G, const Plan& p,
                    moe_bf16* y, int32_t* st, cudaStream_t s) {
  const int rp = pad16(r), sms = sm_count(), ahead = expand_ahead(rp, many_rows(T, G)), bytes = expand_bytes(rp, ahead);
  if (sms < 1) return MOE_ERR_CUDA;
  const int64_t units = (int64_t)max_tiles(T, G) * ((N + TILE - 1) / TILE);
  const int per_sm = 228 * 1024 / (bytes + 2048) < 3 ? 228 * 1024 / (bytes + 2048) : 3;  // (registers: three)
  const int grid = units < sms * per_sm ? (int)units : sms * per_sm, job = expand_job(units, grid);
  CUtensorMap mh, mq, mb, my, mb8, my8;
  if (!map_rows(&mh, hs, 2 * places(T, G), r, rank_cols(rp), TILE) || !map_weight(&mq, Q, G, r, N, rp) ||
      !map_rows(&mb, base ? base : y, T, N, 64, SLAB) || !map_rows(&my, y, T, N, 64, SLAB) ||
      !map_rows(&mb8, base ? base : y, T, N, 64, 8) || !map_rows(&my8, y, T, N, 64, 8))
    return MOE_ERR_CUDA;
  const bool lo = expand_lo_in_tmem(rp);
  return launch(lo ? k_expand<true> : k_expand<false>, grid, 0, EXPAND_THREADS, bytes, EXPAND_MOST, true, s, mh, mq, mb,
                my, mb8, my8, in(hs), in(base), N, r, rp, ahead, job, p, places(T, G), out(y), g_wait_limit_ns.load(), st);
}

moe_status_t rows_launch(const moe_bf16* x, const moe_bf16* P, const moe_bf16* Q, const int32_t* idx, const float* scale,
                         const moe_bf16* base, int T, int K, int N, int r, int G, moe_bf16* y, moe_bf16* h, float* full,
                         cudaStream_t s) {
  int ctas;
  const auto k = rows_kernel(T, r, ctas);
  return launch(k, T * ctas, ctas, ROW_THREADS, 0, 0, false, s, in(x), in(P), in(Q), idx, scale, in(base), K, N, r, G, out(y),
                out(h), full);
}

bool sizes_ok(int T, int K, int N, int r, int G) {
  return T >= 0 && T <= (1 << 27) && K > 0 && N > 0 && K % 8 == 0 && N % 8 == 0 && K <= (1 << 20) && N <= (1 << 20) && r > 0 &&
         r % 8 == 0 && G > 0;
}

struct Span {
  const void* p;
  size_t n;
};
bool overlaps(const Span& out, std::initializer_list<Span> others) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(out.p);
  for (const Span& o : others) {
    const uintptr_t y = reinterpret_cast<uintptr_t>(o.p);
    if (out.p && o.p && x < y + o.n && y < x + out.n) return true;
  }
  return false;
}

}  // namespace lora
}  // namespace moeglu

using namespace moeglu;
using namespace moeglu::lora;

extern "C" size_t moe_lora_fwd_workspace_size(int T, int r, int G) {
  return T <= 0 || r <= 0 || G <= 0 || few_rows(T, r) ? 0 : plan_bytes(T, G) + sorted_bytes(T, 2 * r, G);
}

extern "C" size_t moe_lora_bwd_workspace_size(int T, int r, int G) {
  if (T <= 0 || r <= 0 || G <= 0) return 0;
  return few_grads(T, r, G) ? up256((size_t)T * r * 4) : plan_bytes(T, G) + sorted_bytes(T, 2 * r, G) + sorted_bytes(T, r, G);
}

extern "C" moe_status_t moe_lora_fwd(const moe_bf16* x, const moe_bf16* A, const moe_bf16* B, const int32_t* idx,
                                     const float* scale, const moe_bf16* base, int T, int K, int N, int r, int G,
                                     moe_bf16* y, moe_bf16* h, void* ws, size_t ws_bytes, int32_t* status,
                                     moe_stream_t stream) {
  if (!sizes_ok(T, K, N, r, G)) return MOE_ERR_ARG;
  if (r > MAX_R || G > MAX_G) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const size_t need = moe_lora_fwd_workspace_size(T, r, G);
  if (!x || !A || !B || !idx || !scale || !y || (need && !ws) || ws_bytes < need) return MOE_ERR_ARG;
  if (!aligned16(x) || !aligned16(A) || !aligned16(B) || !aligned16(base) || !aligned16(y) || !aligned16(h) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u))
    return MOE_ERR_ARG;
  const Span sx{x, (size_t)T * K * 2}, sa{A, (size_t)G * r * K * 2}, sb{B, (size_t)G * r * N * 2}, si{idx, (size_t)T * 4},
      sf{scale, (size_t)G * 4}, sy{y, (size_t)T * N * 2}, sh{h, (size_t)T * r * 2}, other{base == y ? nullptr : base, sy.n};
  if (overlaps(sy, {sx, sa, sb, si, sf, sh, other}) || overlaps(sh, {sx, sa, sb, si, sf, other}))
    return MOE_ERR_ARG;
  const cudaStream_t s = as_stream(stream);
  if (few_rows(T, r)) return rows_launch(x, A, B, idx, scale, base, T, K, N, r, G, y, h, nullptr, s);
  const Plan p = plan_at(ws, T, G);
  auto* hs = reinterpret_cast<moe_bf16*>(static_cast<char*>(ws) + plan_bytes(T, G));
  if (const moe_status_t e = group(idx, T, G, p, s)) return e;
  if (const moe_status_t e = shrink(x, A, scale, T, K, r, G, p, h, hs, nullptr, nullptr, status, s)) return e;
  return expand(hs, B, base, T, N, r, G, p, y, status, s);
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
  if (!dy || !x || !h || !A || !B || !idx || !scale || !dx || !ws ||
      ws_bytes < moe_lora_bwd_workspace_size(T, r, G))
    return MOE_ERR_ARG;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(h) || !aligned16(A) || !aligned16(B) || !aligned16(base) ||
      !aligned16(dx) || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return MOE_ERR_ARG;
  const Span sx{x, (size_t)T * K * 2}, sy{dy, (size_t)T * N * 2}, sh{h, (size_t)T * r * 2}, sa{A, (size_t)G * r * K * 2},
      sb{B, (size_t)G * r * N * 2}, si{idx, (size_t)T * 4}, sf{scale, (size_t)G * 4}, other{base == dx ? nullptr : base, sx.n},
      odx{dx, sx.n}, oda{dA, sa.n}, odb{dB, sb.n};
  if (overlaps(odx, {sx, sy, sh, sa, sb, si, sf, other}) ||
      overlaps(oda, {sx, sy, sh, sa, sb, si, sf, other, odx}) || overlaps(odb, {sx, sy, sh, sa, sb, si, sf, other, odx, oda}))
    return MOE_ERR_ARG;
  if (few_grads(T, r, G)) {
    auto* u = static_cast<float*>(ws);
    if (const moe_status_t e = rows_launch(dy, B, A, idx, scale, base, T, N, K, r, G, dx, nullptr, u, s)) return e;
    const dim3 grid((K + GRAD_COLS - 1) / GRAD_COLS + (N + GRAD_COLS - 1) / GRAD_COLS, G);
    return launch(k_row_grads, grid, 0, GRAD_THREADS, 0, 0, true, s, in(x), u, in(dy), in(h), idx, T, K, N, r, out(dA), out(dB));
  }
  const Plan p = plan_at(ws, T, G);
  auto* us = reinterpret_cast<moe_bf16*>(static_cast<char*>(ws) + plan_bytes(T, G));
  auto* hs = us + sorted_bytes(T, 2 * r, G) / 2;
  if (const moe_status_t e = group(idx, T, G, p, s)) return e;
  if (const moe_status_t e = shrink(dy, B, scale, T, N, r, G, p, nullptr, us, h, hs, status, s)) return e;
  // (the gradients next, while part of dy is in L2; k_expand, whose jobs any CTA takes, then fills the SMs that they leave:
  // 8192 x 7168 with rank 32 122.7 us, rank 128 179; dx before them 122.7 and 184)
  if (const moe_status_t e = wgrad(x, us, K, dA, dy, hs, N, dB, T, r, G, p, status, s)) return e;
  return expand(us, A, base, T, K, r, G, p, dx, status, s);
}
