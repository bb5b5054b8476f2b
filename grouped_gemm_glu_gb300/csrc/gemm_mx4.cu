// Grouped products of MXFP8 rows with MXFP4 weights on tcgen05 CTA pairs:
//   y[rows of e] = a[rows] . W[e]^T   (FC2, or FC1 with the fused activation)
// kind::mxf8f6f4 with E2M1 x E4M3 operands, one E8M0 scale per 32 elements of
// K on each side, fp32 accumulators in tensor memory.
//
// The weight is the MMA's M operand and the rows are its N operand, because
// the weight is what has to be read: an expert with one row costs an N of 32,
// one with hundreds an N of up to 224.  A pair (cluster of two CTAs,
// cta_group::2) computes 256 weight rows x N rows: each CTA holds 128 weight
// rows and half of the N rows in its shared memory, so a 128-wide step of K
// moves 16 + 16 KB into and out of an SM's shared memory where one CTA on a
// 128 x 256 tile moves 16 + 32 KB: at 128 bytes a clock each way more clocks
// than its MMAs take.  (Cutting the tiles of a call of few tiles along K as
// well, with partial sums joined by the last part to arrive, made one token's
// 16 us 31: a part's store, fence and count take longer than its share of K.)
//
// Weights cross HBM and L2 as 4 bits: the TMA unpacks every 16 elements into
// 16 bytes of shared memory (8 of codes, 8 unused), the form in which this MMA
// kind reads 4-bit elements next to 8-bit ones.
//
// An expert's rows (padded to 32) are cut into ceil(blocks / NB) tiles of
// nearly equal numbers of 32-row blocks, so no tile is a sliver.  With NB = 7
// two accumulators of 224 columns and the scales fill the 512 columns of
// tensor memory: a tile is written out while the next one is multiplied.
//
// Two launches: k_mx4_scales gathers the rows' scales of every row tile into
// the order tcgen05.cp consumes (byte 16 l + 4 j + i of 512 = row 32 j + l,
// k sub-block i; [row tile][k-block][XB][512]), k_grouped_mx4 multiplies.  The
// second is launched as a programmatic dependent of the first: its prologue
// runs meanwhile, and only its rows' producer waits (one token 19.1 -> 16.9
// us).  Gathering inside the second kernel, by a warp that wrote each stage's
// scales itself, was several times slower.
//
// Warps (11 per CTA, one CTA per SM, persistent over the tiles):
//   0-7  epilogue (16 of them, each with half the blocks, were slower: 2880 x
//        5760 prompt 664 -> 682 us, 4032 x 224 102 -> 121): warp (q, h) takes the 32 weight rows of lane quarter q and
//        the 32-row groups h, h + 2, ...; a thread owns one output column and
//        32 rows.  GLU: quarters 2i / 2i + 1 hold the input / gate halves of
//        one packed block of 64, the gate warp hands its values over through
//        shared memory
//   8    TMA producer of the weight: tiles and scales of each stage
//   10   TMA producer of the rows: likewise (two issuing warps: the 64-token
//        batch below 61.5 -> 60.5 us); all copies of both CTAs complete on
//        the even CTA's stage barrier
//   9    tensor-memory owner; in the even CTA the MMA issuer: scales into
//        tensor memory (tcgen05.cp), then 4 MMAs of K = 32
// Every wait is bounded (MOE_ERR_TIMEOUT + early exit, never a trap).
//
// Bound: with many rows by the tensor pipe (16384 tokens, top-4, 2880 x 5760
// with bias and clamped SwiGLU: 661 us, 3290 TFLOP/s, in bursts of some tens of
// milliseconds, a k-block of 224 rows in about 460 cycles where its MMAs take
// 448; 760 us, 2860 TFLOP/s, in passes that go on for seconds under the power
// cap), with few by reading the live
// experts' weights (64 tokens, top-8 of 32 experts, 2048 x 7168: 49.8 us, 5.2
// TB/s), with one token by the two launches and one tile's latency (15.6 us,
// where the weights' bytes take 5.2).
#include "common.cuh"
#include "epilogue.cuh"
#include "host_common.h"

namespace moeglu {
namespace gmx4 {

constexpr int BW = 128;             // weight rows per CTA
constexpr int BK = 128;             // elements of K per k-block
constexpr int EPI_WARPS = 8;
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9, ROWS_WARP = 10;
constexpr int THREADS = 11 * 32;
constexpr int W_TILE = BW * BK;                // unpacked
constexpr int W_TX = BW * BK / 2;              // bytes the unpacking load counts
constexpr int KS = 2;                          // k-blocks per stage
constexpr int SCRATCH = 2048;                  // per epilogue warp
constexpr int E_MAX = 1024;
constexpr uint32_t TMEM_COLS = 512;

// NB: 32-row blocks per tile, at most.  7 is what tensor memory takes twice;
// 2 leaves shared memory for 8 k-blocks instead of 6, for calls whose experts
// have few rows: there the weights stream from HBM (64 tokens, top-8 of 32
// experts, 2048 x 7168: 60.5 us with NB = 7, 54.9 with NB = 2).  A stage holds
// KS = 2 k-blocks, so that a barrier round trip, a commit and the scales' two
// copies are paid once for both (one per stage: 54.4 us against 51.8 there,
// and 730 us against 712 for 16384 tokens, top-4, 2880 x 5760, in one run).
template <int NB>
struct Lay {
  static constexpr int NT = 32 * NB;  // rows per tile
  static constexpr int XB = NB > 4 ? 2 : 1;                      // 512-byte scale blocks of the rows
  static constexpr int STAGES = NB > 4 ? 3 : 4;
  static constexpr int X_TILE = (NT / 2 * BK + 1023) / 1024 * 1024;
  static constexpr int STAGE_BYTES = KS * (W_TILE + X_TILE);     // the k-blocks' weight tiles, then their row tiles
  static constexpr int SF_STAGE = KS * (512 + 512 * XB);         // likewise their scales
  static constexpr int OFF_SF = STAGES * STAGE_BYTES;
  static constexpr int OFF_SCRATCH = OFF_SF + STAGES * SF_STAGE;
  static constexpr int OFF_PREF = OFF_SCRATCH + EPI_WARPS * SCRATCH;
  static constexpr int OFF_BARS = OFF_PREF + (3 * E_MAX + 4) * 4;  // prefix, counts, offsets
  static constexpr int NUM_BARS = 2 * STAGES + 5;
  static constexpr int OFF_MISC = OFF_BARS + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = 1024 + OFF_MISC + 64;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(OFF_BARS % 8 == 0 && OFF_SF % 1024 == 0 && OFF_SCRATCH % 16 == 0, "alignment");
  // scale columns of tensor memory: 4 of the weight and 4 XB of the rows per k-block of a stage
  static constexpr uint32_t SFW_COL = 2 * NT, SFX_COL = SFW_COL + 4 * KS;
  static_assert(SFX_COL + 4 * XB * KS <= TMEM_COLS, "tensor memory");
};

struct Args {
  const int32_t* counts;
  const int32_t* offsets;
  int E, N, K, R_cap, n_tiles, num_kb;
  const uint8_t* xs;  // scales of the rows, [R_cap][K/32]
  uint8_t* xs_tiled;  // [row tile][num_kb][XB][512]
  int mt_cap;         // row tiles that fit xs_tiled
  int32_t* status;
  uint64_t wait_ns;
  const uint16_t* bias;    // [E][N] bf16 or null
  const float* row_scale;  // [R_cap] or null
  uint16_t* pre_out;       // [R_cap][N] bf16 or null
  GluParams prm;
  // outputs
  int out_mode, out_N;
  uint8_t* q_row;
  uint8_t* s_row;
  uint8_t* q_col;
  uint8_t* s_col;
  uint16_t* y;
  float* amax;
};

enum Epi { PLAIN = 0, GLU = 1, GLU_L1 = 2, GLU_L2 = 3, GLU_L3 = 4, ELT = 5 };

__device__ __forceinline__ void umma_mxf8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
      : "memory");
}
// In each CTA of the pair: 32 rows x 16 bytes of its own shared memory into 4
// columns of each 32-lane sub-partition of its tensor memory.
__device__ __forceinline__ void tc_cp_32x128b_x4_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

struct Tile {
  int e, n0;      // expert, first weight row of the pair's tile
  int mt;         // row tile (over all experts)
  int row0;       // first row
  int nb, valid;  // 32-row blocks, real rows
};

__device__ __forceinline__ int row_blocks(int count) { return (max(count, 0) + 31) / 32; }

// The experts' row tiles in shared memory: pref[0..E] their exclusive prefix,
// cnt[0..E-1] and off[0..E-1] the counts and offsets.
struct Rows {
  int32_t *pref, *cnt, *off;
};

// Row tile m of expert e, which has mt of them: the first blocks % mt tiles
// have one block more than the others.
__device__ __forceinline__ void row_tile(const Args& a, const Rows& r, int e, int m, int mt, Tile& ti) {
  const int cnt = r.cnt[e], off = r.off[e];
  const unsigned blocks = (unsigned)row_blocks(cnt), base = blocks / (unsigned)mt, more = blocks - base * (unsigned)mt;
  const int b0 = (int)((unsigned)m * base + min((unsigned)m, more));
  const int nb = (int)base + ((unsigned)m < more ? 1 : 0);
  ti.e = e;
  ti.row0 = off + 32 * b0;
  // (offsets and counts are device data: a tile never reaches past the buffers)
  ti.nb = off < 0 ? 0 : max(0, min(nb, (a.R_cap - ti.row0) / 32));
  ti.valid = min(cnt - 32 * b0, 32 * ti.nb);
}

__device__ __forceinline__ int find_expert(const int32_t* pref, int E, int x) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pref[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Tile t of the sequence; e: the expert of a tile before it (every role goes
// through its tiles in order).  A search from scratch and 64-bit divisions
// took each role 2000 to 3000 cycles per tile, a quarter of a tile's time at
// K = 2880.
__device__ __forceinline__ Tile decode(int t, int& e, const Rows& r, const Args& a) {
  while (e + 1 < a.E && r.pref[e + 1] * a.n_tiles <= t) ++e;
  const int first = r.pref[e], mt = r.pref[e + 1] - first;
  const int local = t - first * a.n_tiles;
  // row tiles of one weight tile follow each other (the weight stays in L2)
  const int n = mt == 1 ? local : (int)((unsigned)local / (unsigned)mt), m = local - n * mt;
  Tile ti;
  row_tile(a, r, e, m, mt, ti);
  ti.n0 = n * 2 * BW;
  ti.mt = first + m;
  if (ti.mt >= a.mt_cap) ti.nb = 0;  // (only with counts that exceed the buffers)
  return ti;
}

// The same in every lane, known as such to the compiler.
__device__ __forceinline__ Tile uniform(Tile t) {
  t.e = __shfl_sync(0xFFFFFFFFu, t.e, 0);
  t.n0 = __shfl_sync(0xFFFFFFFFu, t.n0, 0);
  t.mt = __shfl_sync(0xFFFFFFFFu, t.mt, 0);
  t.row0 = __shfl_sync(0xFFFFFFFFu, t.row0, 0);
  t.nb = __shfl_sync(0xFFFFFFFFu, t.nb, 0);
  t.valid = __shfl_sync(0xFFFFFFFFu, t.valid, 0);
  return t;
}
// Whether the phase is over, without waiting for it.
__device__ __forceinline__ uint32_t mbar_peek(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok;
}
// True in one lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// Fills Rows with tiles of at most NB blocks (whole CTA); returns offsets[E].
template <int NB>
__device__ __forceinline__ int build_rows(const Args& a, const Rows& r) {
  const int E = a.E, lane = threadIdx.x & 31;
  const int end_row = __ldg(a.offsets + E);
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const int c = __ldg(a.counts + e);
    r.cnt[e] = c;
    r.off[e] = __ldg(a.offsets + e);
    r.pref[e + 1] = (row_blocks(c) + NB - 1) / NB;
  }
  if (threadIdx.x == 0) r.pref[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int per = (E + 31) / 32;
    const int beg = 1 + lane * per, end = min(E + 1, beg + per);
    int sum = 0;
    for (int i = beg; i < end; ++i) sum += r.pref[i];
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += v;
    }
    int run = incl - sum;
    for (int i = beg; i < end; ++i) {
      run += r.pref[i];
      r.pref[i] = run;
    }
  }
  __syncthreads();
  return end_row;
}

__device__ __forceinline__ void warp_pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

// Whether ok holds in both warps of a pair (which both call this).
__device__ __forceinline__ int both_warps(int ok, int id) {
  int r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n bar.red.and.pred q, %2, 64, p;\n selp.s32 %0, 1, 0, q;\n}\n"
               : "=r"(r)
               : "r"(ok), "r"(id)
               : "memory");
  return r;
}

template <int EPI>
__device__ __forceinline__ float activate(const GluParams& p, float u, float g) {
  if (EPI == GLU_L1) return swiglu_fwd_lean(p, u, g);
  if (EPI == GLU_L2) return swiglu_fwd_lean_clamped(p, u, g);
  if (EPI == GLU_L3) return geglu_fwd_lean(p, u, g);
  return act_fwd(p, u, g);
}

// 16 values of a block on its scale, as E4M3 codes.
__device__ __forceinline__ uint4 codes16(const float* v, uint32_t sb) {
  const float inv = mx_inv_scale(sb);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = sb == 0xFFu ? 0x7F7F7F7Fu
                       : e4m3x2(v[4 * i] * inv, v[4 * i + 1] * inv) |
                             (e4m3x2(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int R>
__device__ __forceinline__ uint32_t amax_bits_of(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) m = max(m, abs_bits(v[i]));
  return m;
}

// 16 rows from r0 of one output column per lane (a warp: 32 neighbouring
// columns, one scale per row, `col` the first) as MXFP8 rows, turned over in
// the warp's 2 KB of shared memory: afterwards a lane has half a row, so a
// row's amax is 16 maxima and one shuffle and its scale is found once (11957
// tokens, top-4, 224 x 4032: 186 us with a warp-wide reduction and the scale
// found in every lane, row by row, 151 like this).
// (A row's 16-byte chunks are permuted by its number: no bank conflicts.)
__device__ __forceinline__ void emit_mx_rows16(const Args& a, const float* o, int col, int r0, int lane,
                                               uint8_t* stage) {
  const size_t N = (size_t)a.out_N;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 16; ++j)
    reinterpret_cast<float*>(stage)[j * 32 + (((lane >> 2) ^ (j & 7)) << 2) + (lane & 3)] = o[j];
  __syncwarp();
  const int row = lane >> 1, half = lane & 1;
  float v[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 x = reinterpret_cast<const float4*>(stage)[row * 8 + ((4 * half + i) ^ (row & 7))];
    v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
  }
  uint32_t m = amax_bits_of<16>(v);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  const uint32_t sb = e8m0_from_amax_bits(m);
  *reinterpret_cast<uint4*>(a.q_row + (size_t)(r0 + row) * N + col + 16 * half) = codes16(v, sb);
  if (half == 0) a.s_row[(size_t)(r0 + row) * (N / 32) + col / 32] = (uint8_t)sb;
}

// Rows r0 .. r0 + R - 1 (R = 16 or 32) of one output column per lane as bf16,
// bf16 plus amax, or MXFP8 rows.  The block is turned over in the warp's 2 KB
// of shared memory, so that it leaves in 16-byte stores (gated 4160 x 960,
// 12283 tokens, bf16: 217 us with 2-byte stores, 211 like this; without a gate
// both take 102 us at 4032 x 224).  The caller's reads of `stage` are complete.
template <int R>
__device__ __forceinline__ void emit_rows(const Args& a, const float* o, int col, int r0, int lane, uint8_t* stage,
                                          Amax& amax_bits) {
  const size_t N = (size_t)a.out_N;
  if (a.out_mode == MOE_OUT_MXFP8) {
#pragma unroll
    for (int i = 0; i < R / 16; ++i) emit_mx_rows16(a, o + 16 * i, col, r0 + 16 * i, lane, stage);
    return;
  }
  __syncwarp();
  // words of two rows of a column: [row pair][32 columns]
  uint32_t* w = reinterpret_cast<uint32_t*>(stage);
#pragma unroll
  for (int j = 0; j < R / 2; ++j) w[j * 32 + lane] = pack_bf16x2(o[2 * j], o[2 * j + 1]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < R / 16; ++i) {
    const int c = lane + 32 * i, p = c >> 2, f = p & 1;  // eight columns 8 (c % 4) of row pair p; odd pairs read their
    const uint4* src = reinterpret_cast<const uint4*>(w + p * 32 + 8 * (c & 3));  // halves in the other order (banks)
    const uint4 x = src[f], y = src[f ^ 1];
    const uint4 lo = f ? y : x, hi = f ? x : y;
    uint16_t* d = a.y + (size_t)(r0 + 2 * p) * N + col + 8 * (c & 3);
    *reinterpret_cast<uint4*>(d) = make_uint4(__byte_perm(lo.x, lo.y, 0x5410), __byte_perm(lo.z, lo.w, 0x5410),
                                              __byte_perm(hi.x, hi.y, 0x5410), __byte_perm(hi.z, hi.w, 0x5410));
    *reinterpret_cast<uint4*>(d + N) = make_uint4(__byte_perm(lo.x, lo.y, 0x7632), __byte_perm(lo.z, lo.w, 0x7632),
                                                  __byte_perm(hi.x, hi.y, 0x7632), __byte_perm(hi.z, hi.w, 0x7632));
  }
  if (a.out_mode == MOE_OUT_NVFP4) {
#pragma unroll
    for (int j = 0; j < R; ++j) amax_bits.plain = max(amax_bits.plain, abs_bits(o[j]));
  }
}

// R rows from r0 of the lane's output column c as (part of) one 32-row block
// of the column-wise MXFP8 copy, whose amax is m.  (The two warps of a gated
// block quantise their own 16 rows; with the input warp doing all 32 rows,
// 16384 tokens, top-4, 2880 x 5760 took 1457 us with both copies, 800 like this.)
template <int R>
__device__ __forceinline__ void emit_col(const Args& a, const float* o, int c, int r0, uint32_t m) {
  const uint32_t sb = e8m0_from_amax_bits(m);
  uint4* dst = reinterpret_cast<uint4*>(a.q_col + (size_t)c * a.R_cap + r0);
#pragma unroll
  for (int i = 0; i < R / 16; ++i) dst[i] = codes16(o + 16 * i, sb);
  if (r0 % 32 == 0) a.s_col[(size_t)c * (a.R_cap / 32) + r0 / 32] = (uint8_t)sb;
}

// Hands an accumulator back to the MMA issuer (a barrier's cluster address).
// Relaxed: what has to come first is this warp's reads of tensor memory, which
// tcgen05.wait::ld and the fence order; a release would wait for the warp's
// stores of the tile as well, 2000 to 3000 cycles per tile.
__device__ __forceinline__ void release_accumulator(uint32_t bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One tile of this CTA: accumulator lane i is weight row n0 + 128 rank + i,
// column j is row row0 + j.  GLU: lane quarters 2i and 2i + 1 hold the input
// and the gate half of one packed block of 64; the two warps swap halves
// through 4 KB of shared memory, so that each computes 16 of the 32 rows.
template <int EPI>
__device__ __forceinline__ void epilogue(const Args& a, const Tile& ti, uint32_t tacc, int q, int h, int lane, int rank,
                                         uint8_t* scratch, float bias, Amax& amax_bits) {
  const int colbase = ti.n0 + rank * BW + q * 32;
  if (colbase >= a.N) return;  // N is a multiple of 64 (gated) or 32: warps that share a block drop out together
  const int col = colbase + lane;
  constexpr bool GATED = EPI >= GLU && EPI <= GLU_L3;
#pragma unroll 1
  for (int g = h; g < ti.nb; g += 2) {
    const int rb = ti.row0 + 32 * g;
    const int nvalid = max(0, min(32, ti.valid - 32 * g));
    float v[32];
    tmem_ld32(tacc + 32 * g, v);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += bias;
    if (nvalid < 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = j < nvalid ? v[j] : 0.0f;
    }
    if (EPI != PLAIN && a.pre_out != nullptr) {
      uint16_t* pp = a.pre_out + (size_t)rb * a.N + col;
#pragma unroll
      for (int j = 0; j < 32; ++j) pp[(size_t)j * a.N] = __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
    }
    if (GATED) {
      float* xs = reinterpret_cast<float*>(scratch);  // [2][16 rows][32 lanes]: to the gate warp, to the input warp
      const bool gate_warp = (q & 1) != 0;
      const int id = 1 + h * 2 + (q >> 1), f = (colbase / 64) * 32;
      warp_pair_sync(id);  // both warps have read what was there
#pragma unroll
      for (int j = 0; j < 16; ++j) xs[((gate_warp ? 16 : 0) + j) * 32 + lane] = v[gate_warp ? j : 16 + j];
      warp_pair_sync(id);
      float o[16];
      const int r0 = rb + (gate_warp ? 16 : 0), live = nvalid - (gate_warp ? 16 : 0);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float m = xs[((gate_warp ? 0 : 16) + j) * 32 + lane];
        o[j] = activate<EPI>(a.prm, gate_warp ? m : v[j], gate_warp ? v[16 + j] : m);
      }
      if (a.row_scale != nullptr) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j < live) o[j] *= __ldg(a.row_scale + r0 + j);
      }
      if (live < 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = j < live ? o[j] : 0.0f;
      }
      // (each warp turns its rows over in the half of the scratch that it has read)
      uint8_t* mine = scratch + (gate_warp ? 0 : 2048);
      emit_rows<16>(a, o, f, r0, lane, mine, amax_bits);
      if (a.q_col != nullptr && a.out_mode == MOE_OUT_MXFP8) {  // the column's other 16 rows are with the other warp
        const uint32_t m = amax_bits_of<16>(o);
        __syncwarp();
        reinterpret_cast<uint32_t*>(mine)[lane] = m;
        warp_pair_sync(id);
        emit_col<16>(a, o, f + lane, r0, max(m, reinterpret_cast<const uint32_t*>(scratch + (gate_warp ? 2048 : 0))[lane]));
      }
    } else {
      if (EPI == ELT) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float rs = (a.row_scale != nullptr && j < nvalid) ? __ldg(a.row_scale + rb + j) : 1.0f;
          v[j] = j < nvalid ? act_fwd(a.prm, v[j], 0.0f) * rs : 0.0f;
        }
      }
      emit_rows<32>(a, v, colbase, rb, lane, scratch + (q & 1) * SCRATCH, amax_bits);
      if (a.q_col != nullptr && a.out_mode == MOE_OUT_MXFP8) emit_col<32>(a, v, col, rb, amax_bits_of<32>(v));
    }
  }
}

// The four scale bytes that start `at` bytes into the rows' scales (4-byte
// aligned base, `total` bytes, a multiple of 4).  At a row's end, bytes of
// the next row may fill the word: no MMA reads them.
__device__ __forceinline__ uint32_t row_scales(const uint8_t* base, size_t at, size_t total) {
  const size_t w = at & ~(size_t)3;
  const int sh = (int)(at & 3) * 8;
  const uint32_t lo = __ldg(reinterpret_cast<const uint32_t*>(base + w));
  if (sh == 0) return lo;
  const uint32_t hi = w + 4 < total ? __ldg(reinterpret_cast<const uint32_t*>(base + w + 4)) : 0u;
  return __funnelshift_r(lo, hi, sh);
}

// One warp per (row tile, k-block).
template <int NB>
__global__ void __launch_bounds__(256) k_mx4_scales(const Args a) {
  constexpr int XB = Lay<NB>::XB;
  __shared__ int32_t sm[3 * E_MAX + 1];
  const Rows r{sm, sm + E_MAX + 1, sm + 2 * E_MAX + 1};
  launch_dependents();
  if (build_rows<NB>(a, r) > a.R_cap) return;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int ks = a.K / 32;
  const size_t total = (size_t)a.R_cap * ks;
  const int items = min(r.pref[a.E], a.mt_cap) * a.num_kb;
  for (int it = blockIdx.x * warps + (threadIdx.x >> 5); it < items; it += gridDim.x * warps) {
    const int mt = it / a.num_kb, kb = it - mt * a.num_kb;
    const int e = find_expert(r.pref, a.E, mt);
    Tile ti;
    row_tile(a, r, e, mt - r.pref[e], r.pref[e + 1] - r.pref[e], ti);
    uint32_t v[4 * XB];
#pragma unroll
    for (int j = 0; j < 4 * XB; ++j)
      v[j] = j < ti.nb ? row_scales(a.xs, (size_t)(ti.row0 + 32 * j + lane) * ks + 4 * kb, total) : 0u;
    uint4* dst = reinterpret_cast<uint4*>(a.xs_tiled + (size_t)it * (512 * XB));
#pragma unroll
    for (int b = 0; b < XB; ++b)
      if (ti.nb > 4 * b) dst[32 * b + lane] = make_uint4(v[4 * b], v[4 * b + 1], v[4 * b + 2], v[4 * b + 3]);
  }
}

template <int EPI, int NB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    k_grouped_mx4(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX64,
                  const __grid_constant__ CUtensorMap tmX32, const __grid_constant__ CUtensorMap tmX16,
                  const __grid_constant__ CUtensorMap tmWs, const __grid_constant__ CUtensorMap tmXs, const Args a) {
  using L = Lay<NB>;
  constexpr int STAGES = L::STAGES, STAGE_BYTES = L::STAGE_BYTES, SF_STAGE = L::SF_STAGE;
  constexpr uint32_t SFW_COL = L::SFW_COL, SFX_COL = L::SFX_COL;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sf = smem + L::OFF_SF;
  uint8_t* scratch_all = smem + L::OFF_SCRATCH;
  int32_t* rows_sm = reinterpret_cast<int32_t*>(smem + L::OFF_PREF);
  const Rows rows{rows_sm, rows_sm + E_MAX + 1, rows_sm + 2 * E_MAX + 1};
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BARS);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = full + 2 * STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);  // warp-uniform for the compiler
  const int E = a.E;
  const int rank = (int)cluster_ctarank();
  const int cl = blockIdx.x >> 1, ncl = gridDim.x >> 1;

  if (warp == PRODUCER_WARP && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, 2 * EPI_WARPS);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_async_shared();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX64);
    tma_prefetch_desc(&tmX32);
    tma_prefetch_desc(&tmX16);
    tma_prefetch_desc(&tmWs);
    tma_prefetch_desc(&tmXs);
  }
  if (warp == MMA_WARP) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  const int end_row = build_rows<NB>(a, rows);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and tensor memory exist before any cross-CTA use
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const bool over = end_row > a.R_cap;
  if (over && threadIdx.x == 0) set_status(a.status, MOE_ERR_CAPACITY);
  const int total = over ? 0 : rows.pref[E] * a.n_tiles;
  WaitGuard guard{abort_flag, a.status, a.wait_ns};

  // The producer's and the MMA issuer's loops are run by their whole warps, in
  // step, and one elected lane issues: the operands of TMA and tcgen05
  // instructions are uniform registers, and in a loop that only one lane runs
  // each of them is moved there one by one (110 to 140 cycles per
  // instruction, 1000 per k-block, measured with the clock).
  if (warp == PRODUCER_WARP || warp == ROWS_WARP) {
    const bool weight = warp == PRODUCER_WARP;
    int stage = 0, e = 0;
    uint32_t phase = 0, issued = 0, issued_parity = 0;
    const uint32_t full0 = mapa_shared(smem_u32(full), 0);
    if (!weight) wait_for_primary();  // the tiled scales of the rows (in every CTA: the grid ends after its primary)
    for (int t = cl; t < total; t += ncl) {
      const Tile ti = uniform(decode(t, e, rows, a));
      if (ti.nb == 0) continue;
      const uint32_t tx = 2u * (KS * W_TX + SF_STAGE) + (uint32_t)(KS * ti.nb * 32 * BK);  // both CTAs' bytes
      const int xrow = ti.row0 + rank * 16 * ti.nb, wrow = ti.e * a.N + ti.n0 + rank * BW;
      const int ws_blk = (ti.e * a.n_tiles + ti.n0 / (2 * BW)) * a.num_kb, xs_row = ti.mt * a.num_kb * L::XB;
      const int r2 = (ti.nb & 4) * 16, r1 = (ti.nb & 6) * 16;
      bool ok = true;
      // (a last stage of fewer k-blocks is filled up with zeros or with blocks that no MMA reads)
      for (int kb = 0; kb < a.num_kb; kb += KS) {
        if (!__all_sync(0xFFFFFFFFu, mbar_peek(empty + stage, phase ^ 1u)) &&
            !__all_sync(0xFFFFFFFFu, mbar_wait(empty + stage, phase ^ 1u, guard))) {
          ok = false;
          break;
        }
        uint8_t* dst = smem + stage * STAGE_BYTES;
        uint8_t* sd = sf + stage * SF_STAGE;
        const uint32_t bar = full0 + 8 * stage;
        if (elect_one()) {
          if (weight) {
            if (rank == 0) mbar_arrive_expect_tx(full + stage, tx);
            tma_load_3d_pair(dst, &tmW, bar, 0, wrow, kb);
            tma_load_3d_pair(sd, &tmWs, bar, 0, rank, ws_blk + kb);
          } else {
            // this CTA's 16 nb rows in boxes of 64, 32 and 16
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
              uint8_t* xd = dst + KS * W_TILE + kk * L::X_TILE;
              const int c = (kb + kk) * BK;
              if (NB >= 4 && (ti.nb & 4)) tma_load_2d_pair(xd, &tmX64, bar, c, xrow);
              if (ti.nb & 2) tma_load_2d_pair(xd + r2 * BK, &tmX32, bar, c, xrow + r2);
              if (ti.nb & 1) tma_load_2d_pair(xd + r1 * BK, &tmX16, bar, c, xrow + r1);
            }
            tma_load_2d_pair(sd + KS * 512, &tmXs, bar, 0, xs_row + L::XB * kb);
          }
        }
        __syncwarp();
        issued |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
    }
    if (rank == 0 && lane == 0 && *abort_flag) {  // let the copies in flight land (they complete on these barriers)
      volatile int never = 0;
      WaitGuard drain{&never, a.status, 100000000ull};
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) mbar_wait(full + s, (issued_parity >> s) & 1u, drain);
    }
  } else if (warp == MMA_WARP) {
    if (rank == 0) {
      int stage = 0, lt = 0, e = 0;
      uint32_t phase = 0;
      for (int t = cl; t < total; t += ncl) {
        const Tile ti = uniform(decode(t, e, rows, a));
        if (ti.nb == 0) continue;
        const int buf = lt & 1;
        const uint32_t aph = (uint32_t)(lt >> 1) & 1u;
        ++lt;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(acc_empty + buf, aph ^ 1u, guard))) break;
        tc_fence_after();
        const uint32_t idesc = idesc_mxf8_e8m0(2 * BW, 32 * ti.nb) | IDESC_A_E2M1;
        const uint32_t d_tmem = tmem_base + (uint32_t)(buf * L::NT);
        bool ok = true;
        uint32_t ready = mbar_peek(full + stage, phase);
        for (int kb = 0; kb < a.num_kb; kb += KS) {
          if (!__all_sync(0xFFFFFFFFu, ready) && !__all_sync(0xFFFFFFFFu, mbar_wait(full + stage, phase, guard))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w_addr = smem_u32(smem) + stage * STAGE_BYTES;
          const uint32_t sf_addr = smem_u32(sf) + stage * SF_STAGE;
          const uint64_t wd = sdesc_kmajor_sw128(w_addr), xd = sdesc_kmajor_sw128(w_addr + KS * W_TILE);
          const uint64_t sd = sdesc_noswizzle(sf_addr, 128);
          const int ksub = (a.K - kb * BK) / 32;  // MMAs of K = 32 left
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
              tc_cp_32x128b_x4_pair(tmem_base + SFW_COL + 4 * kk, sd + (512 >> 4) * kk);
              tc_cp_32x128b_x4_pair(tmem_base + SFX_COL + 4 * L::XB * kk, sd + (512 >> 4) * (KS + L::XB * kk));
              if (NB > 4 && ti.nb > 4)
                tc_cp_32x128b_x4_pair(tmem_base + SFX_COL + 4 * L::XB * kk + 4, sd + (512 >> 4) * (KS + L::XB * kk + 1));
            }
#pragma unroll
            for (int k = 0; k < 4 * KS; ++k)
              if (k < ksub)
                umma_mxf8_pair(d_tmem, wd + (W_TILE >> 4) * (k / 4) + 2 * (k % 4), xd + (L::X_TILE >> 4) * (k / 4) + 2 * (k % 4),
                               idesc_with_sf_ids(idesc, (uint32_t)(k % 4), (uint32_t)(k % 4)),
                               tmem_base + SFW_COL + 4 * (k / 4), tmem_base + SFX_COL + 4 * L::XB * (k / 4),
                               (kb | k) != 0 ? 1u : 0u);
            tc_commit_pair_mc(empty + stage, 0x3);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          ready = mbar_peek(full + stage, phase);  // the next stage, while this one is multiplied
        }
        if (!ok) break;
        if (elect_one()) tc_commit_pair_mc(acc_full + buf, 0x3);
        __syncwarp();
      }
      // (the same lane is elected throughout: its commit covers everything issued)
      if (elect_one()) tc_commit_pair_mc(mma_done, 0x1);
      __syncwarp();
      volatile int never = 0;
      WaitGuard drain{&never, a.status, 100000000ull};
      mbar_wait(mma_done, 0, drain);
    }
  } else {
    const int q = warp & 3, h = warp >> 2;
    Amax amax_bits{0u, 0u};
    int lt = 0, e = 0;
    // With few rows the next tile and its bias are fetched before a tile is
    // written out (one token 16.0 -> 15.6 us; with NB = 7 the same made products
    // with a short K 4% slower).
    constexpr bool AHEAD = NB <= 4;
    Tile next;
    uint16_t next_bias;
    auto fetch = [&](int t) {
      next.nb = 0;
      next_bias = 0;
      if (t >= total) return;
      next = decode(t, e, rows, a);
      const int col = next.n0 + rank * BW + q * 32 + lane;
      if (a.bias != nullptr && col < a.N) next_bias = __ldg(a.bias + (size_t)next.e * a.N + col);
    };
    if (AHEAD) fetch(cl);
    for (int t = cl; t < total; t += ncl) {
      if (!AHEAD) fetch(t);
      const Tile ti = next;
      const float bias = bf16_lo(next_bias);
      if (AHEAD) fetch(t + ncl);
      if (ti.nb == 0) continue;
      const int buf = lt & 1;
      const uint32_t aph = (uint32_t)(lt >> 1) & 1u;
      ++lt;
      int ok = 1;
      if (lane == 0) ok = mbar_wait(acc_full + buf, aph, guard) ? 1 : 0;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      // the two warps that share a block meet at barriers below: both go on or neither does
      if (EPI >= GLU && EPI <= GLU_L3) ok = both_warps(ok, 1 + h * 2 + (q >> 1));
      if (!ok) break;
      tc_fence_after();
      epilogue<EPI>(a, ti, tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * L::NT), q, h, lane, rank,
                    scratch_all + (warp & ~1) * SCRATCH, bias, amax_bits);
      release_accumulator(mapa_shared(smem_u32(acc_empty + buf), 0), lane);
    }
    if (a.out_mode == MOE_OUT_NVFP4 && a.amax != nullptr) {
      const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, amax_bits.plain);
      if (lane == 0 && m != 0) atomicMax(reinterpret_cast<int*>(a.amax), (int)m);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still touch its memory
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

struct Maps {
  CUtensorMap w, x64, x32, x16, ws, xs;
};

template <int EPI, int NB>
static moe_status_t launch_nb(const Maps& m, const Args& a, int sm_margin, cudaStream_t stream) {
  using L = Lay<NB>;
  const void* kfn = (const void*)k_grouped_mx4<EPI, NB>;
  if (!set_smem_limit(kfn, L::SMEM_BYTES)) return MOE_ERR_CUDA;
  const int sms = sm_count();
  int clusters = max_active_pairs(kfn, THREADS, L::SMEM_BYTES);
  if (clusters <= 0 || sms <= 0) return MOE_ERR_CUDA;
  const int by_margin = (sms - sm_margin) / 2;
  if (clusters > by_margin) clusters = by_margin;
  const long long tiles_bound = (long long)a.mt_cap * a.n_tiles;
  if (clusters > tiles_bound) clusters = (int)tiles_bound;
  if (clusters < 1) clusters = 1;
  const long long items = ((long long)a.mt_cap * a.num_kb + 7) / 8;
  k_mx4_scales<NB><<<(int)(items < 8ll * sms ? items : 8ll * sms), 256, 0, stream>>>(a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = L::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k_grouped_mx4<EPI, NB>, m.w, m.x64, m.x32, m.x16, m.ws, m.xs, a) != cudaSuccess)
    return MOE_ERR_CUDA;
  count_launch(2);
  return launch_status();
}

// Few rows per expert: at most FEW of them on average over the buffers, which
// hold up to 31 rows of padding per expert.  32 experts, 2880 x 5760 gated: 61
// us with NB = 2 against 70 with 7 at 64 rows each, 94 against 73 at 96; 2048 x
// 7168: 51 against 57 and 79 against 60.  The counts are device data, so
// R_cap has to stand for them.  Where one expert has a quarter of the rows, its
// many low tiles read the weight again: 64 experts, 2048 x 7168, 32 rows each on
// average 108 us with NB = 2 against 111, 48 121 against 117, 64 132 against
// 122; 32 experts, 2880 x 5760 gated 67 against 70, 75 against 77, 83 against
// 78.  Buffers larger than the rows need take NB = 7 and lose the first
// figures' 12 to 15%.
constexpr int FEW = 96;
static bool few_rows(int E, int R_cap) { return R_cap <= (long long)FEW * E; }

template <int EPI>
static moe_status_t launch(const Maps& m, const Args& a, int sm_margin, cudaStream_t stream) {
  return few_rows(a.E, a.R_cap) ? launch_nb<EPI, 2>(m, a, sm_margin, stream) : launch_nb<EPI, 7>(m, a, sm_margin, stream);
}

// Row tiles a call can have: at most one partly filled tile per expert.
static int row_tiles_cap(int E, int R_cap) { return R_cap / (few_rows(E, R_cap) ? Lay<2>::NT : Lay<7>::NT) + E; }
static int scale_blocks(int E, int R_cap) { return few_rows(E, R_cap) ? Lay<2>::XB : Lay<7>::XB; }

}  // namespace gmx4

size_t grouped_gemm_mxfp4_workspace(int E, int K, int R_cap) {
  return (size_t)gmx4::row_tiles_cap(E, R_cap) * ((K + gmx4::BK - 1) / gmx4::BK) * gmx4::scale_blocks(E, R_cap) * 512;
}

// See host_common.h.  The entry points (gemm_mx.cu) have checked the arguments.
moe_status_t grouped_gemm_mxfp4(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws,
                                const int32_t* counts, const int32_t* offsets, int E, int K, int N, int R_cap,
                                const moe_glu_params_t* params, const moe_bf16* bias, const float* row_scale,
                                int out_mode, const moe_act_out_t* out, void* work, size_t work_bytes, int sm_margin,
                                int32_t* status, cudaStream_t stream) {
  using namespace gmx4;
  const int n_tiles = (N + 2 * BW - 1) / (2 * BW), num_kb = (K + BK - 1) / BK, mt_cap = row_tiles_cap(E, R_cap);
  const int xb = scale_blocks(E, R_cap);
  if (!work || (reinterpret_cast<uintptr_t>(work) & 255) || work_bytes < grouped_gemm_mxfp4_workspace(E, K, R_cap))
    return MOE_ERR_ARG;
  if ((long long)E * n_tiles * num_kb * 2 > INT32_MAX || (long long)E * N > INT32_MAX - 256 || (long long)mt_cap * num_kb * 2 > INT32_MAX ||
      (long long)mt_cap * n_tiles > INT32_MAX)
    return MOE_ERR_ARG;
  Maps m;
  {
    // the unpacking load wants whole 128-element boxes and 32-byte row pitches
    const uint64_t kp = (uint64_t)(K + BK - 1) / BK * BK;
    // as [k-block][row of any expert][128 elements]: rows past an expert's last are the next one's (or zeros),
    // and no output is stored for them
    const uint64_t dims[3] = {BK, (uint64_t)E * N, kp / BK};
    const uint64_t strides[2] = {kp / 2, BK / 2};
    const uint32_t box[3] = {BK, BW, (uint32_t)KS};
    if (!encode_tmap(&m.w, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, wq, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B))
      return MOE_ERR_CUDA;
  }
  CUtensorMap* xmaps[3] = {&m.x64, &m.x32, &m.x16};
  for (int i = 0; i < 3; ++i) {
    const uint64_t dims[2] = {(uint64_t)K, (uint64_t)R_cap};
    const uint64_t strides[1] = {(uint64_t)K};
    const uint32_t box[2] = {BK, 64u >> i};
    if (!encode_tmap(xmaps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, xq, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return MOE_ERR_CUDA;
  }
  {  // scale blocks as rows of 128 words: the weight's [expert, tile and k-block][half], the rows' in one run
    const uint64_t dims[3] = {128, 2, (uint64_t)E * n_tiles * num_kb};
    const uint64_t strides[2] = {512, 1024};
    const uint32_t box[3] = {128, 1, (uint32_t)KS};
    if (!encode_tmap(&m.ws, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, ws, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE))
      return MOE_ERR_CUDA;
    const uint64_t xdims[2] = {128, (uint64_t)mt_cap * num_kb * xb};
    const uint64_t xstrides[1] = {512};
    const uint32_t xbox[2] = {128, (uint32_t)(xb * KS)};
    if (!encode_tmap(&m.xs, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, work, xdims, xstrides, xbox, CU_TENSOR_MAP_SWIZZLE_NONE))
      return MOE_ERR_CUDA;
  }
  Args a{};
  a.counts = counts;
  a.offsets = offsets;
  a.E = E;
  a.N = N;
  a.K = K;
  a.R_cap = R_cap;
  a.n_tiles = n_tiles;
  a.num_kb = num_kb;
  a.xs = xs;
  a.xs_tiled = static_cast<uint8_t*>(work);
  a.mt_cap = mt_cap;
  a.status = status;
  a.wait_ns = g_wait_limit_ns.load();
  a.bias = reinterpret_cast<const uint16_t*>(bias);
  a.row_scale = row_scale;
  a.pre_out = reinterpret_cast<uint16_t*>(out->pre);
  a.out_mode = out_mode;
  a.q_row = out->q_row;
  a.s_row = out->s_row;
  a.q_col = out->q_col;
  a.s_col = out->s_col;
  a.y = reinterpret_cast<uint16_t*>(out->y);
  a.amax = out->amax;
  if (out_mode == MOE_OUT_NVFP4 && a.amax && cudaMemsetAsync(a.amax, 0, sizeof(float), stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (!params) {
    a.out_N = N;
    return launch<PLAIN>(m, a, sm_margin, stream);
  }
  const int lean = glu_lean_kind(params);
  a.prm = GluParams{params->act,   params->alpha, params->up_offset, params->gate_lo, params->gate_hi,
                    params->up_lo, params->up_hi, lean,              -params->alpha * 1.4426950408889634f};
  if (params->act == MOE_ACT_SRELU) {
    a.out_N = N;
    return launch<ELT>(m, a, sm_margin, stream);
  }
  a.out_N = N / 2;
  return lean == 1   ? launch<GLU_L1>(m, a, sm_margin, stream)
         : lean == 2 ? launch<GLU_L2>(m, a, sm_margin, stream)
         : lean == 3 ? launch<GLU_L3>(m, a, sm_margin, stream)
                     : launch<GLU>(m, a, sm_margin, stream);
}

}  // namespace moeglu

extern "C" size_t moe_grouped_mxfp4_workspace_size(int E, int K, int R_cap) {
  if (E <= 0 || K <= 0 || R_cap <= 0) return 0;
  return moeglu::grouped_gemm_mxfp4_workspace(E, K, R_cap);
}
