// MXFP4 weights (OCP microscaling: E2M1 elements, one E8M0 scale per 32 along
// the contraction): the cast from bf16 and the read-back.
//
//   scale byte = floor(log2 amax) - 2 + 127, clamped to [0, 254] (0xFF for a
//   block holding NaN or Inf); element = round to nearest even of
//   v 2^(127 - byte) on {0, .5, 1, 1.5, 2, 3, 4, 6}, saturating.  The scaling
//   is by a power of two, so both roundings are decided exactly.
//
// The weight of a product y = a . W^T is stored as the tensor cores read it:
// W [G][N][K] as codes q [G][N][Kp / 2] (element 2i in the low nibble of byte
// i; rows of Kp = K rounded up to 128 elements, zero codes past K) and scales
// in the block-scaled GEMM's order (moe_mxfp4_scale_bytes).
//
// Memory bound: 2 bytes per element read and 0.53 written, the read-back the
// other way round.  32 x 2880 x 2880 transposed: cast 105 us (6.4 TB/s), read-
// back 117 us (5.7 TB/s).
#include "common.cuh"
#include "host_common.h"

namespace moeglu {
namespace mxfp4 {

constexpr int TILE = 128;                        // rows and columns of a staged tile
constexpr int TILE_BYTES = TILE * TILE * 2;
constexpr int STAGES = 2;
constexpr int CODE_ROW = 64 + 16;                // staged codes of one output row, padded
constexpr int OFF_CODE = STAGES * TILE_BYTES;
constexpr int OFF_SCALE = OFF_CODE + TILE * CODE_ROW;
constexpr int OFF_BARS = OFF_SCALE + TILE * 4;
constexpr int OFF_MISC = OFF_BARS + STAGES * 8;
constexpr int SMEM = OFF_MISC + 16;

// The 32 values of a block -> scale byte and 16 bytes of codes.
__device__ __forceinline__ uint32_t codes8(const float* v, float inv) {
  return e2m1x8(make_float2(v[0] * inv, v[1] * inv), make_float2(v[2] * inv, v[3] * inv),
                make_float2(v[4] * inv, v[5] * inv), make_float2(v[6] * inv, v[7] * inv));
}

// A CTA streams 128 x 128 tiles of src [G][R][C] through two shared-memory
// buffers filled by TMA (thread 0 issues, one mbarrier per buffer; the load
// of a tile is in flight while the one before it is cast).  A tile is exactly
// one 512-byte block of scales.  Elements past R or C arrive as zeros: they
// make the zero codes of the padding.
//   COL = false: blocks along C.  Thread t holds 8 elements of a row (one
//     16-byte shared load), four neighbouring threads share an amax; a row's
//     64 bytes of codes leave from 16 lanes.
//   COL = true: blocks along R (transposed output).  Thread (column pair p,
//     block b) reads 32 words of two columns (consecutive lanes read
//     consecutive words), casts both columns, and the codes leave through
//     shared memory, 64 bytes per output row.
template <bool COL>
__global__ void __launch_bounds__(256) k_mxfp4_cast(const __grid_constant__ CUtensorMap tm, int G, int R, int C,
                                                    uint8_t* __restrict__ q, uint8_t* __restrict__ s, int32_t* status,
                                                    uint64_t wait_ns) {
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t* tcode = sm + OFF_CODE;
  uint8_t* tscale = sm + OFF_SCALE;  // [128 output rows][4 blocks]
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + OFF_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + OFF_MISC);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) {
    for (int st = 0; st < STAGES; ++st) mbar_init(full + st, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm);
  }
  __syncthreads();
  const int N = COL ? C : R, K = COL ? R : C;
  const int row_tiles = (R + TILE - 1) / TILE, col_tiles = (C + TILE - 1) / TILE;
  const int total = G * row_tiles * col_tiles;
  const size_t pitch = (size_t)(K + TILE - 1) / TILE * (TILE / 2);
  const int nt = (N + 255) / 256, kbs = (K + TILE - 1) / TILE;
  auto issue = [&](int i, int st) {
    const int ct = i % col_tiles, rest = i / col_tiles;
    mbar_arrive_expect_tx(full + st, TILE_BYTES);
    tma_load_3d(sm + st * TILE_BYTES, &tm, full + st, ct * TILE, (rest % row_tiles) * TILE, rest / row_tiles);
  };
  if (t == 0)
    for (int st = 0; st < STAGES; ++st)
      if (blockIdx.x + st * gridDim.x < total) issue(blockIdx.x + st * gridDim.x, st);
  WaitGuard guard{abort_flag, status, wait_ns};
  int k = 0;
  for (int i = blockIdx.x; i < total; i += gridDim.x, ++k) {
    const int st = k % STAGES;
    const int ct = i % col_tiles, rest = i / col_tiles;
    const int g = rest / row_tiles, r0 = (rest % row_tiles) * TILE, c0 = ct * TILE;
    const int n0 = COL ? c0 : r0, k0 = COL ? r0 : c0;
    const bool ok = mbar_wait(full + st, (uint32_t)(k / STAGES) & 1u, guard);
    if (__syncthreads_or(ok ? 0 : 1)) break;
    const uint8_t* tile = sm + st * TILE_BYTES;
    if (!COL) {
      const int part = t & 15;
#pragma unroll 4
      for (int it = 0; it < TILE / 16; ++it) {
        const int lr = it * 16 + (t >> 4);
        const uint4 x = *reinterpret_cast<const uint4*>(tile + lr * (TILE * 2) + part * 16);
        uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                              __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
        m = max(m & 0xFFFFu, m >> 16);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const uint32_t sb = e8m0_fp4_from_amax_bits(m << 16);
        const float v[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                            bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
        const uint32_t code = sb == 0xFFu ? 0x77777777u : codes8(v, mx_inv_scale(sb));
        if (n0 + lr < N)
          *reinterpret_cast<uint32_t*>(q + ((size_t)g * N + n0 + lr) * pitch + k0 / 2 + part * 4) = code;
        if ((part & 3) == 0) tscale[lr * 4 + (part >> 2)] = (uint8_t)sb;
      }
    } else {
      const int b = warp >> 1, p = (warp & 1) * 32 + lane;
      const uint8_t* src = tile + (32 * b) * (TILE * 2) + p * 4;
      uint32_t w[32];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        w[j] = *reinterpret_cast<const uint32_t*>(src + j * TILE * 2);
        m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t sb = e8m0_fp4_from_amax_bits(half ? (m & 0xFFFF0000u) : (m << 16));
        const float inv = sb == 0xFFu ? 0.0f : mx_inv_scale(sb);
        uint32_t code[4];
#pragma unroll
        for (int c8 = 0; c8 < 4; ++c8) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(half ? (w[8 * c8 + e] & 0xFFFF0000u) : (w[8 * c8 + e] << 16));
          code[c8] = sb == 0xFFu ? 0x77777777u : codes8(v, inv);
        }
        const int cl = 2 * p + half;
        *reinterpret_cast<uint4*>(tcode + cl * CODE_ROW + 16 * b) = make_uint4(code[0], code[1], code[2], code[3]);
        tscale[cl * 4 + b] = (uint8_t)sb;
      }
    }
    __syncthreads();
    // the buffer is free again: fetch the tile STAGES steps ahead
    if (t == 0 && i + STAGES * gridDim.x < total) issue(i + STAGES * gridDim.x, st);
    if (COL) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int cl = warp * 16 + h * 8 + (lane >> 2), part = lane & 3;
        if (n0 + cl < N)
          *reinterpret_cast<uint4*>(q + ((size_t)g * N + n0 + cl) * pitch + k0 / 2 + part * 16) =
              *reinterpret_cast<const uint4*>(tcode + cl * CODE_ROW + part * 16);
      }
    }
    if (warp == 0) {  // the tile's scale block: lane l writes bytes 16 l .. 16 l + 15
      const uint32_t* ts = reinterpret_cast<const uint32_t*>(tscale);
      const int gi = n0 / TILE;
      uint8_t* dst = s + ((((size_t)g * nt + (gi >> 1)) * kbs + k0 / TILE) * 2 + (gi & 1)) * 512;
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(ts[lane], ts[32 + lane], ts[64 + lane], ts[96 + lane]);
      // the other half of a last column tile that has none: zero scales
      if ((gi & 1) == 0 && n0 + TILE >= N) reinterpret_cast<uint4*>(dst + 512)[lane] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();  // tcode / tscale are rewritten by the next tile
  }
  // after a timeout: let the loads that were issued land before the CTA exits
  if (t == 0 && *abort_flag) {
    volatile int never = 0;
    WaitGuard drain{&never, status, 100000000ull};
    for (int j = k; j < k + STAGES; ++j)
      if (blockIdx.x + j * gridDim.x < total) mbar_wait(full + j % STAGES, (uint32_t)(j / STAGES) & 1u, drain);
  }
}

// W [G][N][K] bf16 back from codes and scales: e2m1 * 2^(byte - 127), exact
// while it is in bf16's range.  A row belongs to `lpr` lanes (a power of two
// up to 32: the row's index arithmetic is then done once), a lane converts 8
// elements at a time (4 bytes in, 16 out), DQ_UNROLL of them in flight.
constexpr int DQ_UNROLL = 4;
__global__ void __launch_bounds__(256) k_mxfp4_dequant(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                       int N, int K, int rows, int lpr, uint4* __restrict__ out) {
  const int k8s = K / 8, nt = (N + 255) / 256, kbs = (K + TILE - 1) / TILE;
  const size_t pitch = (size_t)kbs * (TILE / 2);
  const int sub = threadIdx.x & (lpr - 1), per_cta = 256 / lpr;
  for (int row = blockIdx.x * per_cta + threadIdx.x / lpr; row < rows; row += gridDim.x * per_cta) {
    const int g = row / N, n = row - g * N;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(q + row * pitch);
    const uint8_t* sc = s + (((size_t)g * nt + n / 256) * kbs) * 1024 + (n % 256 / 128) * 512 + 16 * (n % 32) +
                        4 * (n % 128 / 32);
    uint4* dst = out + (size_t)row * k8s;
    for (int k0 = sub; k0 < k8s; k0 += DQ_UNROLL * lpr) {
      uint32_t w[DQ_UNROLL], b[DQ_UNROLL];
#pragma unroll
      for (int u = 0; u < DQ_UNROLL; ++u) {
        const int k8 = k0 + u * lpr;
        w[u] = b[u] = 0;
        if (k8 < k8s) {
          w[u] = __ldg(src + k8);
          b[u] = __ldg(sc + (size_t)(k8 / 16) * 1024 + k8 % 16 / 4);
        }
      }
#pragma unroll
      for (int u = 0; u < DQ_UNROLL; ++u) {
        const int k8 = k0 + u * lpr;
        if (k8 >= k8s) break;
        const float f = e8m0_value(b[u]);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((w[u] >> (8 * j)) & 0xFFu), __NV_E2M1);
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
          o[j] = pack_bf16x2(v.x * f, v.y * f);
        }
        dst[k8] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

}  // namespace mxfp4
}  // namespace moeglu

using namespace moeglu;

extern "C" size_t moe_mxfp4_code_bytes(int G, int N, int K) {
  if (G <= 0 || N <= 0 || K <= 0) return 0;
  return (size_t)G * N * ((K + 127) / 128) * 64;
}

extern "C" size_t moe_mxfp4_scale_bytes(int G, int N, int K) {
  if (G <= 0 || N <= 0 || K <= 0) return 0;
  return (size_t)G * ((N + 255) / 256) * ((K + 127) / 128) * 1024;
}

extern "C" moe_status_t moe_quantize_mxfp4(const moe_bf16* src, int G, int R, int C, int col, uint8_t* q, uint8_t* s,
                                           int32_t* status, moe_stream_t stream) {
  using namespace mxfp4;
  if (!src || !q || !s || G <= 0 || R <= 0 || C <= 0 || (R % 32) || (C % 32)) return MOE_ERR_ARG;
  if (!aligned16(src) || !aligned16(q) || !aligned16(s)) return MOE_ERR_ARG;
  const size_t tiles = (size_t)G * ((R + TILE - 1) / TILE) * ((C + TILE - 1) / TILE);
  if (tiles > (size_t)INT32_MAX / 2) return MOE_ERR_ARG;
  CUtensorMap tm;
  const uint64_t dims[3] = {(uint64_t)C, (uint64_t)R, (uint64_t)G};
  const uint64_t strides[2] = {(uint64_t)C * 2, (uint64_t)R * C * 2};
  const uint32_t box[3] = {TILE, TILE, 1};
  if (!encode_tmap(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, src, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE))
    return MOE_ERR_CUDA;
  const void* kfn = col ? (const void*)k_mxfp4_cast<true> : (const void*)k_mxfp4_cast<false>;
  if (!set_smem_limit(kfn, SMEM)) return MOE_ERR_CUDA;
  const int occ = max(1, max_active_blocks(kfn, 256, SMEM));
  size_t grid = (size_t)sm_count() * occ;
  if (grid == 0) return MOE_ERR_CUDA;
  if (grid > tiles) grid = tiles;
  if (col)
    k_mxfp4_cast<true><<<(int)grid, 256, SMEM, as_stream(stream)>>>(tm, G, R, C, q, s, status, g_wait_limit_ns.load());
  else
    k_mxfp4_cast<false><<<(int)grid, 256, SMEM, as_stream(stream)>>>(tm, G, R, C, q, s, status, g_wait_limit_ns.load());
  count_launch();
  return launch_status();
}

extern "C" moe_status_t moe_dequantize_mxfp4(const uint8_t* q, const uint8_t* s, int G, int N, int K, moe_bf16* out,
                                             moe_stream_t stream) {
  using namespace mxfp4;
  if (!q || !s || !out || G <= 0 || N <= 0 || K <= 0 || (K % 32)) return MOE_ERR_ARG;
  if (!aligned16(q) || !aligned16(out)) return MOE_ERR_ARG;
  const size_t rows = (size_t)G * N;
  if (rows > (size_t)INT32_MAX / 2) return MOE_ERR_ARG;
  int lpr = 4;
  while (lpr < 32 && lpr < K / 8) lpr *= 2;
  const size_t per_cta = 256 / lpr, cap = (size_t)sm_count() * 8;
  size_t grid = (rows + per_cta - 1) / per_cta;
  if (cap == 0) return MOE_ERR_CUDA;
  if (grid > cap) grid = cap;
  k_mxfp4_dequant<<<(int)grid, 256, 0, as_stream(stream)>>>(q, s, N, K, (int)rows, lpr, reinterpret_cast<uint4*>(out));
  count_launch();
  return launch_status();
}
