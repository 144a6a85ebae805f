// fp8.cu -- linear layers in 8-bit floating point (include/moe_fp8.h).
//
// Mathematics: with 128 inputs to a block b,
//     out[t][n] = sum_b (xs[t][b] ws[n/128][b]) sum_{k in b} xq[t][k] w[n][k].
// The inner sums are products of e4m3 codes on the tensor cores
// (tcgen05.mma kind::f8f6f4, fp32 accumulators in tensor memory, one fresh
// accumulator per block); the outer sum adds the scaled block sums in fp32
// registers.
//
// Layout: 128 outputs (weight rows) are the MMA's M, so a tile's weight scale
// is one number per block; BN rows of x are its N.  Few rows of x thus leave
// no tensor-core row idle, and the weights, which bound that case, are read
// once.  Roles: one warp loads (TMA tiles of w, bulk copies of x), one issues
// the MMAs, one multiplies the scales of each block into shared memory, four
// or eight read the accumulators.  There are four accumulators in tensor
// memory, so the MMAs of the next blocks run while a block is scaled.  More
// than 128 rows go to pairs of SMs, below.
//
// Bound: reading w for few rows, the tensor cores' round trip for many.  With
// fewer tiles than SMs a cluster of 2 or 4 CTAs splits the blocks of a tile and
// joins its partial sums through distributed shared memory in rank order.
// Measured: 16 x 131072 x 7168 to fp32 146 to 154 us (6.2 to 6.5 TB/s, 91 to
// 95% of the measured copy rate; 1024 tiles on 152 SMs leave the last round a
// quarter empty); 1 x 2048 x 2048 5.4 us and 77 x 7000 x 2003 10.9 us a call in
// a graph; 4096 x 7168 x 7168 177 us (2380 TFLOP/s, 127% of the measured bf16
// rate).
#include <cmath>
#include <cstdint>
#include <new>

#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/moe_fp8.h"
#include "common.cuh"
#include "elem.cuh"
#include "tcgen05.cuh"

namespace moe {
int reportf(int code, const char* fmt, ...);

namespace {

namespace cg = cooperative_groups;

constexpr int kBlk = 128;              // inputs per scale block, and outputs per tile
constexpr int kTileW = kBlk * kBlk;    // bytes of a weight tile
constexpr int kScaleRing = 8;          // blocks of prepared scales
constexpr int kMaxSplit = 4;           // CTAs that share a tile
constexpr size_t kCtlBytes = 256;      // control words at the workspace's start ([0] error bits)
constexpr int kMaxRows = 1 << 20;
constexpr uint32_t kMagic = 0x4D6F4638u;

// Workspace: control words, xs [blocks][rows_pad] floats, then the codes of x
// as tiles [row tile of bn][block][bn rows x 128 bytes], each in the 128-byte
// swizzled order the tensor core reads (16-byte piece p of row r at
// r * 128 + ((p ^ (r & 7)) << 4)), so a plain bulk copy loads a tile; for pairs
// of SMs as rows of whole blocks, which tiled loads bring into that order.
struct Layout {
  int bn, row_tiles, rows_pad, blocks;
  size_t xs, codes, bytes;
};

int widest_tile(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256; }

// How a product is cut: rows of x in a tile, and CTAs of a cluster that share
// a tile's blocks.
struct Cut {
  int bn, split;
};

// Where the widest tiles of up to 128 rows leave SMs idle: the cut with the
// most CTAs that still run at once, the wider of equals (77 x 7000 x 2003:
// 128 rows split in 2, 11.1 us, against 64 rows, 13.1; 128 x 2048 x 7168: 64
// rows split in 4, 12.7 us, against 128 rows split in 4, 13.8).  Clusters of
// 8 do not fill the SMs: sixteen of them ran one after the other (1 x 2048 x
// 2048: 7.9 us, split in 4 5.4).  Else the widest tile, so that weights are
// read for 256 rows (fp8_pair_kernel; 512 x 7168 x 7168: 30.3 us, with 128 rows
// 55.6).
Cut cut_of(int rows, int n, int k, int num_sms) {
  const int64_t tiles_n = (n + kBlk - 1) / kBlk, blocks = (k + kBlk - 1) / kBlk;
  Cut best = {widest_tile(rows), 1};
  int64_t most = 0;
  for (int bn = best.bn < 128 ? best.bn : 128; bn >= 16; bn /= 2) {
    const int64_t tiles = (rows + bn - 1) / bn * tiles_n;
    if (tiles > num_sms) break;
    int split = 1;
    while (split < kMaxSplit && tiles * split * 2 <= num_sms && split * 2 <= blocks) split *= 2;
    if (tiles * split > most) most = tiles * split, best = {bn, split};
  }
  return best;
}

Layout layout_of(int rows, int bn, int k) {
  Layout l;
  l.bn = bn;
  l.row_tiles = (rows + l.bn - 1) / l.bn;
  l.rows_pad = l.row_tiles * l.bn;
  l.blocks = (k + kBlk - 1) / kBlk;
  l.xs = kCtlBytes;
  l.codes = (l.xs + sizeof(float) * static_cast<size_t>(l.blocks) * l.rows_pad + 1023) / 1024 * 1024;
  l.bytes = l.codes + static_cast<size_t>(l.blocks) * l.rows_pad * kBlk;
  return l;
}

// ---- quantisation of x -----------------------------------------------------------

struct QuantArgs {
  const void* x;
  int64_t ld;
  int type, rows, k, blocks, rows_pad, bn_log2, vec;
  int plain;  // codes as rows of blocks * 128 bytes, for tiled loads, instead of as tiles
  float* xs;
  uint8_t* codes;
};

// The scale of a block whose largest |x| has these bits: the smallest power
// of two s >= 2^-126 with max <= 448 s (448 = 1.75 * 2^8), 1 for zeros, NaN
// if there is an infinity or a NaN.  `inv` is 1 / s (0 for NaN).
__device__ __forceinline__ float block_scale(uint32_t max_bits, float& inv) {
  if (max_bits == 0) return inv = 1.0f;
  if (max_bits >= 0x7F800000u) {
    inv = 0.0f;
    return __uint_as_float(0x7FC00000u);
  }
  int p = static_cast<int>(max_bits >> 23) - 127 - ((max_bits & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  p = max(p, -126);
  inv = __uint_as_float(static_cast<uint32_t>(127 - p) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + p) << 23);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The codes of 16 inputs (piece `piece` of block b of a row) and the block's
// scale, which the eight threads of the block share.  All lanes take part;
// `in`: this thread has inputs.
__device__ __forceinline__ uint4 quantize_piece(const QuantArgs& q, bool in, int row, int b, int piece, float& scale) {
  const int j = b * kBlk + piece * 16;
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  if (in) {
    const int64_t at = static_cast<int64_t>(row) * q.ld;
    if (q.vec && j + 16 <= q.k) {
      float a[8], c[8];
      load8(q.x, q.type, at + j, a);
      load8(q.x, q.type, at + j + 8, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = a[i], v[8 + i] = c[i];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (j + i < q.k) v[i] = load_elem(q.x, q.type, at + j + i);
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float inv;
  scale = block_scale(m, inv);
  return make_uint4(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv),
                    e4m3x4(v[8] * inv, v[9] * inv, v[10] * inv, v[11] * inv),
                    e4m3x4(v[12] * inv, v[13] * inv, v[14] * inv, v[15] * inv));
}

// Eight threads per (row, block), 16 inputs each.  At most 2^20 rows of 512
// blocks: a unit's index fits 32 bits.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantArgs q) {
  pdl_launch_dependents();
  const uint32_t unit = blockIdx.x * 32u + (threadIdx.x >> 3), blocks = static_cast<uint32_t>(q.blocks);
  const int piece = threadIdx.x & 7;
  const bool in = unit < static_cast<uint32_t>(q.rows) * blocks;
  const int row = in ? static_cast<int>(unit / blocks) : 0, b = in ? static_cast<int>(unit - row * blocks) : 0;
  float s;
  const uint4 w = quantize_piece(q, in, row, b, piece, s);
  if (!in) return;
  if (q.plain) {
    *reinterpret_cast<uint4*>(q.codes + (static_cast<size_t>(row) * blocks + b) * kBlk + piece * 16) = w;
  } else {
    const int tile = row >> q.bn_log2, r = row - (tile << q.bn_log2);
    uint8_t* t = q.codes + (((static_cast<size_t>(tile) * blocks + b) * kBlk) << q.bn_log2);
    *reinterpret_cast<uint4*>(t + r * kBlk + ((piece ^ (r & 7)) << 4)) = w;
  }
  if (piece == 0) q.xs[static_cast<size_t>(b) * q.rows_pad + row] = s;
}

// One 128 x 128 block of weights per thread block.
__global__ void __launch_bounds__(256) quantize_weights_kernel(const void* w, int type, int64_t ld, int n, int k,
                                                               uint8_t* codes, int64_t ldc, float* scales) {
  __shared__ uint32_t wmax[8];
  const int nb = blockIdx.y, kb = blockIdx.x;
  uint32_t m = 0;
  for (int i = threadIdx.x; i < kBlk * kBlk; i += 256) {
    const int r = nb * kBlk + i / kBlk, c = kb * kBlk + i % kBlk;
    if (r < n && c < k) m = max(m, __float_as_uint(load_elem(w, type, r * ld + c)) & 0x7FFFFFFFu);
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, wmax[i]);
  // 0 if there is nothing, or nothing that the quotient can tell from it (up to
  // 224 units of 2^-149): such a block's codes are zeros
  const float quotient = __uint_as_float(m) / 448.0f, s = quotient > 0.0f ? quotient : 1.0f;
  if (threadIdx.x == 0) scales[static_cast<size_t>(nb) * gridDim.x + kb] = s;
  for (int i = threadIdx.x; i < kBlk * kBlk; i += 256) {
    const int r = nb * kBlk + i / kBlk;
    const int64_t c = static_cast<int64_t>(kb) * kBlk + i % kBlk;
    if (r >= n || c >= ldc) continue;
    const float v = c < k ? load_elem(w, type, r * ld + c) / s : 0.0f;
    codes[r * ldc + c] = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
  }
  // the last blocks of a row: zeros from their end to the row's, 16 bytes at a
  // time (codes and ldc are multiples of 16)
  const int64_t end = static_cast<int64_t>(kb + 1) * kBlk;
  if (kb == static_cast<int>(gridDim.x) - 1 && end < ldc) {
    const int64_t pieces = (ldc - end) / 16;
    for (int r = nb * kBlk; r < min(n, (nb + 1) * kBlk); ++r)
      for (int64_t i = threadIdx.x; i < pieces; i += 256)
        *reinterpret_cast<uint4*>(codes + r * ldc + end + 16 * i) = make_uint4(0, 0, 0, 0);
  }
}

// ---- tensor-core helpers -------------------------------------------------------------

// 128-byte swizzled K-major operand: rows of 128 bytes, groups of 8 rows
// 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= 1ull << 16;                                   // leading offset: unused with a swizzle
  d |= static_cast<uint64_t>(1024 >> 4) << 32;       // stride offset
  d |= 1ull << 46;                                   // descriptor version
  d |= 2ull << 61;                                   // 128-byte swizzle
  return d;
}

// kind::f8f6f4: fp32 accumulator, e4m3 A and B, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Sixteen consecutive columns of this warp's 32 lanes; asynchronous until tmem_wait.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Sixteen bytes at the shared-memory address `at` of CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster(uint32_t at, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(at), "r"(rank)
      : "memory");
  return v;
}

// ---- the product -----------------------------------------------------------------------

struct GemmArgs {
  const float* ws;       // [row block of w][blocks]
  const float* xs;       // [blocks][rows_pad]
  const uint8_t* codes;  // tiles of x
  void* out;
  int64_t ld_out;
  int out_type;
  int n, rows, rows_pad, blocks;
  int tiles_n, tiles_m, split;
  int out_vec;           // rows of out start on 16 bytes
  unsigned* ctl;
};

constexpr int kDirectBlocks = 16;   // blocks of x a CTA quantises itself at most ...
constexpr int kDirectPieces = 768;  // ... and pieces of 16 inputs

// DIRECT: few rows and few blocks a CTA; it quantises its part of x itself.
template <int BN, bool DIRECT>
struct Cfg {
  static constexpr int kEpi = BN >= 128 ? 8 : 4;               // warps that read accumulators
  static constexpr int kThreads = 128 + 32 * kEpi;
  static constexpr int kCols = BN / (kEpi / 4);                // columns per thread
  static constexpr int kBuf = 4;                               // accumulators in tensor memory
  static constexpr uint32_t kTmem = BN * kBuf;
  static constexpr int kStage = kTileW + (DIRECT ? 0 : BN * kBlk);
  static constexpr int kStages = !DIRECT && (200 * 1024) / kStage < 8 ? (200 * 1024) / kStage : 8;
  static constexpr int kX = DIRECT ? kDirectBlocks * BN * kBlk : 0;  // x of all blocks of a DIRECT CTA
  static constexpr int kScales = DIRECT ? kDirectBlocks : kScaleRing;
  static constexpr int kScaleOff = kStages * kStage + kX;      // [kScales][BN] floats
  static constexpr int kBarOff = kScaleOff + kScales * BN * 4;
  static constexpr int kBars = 2 * kStages + 2 * kBuf + 2 * kScaleRing + 1;
  static constexpr int kSmem = kBarOff + kBars * 8 + 16 + 1024;  // + alignment of the base
  static_assert(kStages >= 2 && kStages * kStage >= BN * kBlk * 4, "the partial sums of a tile fit the ring");
};

template <int BN, bool DIRECT>
__global__ void __launch_bounds__(Cfg<BN, DIRECT>::kThreads, 1)
    fp8_gemm_kernel(const GemmArgs g, const QuantArgs q, const __grid_constant__ CUtensorMap wmap) {
  using C = Cfg<BN, DIRECT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* const xres = sm + C::kStages * C::kStage;
  float* scale_ring = reinterpret_cast<float*>(sm + C::kScaleOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kBarOff);
  uint64_t *full = bars, *empty = full + C::kStages, *tfull = empty + C::kStages, *tempty = tfull + C::kBuf,
           *sfull = tempty + C::kBuf, *sempty = sfull + kScaleRing, *done = sempty + kScaleRing;
  uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = g.split;
  const int part = split > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int worker = blockIdx.x / split, workers = gridDim.x / split;
  const int tiles = g.tiles_n * g.tiles_m;
  const int b0 = static_cast<int>(static_cast<int64_t>(g.blocks) * part / split);
  const int b1 = static_cast<int>(static_cast<int64_t>(g.blocks) * (part + 1) / split);
  const int nb = b1 - b0;

  // rows of a tile
  auto rows_of = [&](int tile) { return min(BN, g.rows - (tile % g.tiles_m) * BN); };
  const int total = ((tiles - worker + workers - 1) / workers) * nb;  // blocks of this CTA's tiles
  const int ahead = min(total, C::kStages);
  const uint64_t wpol = g.tiles_m == 1 ? policy_evict_first() : policy_evict_last();
  auto load_w = [&](int s, int tile, int b) {
    mbar_arrive_expect_tx(full + s, kTileW + (DIRECT ? 0 : (rows_of(tile) + 7) / 8 * 1024));
    tma_load_2d(sm + s * C::kStage, &wmap, b * kBlk, (tile / g.tiles_m) * kBlk, full + s, wpol);
  };

  // The block's first memory requests go out before it meets: the first
  // weight tiles (which do not depend on the quantisation kernel before this
  // one), and with DIRECT its part of x.
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(full + i, 1), mbar_init(empty + i, 1);
    for (int i = 0; i < C::kBuf; ++i) mbar_init(tfull + i, 1), mbar_init(tempty + i, C::kEpi);
    for (int i = 0; i < kScaleRing; ++i) mbar_init(sfull + i, 1), mbar_init(sempty + i, C::kEpi);
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    for (int i = 0; i < ahead; ++i) load_w(i, worker + (i / nb) * workers, b0 + i % nb);
  }
  if (warp == 1) tmem_alloc(smem_u32(slot), C::kTmem);
  if (DIRECT && warp >= 2) {
    const float* ws = g.ws + static_cast<size_t>(worker / g.tiles_m) * g.blocks;
    const int rows = rows_of(worker), row0 = (worker % g.tiles_m) * BN;
    for (int base = 0; base < rows * nb * 8; base += C::kThreads - 64) {
      const int item = base + threadIdx.x - 64, unit = item >> 3, piece = item & 7;
      const int b = unit / rows, row = unit - b * rows;
      const bool in = b < nb;
      const float w = in ? ws[b0 + b] : 0.0f;
      float s;
      const uint4 codes = quantize_piece(q, in, row0 + row, b0 + b, piece, s);
      if (in) {
        *reinterpret_cast<uint4*>(xres + b * (BN * kBlk) + row * kBlk + ((piece ^ (row & 7)) << 4)) = codes;
        if (piece == 0) scale_ring[b * BN + row] = s * w;
      }
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  bool ok = true;

  if (warp == 0) {
    // loads
    if (lane == 0) {
      auto load_x = [&](int s, int tile, int b) {
        if constexpr (!DIRECT)
          bulk_g2s(sm + s * C::kStage + kTileW,
                   g.codes + (static_cast<size_t>(tile % g.tiles_m) * g.blocks + b) * (static_cast<size_t>(BN) * kBlk),
                   (rows_of(tile) + 7) / 8 * 1024, full + s);
      };
      if (!DIRECT) pdl_wait();
      for (int i = 0; i < ahead; ++i) load_x(i, worker + (i / nb) * workers, b0 + i % nb);
      RingPos p;
      int issued = ahead;
      if (ahead == C::kStages) p.ph = 1;
      else p.s = ahead;
      int tile = worker + (ahead / nb) * workers, b = ahead % nb;
      for (; issued < total; ++issued) {
        if (!mbar_wait(empty + p.s, p.ph ^ 1u)) {
          ok = false;
          break;
        }
        load_w(p.s, tile, b0 + b);
        load_x(p.s, tile, b0 + b);
        p.next(C::kStages);
        if (++b == nb) b = 0, tile += workers;
      }
      // a run that gave up leaves no copy in flight
      if (!ok) {
        latch_error(g.ctl, kErrTimeout);
        for (int i = max(0, issued - C::kStages); i < issued; ++i)
          mbar_wait(full + i % C::kStages, static_cast<uint32_t>(i / C::kStages) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      RingPos p, t;
      for (int tile = worker; ok && tile < tiles; tile += workers) {
        const uint32_t idesc = idesc_e4m3(kBlk, (rows_of(tile) + 15) / 16 * 16);
        for (int b = 0; b < nb; ++b) {
          ok = mbar_wait(tempty + t.s, t.ph ^ 1u) && mbar_wait(full + p.s, p.ph);
          if (!ok) break;
          tc_fence_after();
          const uint64_t wd = desc_sw128(smem_u32(sm + p.s * C::kStage));
          const uint64_t xd = desc_sw128(smem_u32(DIRECT ? xres + b * (BN * kBlk) : sm + p.s * C::kStage + kTileW));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3(tmem + t.s * BN, wd + 2 * k, xd + 2 * k, idesc, k > 0);
          mma_commit(smem_u32(empty + p.s));
          mma_commit(smem_u32(tfull + t.s));
          p.next(C::kStages);
          t.next(C::kBuf);
        }
      }
      mma_commit(smem_u32(done));
      if (!mbar_wait(done, 0)) ok = false;
      if (!ok) latch_error(g.ctl, kErrTimeout);
    }
    __syncwarp();
  } else if (warp == 2 && !DIRECT) {
    // scales: xs[b][rows of the tile] * ws[tile][b], kScaleRing blocks ahead
    pdl_wait();
    RingPos p;
    for (int tile = worker; ok && tile < tiles; tile += workers) {
      const float* ws = g.ws + static_cast<size_t>(tile / g.tiles_m) * g.blocks;
      const float* xs = g.xs + (tile % g.tiles_m) * BN;
      for (int b = b0; b < b1; ++b) {
        const float w = ws[b];
        float v[(BN + 31) / 32];
#pragma unroll
        for (int i = 0; i < (BN + 31) / 32; ++i)
          v[i] = 32 * i + lane < BN ? xs[static_cast<size_t>(b) * g.rows_pad + 32 * i + lane] * w : 0.0f;
        if (!mbar_wait_warp(sempty + p.s, p.ph ^ 1u)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int i = 0; i < (BN + 31) / 32; ++i)
          if (32 * i + lane < BN) scale_ring[p.s * BN + 32 * i + lane] = v[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(sfull + p.s);
        p.next(kScaleRing);
      }
    }
    if (!ok && lane == 0) latch_error(g.ctl, kErrTimeout);
  } else if (warp >= 4) {
    const int quad = warp & 3, col0 = ((warp - 4) >> 2) * C::kCols;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    RingPos t, p;
    for (int tile = worker; ok && tile < tiles; tile += workers) {
      float acc[C::kCols];
#pragma unroll
      for (int c = 0; c < C::kCols; ++c) acc[c] = 0.0f;
      for (int b = 0; b < nb; ++b) {
        ok = (DIRECT || mbar_wait_warp(sfull + p.s, p.ph)) && mbar_wait_warp(tfull + t.s, t.ph);
        if (!ok) break;
        tc_fence_after();
        const float4* sc = reinterpret_cast<const float4*>(scale_ring + (DIRECT ? b : p.s) * BN + col0);
#pragma unroll
        for (int c = 0; c < C::kCols; c += 16) {
          uint32_t d[16];
          tmem_ld16(tmem + lane_base + t.s * BN + col0 + c, d);
          tmem_wait();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 s = sc[c / 4 + i];
            acc[c + 4 * i] = fmaf(__uint_as_float(d[4 * i]), s.x, acc[c + 4 * i]);
            acc[c + 4 * i + 1] = fmaf(__uint_as_float(d[4 * i + 1]), s.y, acc[c + 4 * i + 1]);
            acc[c + 4 * i + 2] = fmaf(__uint_as_float(d[4 * i + 2]), s.z, acc[c + 4 * i + 2]);
            acc[c + 4 * i + 3] = fmaf(__uint_as_float(d[4 * i + 3]), s.w, acc[c + 4 * i + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(tempty + t.s);
          if (!DIRECT) mbar_arrive(sempty + p.s);
        }
        t.next(C::kBuf);
        p.next(kScaleRing);
      }
      if (!ok) break;
      const int row = quad * 32 + lane;
      if (split == 1) {
        const int n = (tile / g.tiles_m) * kBlk + row, t0 = (tile % g.tiles_m) * BN + col0;
#pragma unroll
        for (int c = 0; c < C::kCols; ++c)
          if (n < g.n && t0 + c < g.rows) store_elem(g.out, g.out_type, (t0 + c) * g.ld_out + n, acc[c]);
      } else {
        // the ring is idle now: every copy and MMA of this CTA's one tile is done
        float* partial = reinterpret_cast<float*>(sm) + col0 * kBlk + row;
#pragma unroll
        for (int c = 0; c < C::kCols; ++c) partial[c * kBlk] = acc[c];
      }
    }
    if (!ok && lane == 0) latch_error(g.ctl, kErrTimeout);
  }

  if (split > 1) {
    // column c of the tile is summed by CTA c % split of the cluster, four
    // outputs a thread, over the CTAs in order
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int mt = worker % g.tiles_m, cols = (rows_of(worker) - part + split - 1) / split;
#pragma unroll 1
    for (int i = threadIdx.x; i < cols * (kBlk / 4); i += C::kThreads) {
      const int c = part + split * (i / (kBlk / 4)), r = 4 * (i % (kBlk / 4));
      const uint32_t at = smem_u32(sm) + (c * kBlk + r) * 4;
      float4 v[kMaxSplit];
#pragma unroll
      for (int k = 0; k < kMaxSplit; ++k) v[k] = ld_cluster(at, k < split ? k : part);
      float4 s = v[0];
#pragma unroll
      for (int k = 1; k < kMaxSplit; ++k)
        if (k < split) s.x += v[k].x, s.y += v[k].y, s.z += v[k].z, s.w += v[k].w;
      const int n = (worker / g.tiles_m) * kBlk + r;
      const int64_t o = static_cast<int64_t>(mt * BN + c) * g.ld_out + n;
      if (n < g.n) store_elem(g.out, g.out_type, o, s.x);
      if (n + 1 < g.n) store_elem(g.out, g.out_type, o + 1, s.y);
      if (n + 2 < g.n) store_elem(g.out, g.out_type, o + 2, s.z);
      if (n + 3 < g.n) store_elem(g.out, g.out_type, o + 3, s.w);
    }
    cluster.sync();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::kTmem);
}

template <int BN, bool DIRECT>
cudaError_t launch_gemm(const GemmArgs& g, const QuantArgs& q, const CUtensorMap& map, int grid, cudaStream_t st) {
  using C = Cfg<BN, DIRECT>;
  auto kernel = fp8_gemm_kernel<BN, DIRECT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = g.split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = DIRECT ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kernel, g, q, map);
}

// ---- many rows: pairs of SMs -----------------------------------------------------------
// A cluster of two CTAs computes 256 rows of x by 256 outputs with
// tcgen05.mma.cta_group::2: CTA r holds rows 128 r.. of x and outputs
// 128 r.. of w of a block in its shared memory, and the accumulators of its
// own rows (128 lanes x 256 columns, two of them).  Each operand byte thus
// feeds two SMs: 32 KB a block and SM into shared memory and as much out of
// it, where one SM's 128 x 256 tile takes 48 in and 48 out (4096 x 7168 x 7168
// by such tiles: 169 us, by pairs 163).  The rows of x are the accumulator's
// lanes: an epilogue thread has one row and 64 outputs of one weight block, so
// the scale of a block is one number for it.
//
// Bound: the way from an MMA to its scaled sum and back.  A block's MMAs keep
// the tensor pipe busy for some 630 cycles, but with two accumulators (all of
// the tensor memory) the next one waits for commit, read and release of the
// one before the last; measured some 850 cycles a block.

constexpr int kPairStages = 6;
constexpr int kPairStage = 2 * kTileW;
constexpr int kPairEpi = 16;                              // warps that read accumulators, 64 columns each
constexpr int kPairCols = 4 * 2 * kBlk / kPairEpi;
constexpr int kPairThreads = 32 * (4 + kPairEpi);         // load, MMA, scales, idle, epilogue
// Registers of a thread: of the launch's 96 x 640, 56 x 128 and 104 x 512.
constexpr int kPairRegsFew = 56, kPairRegsEpi = 104;
constexpr int kPairOutBytes = 64;                         // of a row that an epilogue warp puts in order at once
constexpr int kPairOutOff = kPairStages * kPairStage;     // [epilogue warp][16 rows][kPairOutBytes]
constexpr int kPairChunk = 8;                             // blocks whose scales are handed over together
constexpr int kPairScaleOff = kPairOutOff + kPairEpi * 16 * kPairOutBytes;  // [2][kPairChunk][2][128] floats
constexpr int kPairBarOff = kPairScaleOff + 2 * kPairChunk * 2 * kBlk * 4;
constexpr int kPairBars = 2 * kPairStages + 4 + 4 + 1;
constexpr int kPairSmem = kPairBarOff + kPairBars * 8 + 16;
static_assert(kPairSmem <= 232448, "shared memory");

// The address of this CTA's shared-memory object in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_cta(uint32_t addr, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}

// An arrival at the barrier at cluster address `addr`.  What it orders are the
// tensor-memory loads before it (waited for, and fenced), not memory: with
// release.cluster here, a fence for every block and warp, 4096 x 7168 x 7168
// took 410 us instead of 201.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// mbar_wait for a phase that the other CTA's threads complete.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
  unsigned long long t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (i == 0) t0 = global_timer_ns();
    else if ((i & 255u) == 0 && global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
}

// Tile load into this CTA's shared memory, counted on the barrier at the
// cluster address `bar` of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void mma_e4m3_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// One arrival at this barrier in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Stores 64 bytes of each of a warp's 32 rows (t0 on; lane r holds row r) from
// output n on, sixteen rows at a time.  `buf`: the warp's 1 KB; 16-byte piece q
// of row r lies at piece q ^ (r / 2 & 3), so that neither side's accesses
// collide.
template <int ES>
__device__ __forceinline__ void store_rows(const GemmArgs& g, uint8_t* buf, const uint4 (&v)[4], int t0, int n) {
  const int lane = threadIdx.x & 31;
  uint8_t* const out = static_cast<uint8_t*>(g.out);
#pragma unroll
  for (int h = 0; h < 2; ++h, t0 += 16) {
    __syncwarp();
    if (lane >> 4 == h) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(buf + (lane & 15) * kPairOutBytes + ((q ^ (lane >> 1 & 3)) << 4)) = v[q];
    }
    __syncwarp();
    if (g.out_vec && n + kPairOutBytes / ES <= g.n) {
      // four lanes a row
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * i + (lane >> 2), q = lane & 3;
        const uint4 w = *reinterpret_cast<const uint4*>(buf + r * kPairOutBytes + ((q ^ (r >> 1 & 3)) << 4));
        if (t0 + r < g.rows)
          *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(t0 + r) * g.ld_out + n) * ES + q * 16) = w;
      }
    } else {
      // a lane an element, a row or two at a time
      constexpr int kCols = kPairOutBytes / ES, kRows = 32 / kCols;
      const int c = lane % kCols;
#pragma unroll 1
      for (int r = lane / kCols; r < 16; r += kRows) {
        const uint8_t* at = buf + r * kPairOutBytes + (((c * ES >> 4) ^ (r >> 1 & 3)) << 4) + (c * ES & 15);
        if (t0 + r < g.rows && n + c < g.n) {
          uint8_t* to = out + (static_cast<int64_t>(t0 + r) * g.ld_out + n + c) * ES;
          if constexpr (ES == 4) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(at);
          else *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<const uint16_t*>(at);
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    fp8_pair_kernel(const GemmArgs g, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ __align__(1024) uint8_t sm[];
  float* scale_ring = reinterpret_cast<float*>(sm + kPairScaleOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kPairBarOff);
  uint64_t *full = bars, *empty = full + kPairStages, *tfull = empty + kPairStages, *tempty = tfull + 2,
           *sfull = tempty + 2, *sempty = sfull + 2, *done = sempty + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(cluster.block_rank());
  const int worker = blockIdx.x >> 1, workers = gridDim.x >> 1;
  const int tiles = g.tiles_n * g.tiles_m, nb = g.blocks;

  if (threadIdx.x == 0) {
    // full, tempty: used in CTA 0, for both
    for (int i = 0; i < kPairStages; ++i) mbar_init(full + i, 1), mbar_init(empty + i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(tfull + i, 1), mbar_init(tempty + i, 2 * kPairEpi);
    for (int i = 0; i < 2; ++i) mbar_init(sfull + i, 1), mbar_init(sempty + i, kPairEpi);
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::);
  }
  tc_fence_before();
  __syncthreads();
  cluster.sync();
  tc_fence_after();
  const uint32_t tmem = *slot;
  bool ok = true;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairRegsFew));
    if (warp == 0) {
      if (lane == 0) {
        const uint64_t keep = policy_evict_last();
        const int total = ((tiles - worker + workers - 1) / workers) * nb;
        const int ahead = min(total, kPairStages);
        auto load_w = [&](int s, int tn, int b) {
          if (cta == 0) mbar_arrive_expect_tx(full + s, 2 * kPairStage);
          tma_load_pair(sm + s * kPairStage + kTileW, &wmap, b * kBlk, (2 * tn + cta) * kBlk, map_cta(smem_u32(full + s), 0), keep);
        };
        auto load_x = [&](int s, int tm, int b) {
          tma_load_pair(sm + s * kPairStage, &xmap, b * kBlk, (2 * tm + cta) * kBlk, map_cta(smem_u32(full + s), 0), keep);
        };
        int tile = worker, b = 0, tm = tile % g.tiles_m, tn = tile / g.tiles_m;
        auto next_block = [&]() {
          if (++b == nb) b = 0, tile += workers, tm = tile % g.tiles_m, tn = tile / g.tiles_m;
        };
        // the weights do not depend on the quantisation kernel before this one
        for (int i = 0; i < ahead; ++i, next_block()) load_w(i, tn, b);
        pdl_wait();
        tile = worker, b = 0, tm = tile % g.tiles_m, tn = tile / g.tiles_m;
        for (int i = 0; i < ahead; ++i, next_block()) load_x(i, tm, b);
        RingPos p;
        if (ahead == kPairStages) p.ph = 1;
        else p.s = ahead;
        int issued = ahead;
        for (; issued < total; ++issued, next_block()) {
          if (!mbar_wait(empty + p.s, p.ph ^ 1u)) {
            ok = false;
            break;
          }
          load_w(p.s, tn, b);
          load_x(p.s, tm, b);
          p.next(kPairStages);
        }
        // a run that gave up leaves no copy in flight: CTA 0's barriers count both CTAs'
        if (!ok) {
          latch_error(g.ctl, kErrTimeout);
          if (cta == 0)
            for (int i = max(0, issued - kPairStages); i < issued; ++i)
              mbar_wait(full + i % kPairStages, static_cast<uint32_t>(i / kPairStages) & 1u);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // the whole warp keeps the loop, so that its values stay uniform; one lane issues
      if (cta == 0) {
        constexpr uint32_t idesc = idesc_e4m3(2 * kBlk, 2 * kBlk);
        const uint32_t ring = smem_u32(sm);
        RingPos p, t;
        for (int tile = worker; ok && tile < tiles; tile += workers) {
          for (int b = 0; b < nb; ++b) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(tempty + t.s, t.ph ^ 1u) && mbar_wait_cluster(full + p.s, p.ph));
            if (!ok) break;
            tc_fence_after();
            const uint64_t xd = desc_sw128(ring + p.s * kPairStage);
            const uint64_t wd = desc_sw128(ring + p.s * kPairStage + kTileW);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_e4m3_pair(tmem + t.s * 2 * kBlk, xd + 2 * k, wd + 2 * k, idesc, k > 0);
              mma_commit_pair(smem_u32(tfull + t.s));
              mma_commit_pair(smem_u32(empty + p.s));
            }
            __syncwarp();
            p.next(kPairStages);
            t.next(2);
          }
        }
        if (elect_one()) mma_commit_pair(smem_u32(done));
        __syncwarp();
        if (!mbar_wait(done, 0)) ok = false;
        if (!ok && lane == 0) latch_error(g.ctl, kErrTimeout);
      }
      __syncwarp();
    } else if (warp == 2) {
      // scales: xs[b][the tile's rows] * ws[either weight block][b], kPairChunk
      // blocks at a time (a wait for each block cost 12 us of 178)
      pdl_wait();
      RingPos p;
      for (int tile = worker; ok && tile < tiles; tile += workers) {
        const int n0 = 2 * (tile / g.tiles_m), n1 = min(n0 + 1, (g.n - 1) / kBlk);
        const float *w0 = g.ws + static_cast<size_t>(n0) * nb, *w1 = g.ws + static_cast<size_t>(n1) * nb;
        const float* xs = g.xs + (2 * (tile % g.tiles_m) + cta) * kBlk + lane * 4;
        for (int b0 = 0; b0 < nb; b0 += kPairChunk) {
          ok = mbar_wait_warp(sempty + p.s, p.ph ^ 1u);
          if (!ok) break;
          float4* to = reinterpret_cast<float4*>(scale_ring + p.s * kPairChunk * 2 * kBlk) + lane;
#pragma unroll 4
          for (int b = b0; b < min(nb, b0 + kPairChunk); ++b, to += kBlk / 2) {
            const float4 x = *reinterpret_cast<const float4*>(xs + static_cast<size_t>(b) * g.rows_pad);
            const float u = w0[b], v = w1[b];
            to[0] = make_float4(x.x * u, x.y * u, x.z * u, x.w * u);
            to[kBlk / 4] = make_float4(x.x * v, x.y * v, x.z * v, x.w * v);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(sfull + p.s);
          p.next(2);
        }
      }
      if (!ok && lane == 0) latch_error(g.ctl, kErrTimeout);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairRegsEpi));
    const int quad = warp & 3, col0 = ((warp - 4) >> 2) * kPairCols, row = quad * 32 + lane;
    const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    const uint32_t freed = map_cta(smem_u32(tempty), 0);
    const float* const scale = scale_ring + (col0 / kBlk) * kBlk + row;
    RingPos t, p;
    for (int tile = worker; ok && tile < tiles; tile += workers) {
      float2 acc[kPairCols / 2];
#pragma unroll
      for (int c = 0; c < kPairCols / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
#pragma unroll 1
      for (int b = 0; b < nb; ++b) {
        if (b % kPairChunk == 0) ok = mbar_wait_warp(sfull + p.s, p.ph);
        const float s1 = scale[(p.s * kPairChunk + b % kPairChunk) * 2 * kBlk];
        ok = ok && mbar_wait_warp(tfull + t.s, t.ph);
        if (!ok) break;
        tc_fence_after();
        const float2 s = make_float2(s1, s1);
#pragma unroll
        for (int c = 0; c < kPairCols; c += 16) {
          uint32_t d[16];
          tmem_ld16(from + t.s * 2 * kBlk + c, d);
          tmem_wait();
          if (c + 16 == kPairCols) {
            // all columns read: the next block but one may have the buffer
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(freed + t.s * 8);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            acc[c / 2 + j] = __ffma2_rn(make_float2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1])), s, acc[c / 2 + j]);
        }
        t.next(2);
        if (b % kPairChunk == kPairChunk - 1 || b == nb - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(sempty + p.s);
          p.next(2);
        }
      }
      if (!ok) break;
      // A thread holds a row; 64 bytes of each of the warp's 32 rows at a time
      // go through shared memory, so that stores cover whole sectors.  (Straight
      // from the registers a tile's stores took 6,800 cycles.)
      const int t0 = (2 * (tile % g.tiles_m) + cta) * kBlk + quad * 32;
      const int n0 = 2 * (tile / g.tiles_m) * kBlk + col0;
      uint8_t* out = sm + kPairOutOff + (warp - 4) * 16 * kPairOutBytes;
      if (g.out_type == MOE_F32) {
#pragma unroll
        for (int c = 0; c < kPairCols; c += 16) {
          uint4 v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            v[q] = make_uint4(__float_as_uint(acc[c / 2 + 2 * q].x), __float_as_uint(acc[c / 2 + 2 * q].y),
                              __float_as_uint(acc[c / 2 + 2 * q + 1].x), __float_as_uint(acc[c / 2 + 2 * q + 1].y));
          store_rows<4>(g, out, v, t0, n0 + c);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kPairCols; c += 32) {
          uint4 v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2* f = acc + c / 2 + 4 * q;
            v[q] = make_uint4(pack2(f[0].x, f[0].y, g.out_type), pack2(f[1].x, f[1].y, g.out_type),
                              pack2(f[2].x, f[2].y, g.out_type), pack2(f[3].x, f[3].y, g.out_type));
          }
          store_rows<2>(g, out, v, t0, n0 + c);
        }
      }
    }
    if (!ok && lane == 0) latch_error(g.ctl, kErrTimeout);
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other, or an MMA of both, may signal it
  if (cta == 1 && threadIdx.x == 0 && !mbar_wait(done, 0)) latch_error(g.ctl, kErrTimeout);
  cluster.sync();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

cudaError_t launch_pair(const GemmArgs& g, const CUtensorMap& wmap, const CUtensorMap& xmap, int num_sms, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(fp8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  if (e) return e;
  const int64_t tiles = static_cast<int64_t>(g.tiles_n) * g.tiles_m;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(tiles < num_sms / 2 ? tiles : num_sms / 2));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fp8_pair_kernel, g, wmap, xmap);
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Tiles of 128 rows x 128 bytes in the order the tensor core reads.
bool encode_tiles(EncodeFn fn, CUtensorMap* m, const uint8_t* codes, int64_t rows, int64_t cols, int64_t ld) {
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {kBlk, kBlk}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dim, stride, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace moe

struct moe_fp8 {
  uint32_t magic;
  int n, k, device, num_sms;
  const float* scales;
  moe::EncodeFn encode;
  CUtensorMap map;
};

using namespace moe;

static bool handle_ok(const moe_fp8* w) { return w && w->magic == kMagic; }

extern "C" int moe_fp8_open(int32_t n, int32_t k, const uint8_t* codes, int64_t ld_codes, const float* scales,
                            moe_fp8** out) {
  if (!out) return reportf(MOE_ERR_ARG, "moe_fp8_open: out is NULL");
  *out = nullptr;
  if (n < 1 || n > (1 << 24) || k < 1 || k > 65536)
    return reportf(MOE_ERR_ARG, "moe_fp8_open: n=%d must be in [1, 2^24], k=%d in [1, 65536]", n, k);
  if (!codes || !scales) return reportf(MOE_ERR_ARG, "moe_fp8_open: codes or scales is NULL");
  if (ld_codes < k || ld_codes % 16 || ld_codes > (1ll << 32))
    return reportf(MOE_ERR_ARG, "moe_fp8_open: ld_codes=%lld must be a multiple of 16 and at least k=%d",
                   static_cast<long long>(ld_codes), k);
  if (reinterpret_cast<uintptr_t>(codes) % 16 || reinterpret_cast<uintptr_t>(scales) % 4)
    return reportf(MOE_ERR_ALIGN, "moe_fp8_open: codes must be 16-byte aligned, scales 4-byte");
  int dev = 0, major = 0, minor = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (!e) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (!e) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (!e) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e) return reportf(MOE_ERR_CUDA, "moe_fp8_open: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  if (major != 10 || minor != 3)
    return reportf(MOE_ERR_UNSUPPORTED, "moe_fp8_open: device %d is sm_%d%d; this library is built for sm_103a", dev,
                   major, minor);
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
  if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn)
    return reportf(MOE_ERR_CUDA, "moe_fp8_open: no cuTensorMapEncodeTiled in this driver");
  moe_fp8* w = new (std::nothrow) moe_fp8;
  if (!w) return reportf(MOE_ERR_NOMEM, "moe_fp8_open: out of host memory");
  w->magic = kMagic, w->n = n, w->k = k, w->device = dev, w->num_sms = sms, w->scales = scales;
  w->encode = reinterpret_cast<EncodeFn>(fn);
  if (!encode_tiles(w->encode, &w->map, codes, n, k, ld_codes)) {
    delete w;
    return reportf(MOE_ERR_CUDA, "moe_fp8_open: cuTensorMapEncodeTiled refused n=%d k=%d ld_codes=%lld", n, k,
                   static_cast<long long>(ld_codes));
  }
  *out = w;
  return MOE_OK;
}

extern "C" void moe_fp8_close(moe_fp8* w) {
  if (!handle_ok(w)) return;
  w->magic = 0;
  delete w;
}

extern "C" size_t moe_fp8_workspace_bytes(const moe_fp8* w, int32_t max_rows) {
  if (!handle_ok(w) || max_rows < 1 || max_rows > kMaxRows) return 0;
  // of the widest tile: any narrower one, and any fewer rows, pad to no more
  return layout_of(max_rows, widest_tile(max_rows), w->k).bytes;
}

extern "C" int moe_fp8_workspace_init(const moe_fp8* w, void* workspace, size_t workspace_bytes, void* stream) {
  if (!handle_ok(w)) return reportf(MOE_ERR_ARG, "moe_fp8_workspace_init: invalid handle");
  if (!workspace || workspace_bytes < kCtlBytes)
    return reportf(MOE_ERR_ARG, "moe_fp8_workspace_init: workspace is NULL or has %zu bytes", workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) % 256)
    return reportf(MOE_ERR_ALIGN, "moe_fp8_workspace_init: workspace must be 256-byte aligned");
  const cudaError_t e = cudaMemsetAsync(workspace, 0, kCtlBytes, static_cast<cudaStream_t>(stream));
  if (e) return reportf(MOE_ERR_CUDA, "moe_fp8_workspace_init: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  return MOE_OK;
}

extern "C" int moe_fp8_linear(moe_fp8* w, const void* x, int32_t x_type, int64_t ld_x, int32_t rows, void* out,
                              int32_t out_type, int64_t ld_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!handle_ok(w)) return reportf(MOE_ERR_ARG, "moe_fp8_linear: invalid handle");
  if (rows < 0 || rows > kMaxRows) return reportf(MOE_ERR_ARG, "moe_fp8_linear: rows=%d must be in [0, %d]", rows, kMaxRows);
  if (rows == 0) return MOE_OK;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != w->device)
    return reportf(MOE_ERR_ARG, "moe_fp8_linear: the handle's device %d must be the current device", w->device);
  if (!x || !out || !workspace) return reportf(MOE_ERR_ARG, "moe_fp8_linear: x, out or workspace is NULL");
  if (!elem_type_ok(x_type) || !elem_type_ok(out_type))
    return reportf(MOE_ERR_ARG, "moe_fp8_linear: unknown type (x %d, out %d)", x_type, out_type);
  if (ld_x < w->k || ld_out < w->n)
    return reportf(MOE_ERR_ARG, "moe_fp8_linear: ld_x=%lld is below k=%d or ld_out=%lld below n=%d",
                   static_cast<long long>(ld_x), w->k, static_cast<long long>(ld_out), w->n);
  if (reinterpret_cast<uintptr_t>(x) % elem_size(x_type) || reinterpret_cast<uintptr_t>(out) % elem_size(out_type) ||
      reinterpret_cast<uintptr_t>(workspace) % 256)
    return reportf(MOE_ERR_ALIGN, "moe_fp8_linear: x or out is not aligned to its elements, or workspace to 256 bytes");
  const Cut cut = cut_of(rows, w->n, w->k, w->num_sms);
  const Layout l = layout_of(rows, cut.bn, w->k);
  const size_t need = moe_fp8_workspace_bytes(w, rows);
  if (workspace_bytes < need)
    return reportf(MOE_ERR_ARG, "moe_fp8_linear: %d rows need %zu bytes of workspace, got %zu", rows, need,
                   workspace_bytes);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(workspace);

  QuantArgs q;
  q.x = x, q.ld = ld_x, q.type = x_type, q.rows = rows, q.k = w->k;
  q.blocks = l.blocks, q.rows_pad = l.rows_pad, q.bn_log2 = l.bn == 16 ? 4 : l.bn == 32 ? 5 : l.bn == 64 ? 6 : l.bn == 128 ? 7 : 8;
  q.vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld_x * elem_size(x_type) % 16 == 0;
  q.xs = reinterpret_cast<float*>(base + l.xs), q.codes = base + l.codes;
  GemmArgs g;
  g.ws = w->scales, g.xs = q.xs, g.codes = q.codes;
  g.out = out, g.ld_out = ld_out, g.out_type = out_type;
  g.n = w->n, g.rows = rows, g.rows_pad = l.rows_pad, g.blocks = l.blocks;
  g.tiles_n = (w->n + kBlk - 1) / kBlk, g.tiles_m = l.row_tiles;
  g.ctl = reinterpret_cast<unsigned*>(base);
  const int64_t tiles = static_cast<int64_t>(g.tiles_n) * g.tiles_m;
  if (tiles > 0x3FFFFFFF) return reportf(MOE_ERR_ARG, "moe_fp8_linear: %d rows x %d outputs are too many tiles", rows, w->n);
  g.split = cut.split;
  g.out_vec = reinterpret_cast<uintptr_t>(out) % 16 == 0 && ld_out * elem_size(out_type) % 16 == 0;
  const bool pair = l.bn == 256;
  q.plain = pair;
  const int grid = tiles <= w->num_sms ? static_cast<int>(tiles) * g.split : w->num_sms;
  const int share = (l.blocks + g.split - 1) / g.split;
  const bool direct = tiles <= w->num_sms && l.bn <= 32 && share <= kDirectBlocks &&
                      (rows < l.bn ? rows : l.bn) * share * 8 <= kDirectPieces;
  cudaError_t e = cudaSuccess;
  if (direct) {
    e = l.bn == 16 ? launch_gemm<16, true>(g, q, w->map, grid, st) : launch_gemm<32, true>(g, q, w->map, grid, st);
  } else {
    const int64_t units = static_cast<int64_t>(rows) * l.blocks;
    quantize_rows_kernel<<<static_cast<unsigned>((units + 31) / 32), 256, 0, st>>>(q);
    e = cudaGetLastError();
    if (!e) {
      switch (l.bn) {
        case 16: e = launch_gemm<16, false>(g, q, w->map, grid, st); break;
        case 32: e = launch_gemm<32, false>(g, q, w->map, grid, st); break;
        case 64: e = launch_gemm<64, false>(g, q, w->map, grid, st); break;
        case 128: e = launch_gemm<128, false>(g, q, w->map, grid, st); break;
        default: {
          CUtensorMap xmap;
          if (!encode_tiles(w->encode, &xmap, q.codes, rows, static_cast<int64_t>(l.blocks) * kBlk, static_cast<int64_t>(l.blocks) * kBlk))
            return reportf(MOE_ERR_CUDA, "moe_fp8_linear: cuTensorMapEncodeTiled refused rows=%d k=%d", rows, w->k);
          g.tiles_n = (w->n + 2 * kBlk - 1) / (2 * kBlk);
          e = launch_pair(g, w->map, xmap, w->num_sms, st);
        }
      }
    }
  }
  if (e) return reportf(MOE_ERR_CUDA, "moe_fp8_linear: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  return MOE_OK;
}

extern "C" int moe_fp8_check(const moe_fp8* w, void* workspace, void* stream) {
  if (!handle_ok(w)) return reportf(MOE_ERR_ARG, "moe_fp8_check: invalid handle");
  if (!workspace) return reportf(MOE_ERR_ARG, "moe_fp8_check: workspace is NULL");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned bits = 0;
  cudaError_t e = cudaMemcpyAsync(&bits, workspace, sizeof bits, cudaMemcpyDeviceToHost, st);
  if (!e) e = cudaStreamSynchronize(st);
  if (!e && bits) {
    e = cudaMemsetAsync(workspace, 0, kCtlBytes, st);
    if (!e) e = cudaStreamSynchronize(st);
  }
  if (e) return reportf(MOE_ERR_CUDA, "moe_fp8_check: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  if (bits) return reportf(MOE_ERR_TIMEOUT, "moe_fp8_check: a bounded device-side wait ran out (bits 0x%x)", bits);
  return MOE_OK;
}

extern "C" int moe_fp8_quantize_weights(const void* weights, int32_t w_type, int64_t ld_w, int32_t n, int32_t k,
                                        uint8_t* codes, int64_t ld_codes, float* scales, void* stream) {
  if (n < 1 || n > (1 << 24) || k < 1 || k > 65536)
    return reportf(MOE_ERR_ARG, "moe_fp8_quantize_weights: n=%d must be in [1, 2^24], k=%d in [1, 65536]", n, k);
  if (!weights || !codes || !scales) return reportf(MOE_ERR_ARG, "moe_fp8_quantize_weights: a pointer is NULL");
  if (!elem_type_ok(w_type)) return reportf(MOE_ERR_ARG, "moe_fp8_quantize_weights: unknown type %d", w_type);
  if (ld_w < k || ld_codes < k || ld_codes % 16)
    return reportf(MOE_ERR_ARG, "moe_fp8_quantize_weights: ld_w=%lld and ld_codes=%lld must be at least k=%d, ld_codes a multiple of 16",
                   static_cast<long long>(ld_w), static_cast<long long>(ld_codes), k);
  if (reinterpret_cast<uintptr_t>(weights) % elem_size(w_type) || reinterpret_cast<uintptr_t>(codes) % 16 ||
      reinterpret_cast<uintptr_t>(scales) % 4)
    return reportf(MOE_ERR_ALIGN, "moe_fp8_quantize_weights: a pointer is misaligned");
  const int nblocks = (n + kBlk - 1) / kBlk;
  // row blocks in the grid's y, which is limited to 65535
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int kblocks = (k + kBlk - 1) / kBlk;
  for (int r0 = 0; r0 < nblocks; r0 += 65535) {
    const int cnt = nblocks - r0 < 65535 ? nblocks - r0 : 65535;
    const int64_t row = static_cast<int64_t>(r0) * kBlk;
    quantize_weights_kernel<<<dim3(kblocks, cnt), 256, 0, st>>>(
        static_cast<const char*>(weights) + row * ld_w * elem_size(w_type), w_type, ld_w, n - static_cast<int>(row), k,
        codes + row * ld_codes, ld_codes, scales + static_cast<size_t>(r0) * kblocks);
    const cudaError_t e = cudaGetLastError();
    if (e) return reportf(MOE_ERR_CUDA, "moe_fp8_quantize_weights: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  }
  return MOE_OK;
}
