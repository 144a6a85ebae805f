// attention_tc.cu -- attention of many rows over the paged cache on the
// fifth-generation tensor cores.
//
// Mathematics: as in attention.cu, a softmax in one pass with a reference m, sum l
// and output o in fp32.  m is the maximum of a row's first tile, and moves to a later
// maximum only when the exponentials relative to it pass kMost, which their sum tells: so
// o, which lies in tensor memory, is seldom touched between products, and no
// maximum is looked for.  It never exceeds the maximum, so l is 1 at least (2^7 with float16,
// whose exponentials carry that factor, as attention.cu's 2^15).
//
// Layout: a unit's tile (attention.cuh) has two halves of 128 rows (heads of up to
// 128) or one (of 256).  z = q k^T is a product of M = 128 rows, N = the key
// tile's positions, both operands in shared memory, the fp32 result in tensor
// memory; a thread of the half's four warps has one row of it, takes exponentials
// and stores them over z as 16-bit values, and o += p v takes them from there, v
// being read position by position (N-major).  With two halves one's softmax runs
// while the other's products do; with one half z has two buffers, so that the next
// tile's product runs during a softmax.
// Roles: eight warps (four with one half) take softmaxes, four bring keys and
// values into a ring of tiles in 128-byte swizzled order, one issues the products, one
// goes from unit to unit ahead of all.  16-bit tiles come by tiled loads, a box of one
// page's positions each (pages that no box of 8 divides by 16-byte copies); e4m3
// codes are read by the four warps and become 16-bit values on the way.
//
// What a row does not see but its tile does (the diagonal, a window's edge) gets
// exponential 0, which an infinity or a NaN among the values would turn into
// NaN: rows whose output is not finite are looked at again one by one.
//
// Bound: the way from a product to its exponentials and back, which the other half's
// product hides in part.  4096 rows behind 12288 of 64 heads of 128: 1395 to 1460 us
// by GPU, 1320 to 1380 TFLOP/s, 67 to 70% of the measured bf16 rate; a tile of 128
// positions and 256 rows takes 3390 clocks, of which its products, by themselves 1055
// to 1090 for 16, are 2130.
// Code that runs once a unit or tile waits for its own instructions, so loops are
// rolled where they can be: of products 1596 -> 1454 us, with exponentials 1454 -> 1400.
#include <cuda.h>
#include <cuda_runtime.h>

#include "attention.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kHalf = 128;         // rows of a half
// How large the exponentials of half a tile's positions may be in sum before the
// row's reference is moved: what the largest float16 leaves room for (65504).
constexpr float kMost = 49152.0f;

// From where on the reference is subtracted from z before the scale is multiplied on, which is
// exact near it.  Below, its rounding (2^-17) shifts a row's exponentials by 2^-17 together; far
// above, it would pass float16's range.  For every tile: prompts 2 to 3% slower.
constexpr float kLarge = 256.0f;

template <bool F16>
__host__ __device__ constexpr float tile_lift() {
  return F16 ? 7.0f : 0.0f;
}

template <int DP>
struct Geo {
  static constexpr int halves = DP <= 128 ? 2 : 1;
  static constexpr int rows = halves * kHalf;
  static constexpr int bn = DP <= 128 ? 128 : 64;
  static constexpr int q_bytes = kHalf * DP * 2;        // of a half
  static constexpr int stage_bytes = bn * DP * 2;       // a tile of keys or of values
  static constexpr int stages = DP == 64 ? 6 : 4;
  static constexpr int smem = halves * q_bytes + stages * stage_bytes + 1024;
  // tensor memory columns: z (and p) at [0, 256), o from 256 on
  static constexpr int z_cols = bn;
  static constexpr int o_col = 256, o_cols = DP;
};

template <int DP>
using TileWalk = Walk<Geo<DP>::rows, Geo<DP>::bn>;

template <int DP>
struct Shared {
  using G = Geo<DP>;
  uint64_t full[G::stages], empty[G::stages];
  uint64_t z_full[2], p_half[2], half_done[2], p_ready[2], o_full[2], q_full[2], pv_done, tail;
  // Of the tiles under way.  A slow producer thread may be at tile t - 1 while a
  // fast one writes tile t + 1; softmaxes may be three tiles behind.
  int64_t off[4][G::bn];                 // byte offsets of a tile's positions, -1: not seen
  int2 place[4][G::bn];                  // their pages and slots
  uint32_t bits[8][G::bn / 32];          // which of its positions count
  uint32_t tmem;
  int failed;
  int holes;                             // a page was missing among those of a tile
  TileWalk<DP> walk, pieces[4];          // one warp goes from piece to piece, the others take them from a ring
  uint64_t piece_full[4], piece_empty[4];
  PlanSmem plan;
};

// Descriptors of operands in 128-byte swizzled slabs of 64 elements.  Upper half:
// 1024 bytes between groups of 8 rows (or positions), descriptor version 1,
// 128-byte swizzle; lower half: start address >> 4 and, of an N-major operand (rows are
// positions, a slab's 64 elements are N), the distance between slabs.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t slab_bytes) { return (saddr >> 4) | (slab_bytes >> 4) << 16; }

// D[tmem] (+)= A[smem] * B[smem]^T and A[tmem] * B[smem], issued by one thread.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(id), "r"(accumulate), "n"(kDescHi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(id), "r"(accumulate), "n"(kDescHi));
}

template <bool F16>
__host__ __device__ constexpr uint32_t idesc(uint32_t N, bool b_n_major) {
  return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (b_n_major ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

template <int N>
__device__ __forceinline__ void reg_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One lane of the warp, the same every time.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// x * s + t of two values at once.
__device__ __forceinline__ void fma_pair(float& a, float& b, float s, float t) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(s), "f"(t));
}
__device__ __forceinline__ void add_pair(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tadd.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

// Waits unless some role has given up; latches the error if this one does.
__device__ __forceinline__ bool wait_long(unsigned* ctl, int* failed, uint64_t* bar, uint32_t parity) {
  if (*reinterpret_cast<volatile int*>(failed)) return false;
  if (mbar_wait(bar, parity)) return true;
  *reinterpret_cast<volatile int*>(failed) = 1;
  latch_error(ctl, kErrTimeout);
  return false;
}
template <class S>
__device__ __forceinline__ bool wait(S& sm, const AttnArgs& a, uint64_t* bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || mbar_try_wait(bar, parity) || wait_long(a.ctl, &sm.failed, bar, parity);
}

// A warp's place in the ring of pieces.  The last one has no tiles.
template <int DP>
struct Pieces {
  Shared<DP>& sm;
  const AttnArgs& a;
  int i = 0;
  __device__ __forceinline__ Pieces(Shared<DP>& s, const AttnArgs& args) : sm(s), a(args) {}
  __device__ __forceinline__ bool ready(int ahead) const {
    return wait(sm, a, &sm.piece_full[(i + ahead) & 3], ((i + ahead) >> 2) & 1);
  }
  __device__ __forceinline__ const TileWalk<DP>& at(int ahead) const { return sm.pieces[(i + ahead) & 3]; }
  __device__ __forceinline__ void done() {  // all lanes
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.piece_empty[i & 3]);
    ++i;
  }
};

// The warp that goes from piece to piece (all lanes).
template <int DP>
__device__ __forceinline__ void walk_role(const AttnArgs& a, Shared<DP>& sm, const Work& work) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) sm.walk.begin(a, work);
  __syncwarp();
#pragma unroll 1
  for (int i = 0;; ++i) {
    if (i >= 4 && !wait(sm, a, &sm.piece_empty[i & 3], ((i >> 2) - 1) & 1)) return;
    sm.pieces[i & 3].become(sm.walk);
    if (lane == 0) mbar_arrive(&sm.piece_full[i & 3]);
    if (!sm.walk.more()) return;
    sm.walk.next(a);
  }
}

// A cached 16-byte piece's eight 16-bit values as the products see them.
template <int K>
__device__ __forceinline__ uint4 values_at(const void* base, int64_t off, int d, float scale) {
  using T = Traits<K>;
  if constexpr (!T::e4m3) {
    return *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + off + d * 2);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + off + d);
    // no warp-wide agreement here: both factors, whatever the scale
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = (i < 2 ? w.x : w.y) >> (16 * (i & 1));
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3)));
      r[i] = pack2(f.x * scale, f.y * scale, T::f16 ? MOE_F16 : MOE_BF16);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
}

// What positions [k0, k1) add to a row's output, taken one position at a time, with
// exponentials relative to z = `ref` (all lanes, one row): lane l returns the sums of
// elements 4 l + 128 i to 4 l + 3 + 128 i.
template <int DP, int K>
__device__ __noinline__ void row_again(const AttnArgs& a, int seq, int head, const uint16_t* q, int k0, int k1, float ref,
                                       float (&o)[(DP + 127) / 128][4]) {
  using T = Traits<K>;
  constexpr int type = T::f16 ? MOE_F16 : MOE_BF16;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < (DP + 127) / 128; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
  for (int b = k0; b < k1; b += 32) {
    const int pos = b + lane;
    int slot = 0;
    const int page = pos < k1 ? page_of(a.q, seq, pos, slot) : -1;
    const int64_t off = page * a.page_stride + slot * a.slot_stride + head * a.head_stride;
    const int64_t soff = page * a.scale_page_stride + slot * a.scale_slot_stride + head * a.scale_head_stride;
    float p = 0.0f, vs = 1.0f;
    if (page >= 0) {
      float ks = 1.0f, z = 0.0f;
      if constexpr (T::e4m3) ks = a.k_scale[soff], vs = a.v_scale[soff];
      for (int d = 0; d < a.head_dim; d += 8) {
        float x[8], y[8];
        unpack8(values_at<K>(a.k, off, d, ks), type, x);
        unpack8(*reinterpret_cast<const uint4*>(q + d), type, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) z = fmaf(x[i], y[i], z);
      }
      // z may differ from the tensor cores' in the last bits: no further above than kMost; NaN stays
      const float e = fmaf(z - ref, a.scale_log2, tile_lift<T::f16>());
      p = half_bits_to_f32(f32_to_half_bits(exp2_approx(e > 15.5f ? 15.5f : e), type), type);
    }
    for (uint32_t m = __ballot_sync(0xFFFFFFFFu, page >= 0); m; m &= m - 1) {
      const int l = __ffs(m) - 1;
      const float w = __shfl_sync(0xFFFFFFFFu, p, l), s = __shfl_sync(0xFFFFFFFFu, vs, l);
      const int64_t at = __shfl_sync(0xFFFFFFFFu, off, l);
#pragma unroll
      for (int i = 0; i < (DP + 127) / 128; ++i) {
        const int d = 4 * lane + 128 * i;
        if (d < a.head_dim) {
          float x[8];
          unpack8(values_at<K>(a.v, at, d & ~7, s), type, x);
#pragma unroll
          for (int c = 0; c < 4; ++c) o[i][c] = fmaf(w, x[(lane & 1) * 4 + c], o[i][c]);
        }
      }
    }
  }
}

// Whether a value among positions [k0, k1) is not finite (all lanes).
template <int K>
__device__ __noinline__ bool odd_values(const AttnArgs& a, int seq, int head, int k0, int k1) {
  bool odd = false;
  for (int pos = k0 + (threadIdx.x & 31); pos < k1; pos += 32) {
    int slot = 0;
    const int page = page_of(a.q, seq, pos, slot);
    if (page < 0) continue;
    const int64_t off = page * a.page_stride + slot * a.slot_stride + head * a.head_stride;
    float s = 1.0f;
    if constexpr (Traits<K>::e4m3) s = a.v_scale[page * a.scale_page_stride + slot * a.scale_slot_stride + head * a.scale_head_stride];
    for (int d = 0; d < a.head_dim; d += 8) {
      const uint4 u = values_at<K>(a.v, off, d, s);
      odd |= odd_value<Traits<K>::f16>(u.x) || odd_value<Traits<K>::f16>(u.y) || odd_value<Traits<K>::f16>(u.z) ||
             odd_value<Traits<K>::f16>(u.w);
    }
  }
  return __any_sync(0xFFFFFFFFu, odd) != 0;
}

template <int DP, int K>
__device__ __forceinline__ void softmax_role(const AttnArgs& a, Shared<DP>& sm, uint8_t* qs, const Work& work,
                                             int half, int wtid) {
  using G = Geo<DP>;
  using T = Traits<K>;
  constexpr int type = T::f16 ? MOE_F16 : MOE_BF16, BN = G::bn;
  const int lane = threadIdx.x & 31, warp = wtid >> 5;
  const uint32_t tm = sm.tmem + (static_cast<uint32_t>(warp * 32) << 16);
  const uint32_t oaddr = tm + G::o_col + (G::halves == 2 ? half * G::o_cols : 0);
  uint32_t n_tile = 0, n_piece = 0, tiles = 0;  // this half's tiles and pieces; all tiles of the CTA
  // A piece's queries are on their way while the one before it ends: from its last
  // product with the old ones on their place is free.
  auto load_q = [&](const TileWalk<DP>& u) {
    const int r = half * kHalf + wtid, row0 = u.at.tile * G::rows;
    const int token = static_cast<int>(divide(row0 + min(r, u.tile.rows - 1), a.by_group)), g = row0 + r - token * a.group;
    const uint16_t* q = static_cast<const uint16_t*>(a.query) + (u.seq.first + token) * a.ld_q +
                        static_cast<int64_t>(u.at.head * a.group + g) * a.head_dim;
    const uint32_t dst = smem_u32(qs) + half * G::q_bytes + wtid * 128;
#pragma unroll 4
    for (int p = 0; p < DP / 8; ++p) {
      const bool on = r < u.tile.rows && p * 8 < a.head_dim;
      cp_async16(dst + (p / 8) * (kHalf * 128) + (((p & 7) ^ (wtid & 7)) << 4), on ? q + p * 8 : a.query, on);
    }
    cp_commit();
  };
  auto hand_q = [&] {
    cp_wait<0>();
    fence_async_smem();
    mbar_arrive(&sm.q_full[half]);
  };
  const auto here = [&](const TileWalk<DP>& u) { return u.more() && half * kHalf < u.tile.rows; };
  Pieces<DP> pieces(sm, a);
  if (!pieces.ready(0)) return;
  if (here(pieces.at(0))) {
    load_q(pieces.at(0));
    hand_q();
  }
#pragma unroll 1
  for (; pieces.at(0).more(); pieces.done()) {
    const TileWalk<DP>&w = pieces.at(0), &nx = pieces.at(1);
    const int nt = w.tb - w.ta;
    if (!here(w)) {
      tiles += nt;
      if (!pieces.ready(1)) return;
      if (here(nx)) {
        load_q(nx);
        hand_q();
      }
      continue;
    }
    const int r = half * kHalf + wtid, rc = min(r, w.tile.rows - 1), row0 = w.at.tile * G::rows;
    const bool valid = r < w.tile.rows;
    const int token = static_cast<int>(divide(row0 + rc, a.by_group));
    const int pos = w.seq.len - w.seq.n + token;
    const int lo = sees_from(a, pos), hi = sees_to(a, w.seq.len, pos);
    const bool some = half * kHalf + warp * 32 < w.tile.rows;  // the warp has rows
    const int all_lo = __reduce_max_sync(0xFFFFFFFFu, lo), all_hi = __reduce_min_sync(0xFFFFFFFFu, hi);
    const int ta = w.ta;
    float m = -INFINITY, l = 0.0f;  // m: the reference
    // Exponentials are 2^(scale z + ref) with the reference in ref, or, where that would be
    // rounded too far, 2^(scale (z - base) + ref); large: some row of the warp has a base.
    float base = 0.0f, ref = 0.0f;
    bool large = false;
#pragma unroll 1
    for (int j = 0; j < nt; ++j, ++n_tile, ++tiles) {
      const int buf = G::halves == 2 ? half : n_tile & 1;
      const uint32_t zaddr = tm + buf * G::z_cols;
      if (!wait(sm, a, &sm.z_full[buf], (G::halves == 2 ? n_tile : n_tile >> 1) & 1)) return;
      tc_fence_after();
      if (j == nt - 1) {
        if (!pieces.ready(1)) return;
        if (here(nx)) load_q(nx);
      }
      if (some) {
        constexpr int HB = BN / 2;
        const int first = (ta + j) * BN;
        // Pages may be missing, which is rare: asked for here, looked at when the first
        // exponentials are there, as shared memory answers late beside the products.
        const int holes = *reinterpret_cast<volatile int*>(&sm.holes);
        bool masked = first < all_lo || first + BN > all_hi || large;
        // z (less the base) of 32 positions, -inf where the row does not see
        auto load = [&](int c, float (&z)[32]) {
          tmem_ld32(zaddr + c, z);
          if (masked) {
            tmem_wait();
            // positions from `from` up to `to`, as bits
            const int from = min(max(lo - first - c, 0), 32), to = min(max(hi - first - c, 0), 32);
            const uint32_t see = sm.bits[tiles & 7][c / 32] & (from < 32 ? ~0u << from : 0u) & (to > 0 ? ~0u >> (32 - to) : 0u);
#pragma unroll
            for (int k = 0; k < 32; ++k) z[k] = see & (1u << k) ? z[k] - base : -INFINITY;
          }
        };
        // One half of the positions after the other, in the same few instructions: code
        // that runs once a tile comes from afar each time.
#pragma unroll 1
        for (int hb = 0; hb < 2; ++hb) {
          uint32_t p[HB / 32][16];
          float sum;
          bool go = hb == 0 && j == 0, far = true;
#pragma unroll 1
          for (;;) {
            if (go) {
              // the reference moves to the maximum from here on, o (products under way
              // first) and l with it
              masked |= holes != 0;
              const bool scale_o = j > 0 || hb > 0;
              if (hb > 0 && !wait(sm, a, &sm.half_done[buf], (G::halves == 2 ? n_tile : n_tile >> 1) & 1)) return;
              if (G::halves == 1 && hb == 0 && j > 0 && !wait(sm, a, &sm.pv_done, (n_tile - 1) & 1)) return;
              float top = -INFINITY;
              base = 0.0f;
#pragma unroll 1
              for (int c = hb * HB; c < BN; c += 32) {
                float z[32];
                load(c, z);
                tmem_wait();
#pragma unroll
                for (int k = 0; k < 32; k += 2) top = fmaxf(fmaxf(top, z[k]), z[k + 1]);
              }
              const float f = far && top > m ? exp2_approx((m - top) * a.scale_log2) : 1.0f;
              if (far && top > m) m = top;
              l *= f;
              const float scaled = m == -INFINITY ? 0.0f : m * a.scale_log2;
              const bool mine = !(fabsf(scaled) <= kLarge);
              base = mine ? m : 0.0f, ref = mine ? tile_lift<T::f16>() : tile_lift<T::f16>() - scaled;
              large = __any_sync(0xFFFFFFFFu, mine);
              masked |= large;
              if (scale_o) {
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < DP; c += 16) {
                  uint32_t x[8], y[8], v[16];
                  tmem_ld8(oaddr + c, x);
                  tmem_ld8(oaddr + c + 8, y);
                  tmem_wait();
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    v[i] = __float_as_uint(__uint_as_float(x[i]) * f), v[8 + i] = __float_as_uint(__uint_as_float(y[i]) * f);
                  tmem_st16(oaddr + c, v);
                }
              }
            }
            // exponentials, as 16-bit values in p, and their sum
            float z[HB / 32][32], s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < HB / 32; ++c) load(hb * HB + 32 * c, z[c]);
            tmem_wait();
#pragma unroll
            for (int c = 0; c < HB / 32; ++c)
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                float x0 = z[c][k], x1 = z[c][k + 1], x2 = z[c][k + 2], x3 = z[c][k + 3];
                fma_pair(x0, x1, a.scale_log2, ref);
                fma_pair(x2, x3, a.scale_log2, ref);
                x0 = exp2_approx(x0), x1 = exp2_approx(x1), x2 = exp2_approx(x2), x3 = exp2_approx(x3);
                add_pair(s[0], s[1], x0, x1);
                add_pair(s[2], s[3], x2, x3);
                p[c][k / 2] = pack2(x0, x1, type), p[c][k / 2 + 1] = pack2(x2, x3, type);
              }
            sum = (s[0] + s[1]) + (s[2] + s[3]);
            if (go) break;
            // a row that has seen nothing yet has no reference
            far = sum > kMost || m == -INFINITY;
            go = __any_sync(0xFFFFFFFFu, far || (holes != 0 && !masked));
            if (!go) break;
          }
          l += sum;
#pragma unroll
          for (int c = 0; c < HB / 32; ++c) tmem_st16(zaddr + hb * (HB / 2) + 16 * c, p[c]);
          tmem_wait_st();
          if (hb == 0) {
            tc_fence_before();
            mbar_arrive(&sm.p_half[buf]);
          }
        }
      } else {
        mbar_arrive(&sm.p_half[buf]);
      }
      tc_fence_before();
      mbar_arrive(&sm.p_ready[buf]);
    }
    if (here(nx)) hand_q();

    // the piece is done: this thread's row
    if (!wait(sm, a, &sm.o_full[half], n_piece++ & 1)) return;
    tc_fence_after();
    if (!some) {
      tc_fence_before();
      continue;
    }
    const bool whole = w.whole();
    const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (w.ta == w.tile.t0 ? 1 : 0);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int head = w.at.head * a.group + (row0 + rc - token * a.group);
    const int64_t row = w.seq.first + token;
    uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.ld_out + static_cast<int64_t>(head) * a.head_dim;
    float* po = a.part_o + (part * G::rows + r) * a.head_dim;
    bool fine = true;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
#pragma unroll 1
    for (int c = 0; c < DP; c += 32) {
      float v[32];
      tmem_ld32(oaddr + c, v);
      tmem_wait();
#pragma unroll
      for (int i = 0; i < 32; i += 16) {
        if (c + i >= a.head_dim) continue;
#pragma unroll
        for (int k = 0; k < 16; ++k) fine &= fabsf(v[i + k]) < INFINITY;
        if (!valid) continue;
        if (whole) {
          uint32_t x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = pack2(v[i + 2 * k] * inv, v[i + 2 * k + 1] * inv, type);
          if (wide) {
            store32(out + c + i, x);
          } else {
            *reinterpret_cast<uint4*>(out + c + i) = make_uint4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<uint4*>(out + c + i + 8) = make_uint4(x[4], x[5], x[6], x[7]);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
            uint32_t x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = __float_as_uint(v[i + h + k]);
            store32(po + c + i + h, x);
          }
        }
      }
    }
    tc_fence_before();
    if (valid) {
      if (!whole) {
        float* ml = a.part_ml + (part * G::rows + r) * 2;
        ml[0] = m, ml[1] = l;
      } else if (a.lse) {
        a.lse[row * a.kv_heads * a.group + head] = l == 0.0f ? -INFINITY : fmaf(m, a.scale, (log2f(l) - tile_lift<T::f16>()) * kLn2);
      }
    }
    // rows that an unseen value of the tiles may have spoilt
    __syncwarp();
    const int k0 = w.ta * BN, k1 = min(w.tb * BN, w.seq.len);
    const int v0 = min(max(k0, lo), max(k0, k1)), v1 = min(k1, hi);
    for (uint32_t bad = __ballot_sync(0xFFFFFFFFu, valid && !fine && (v0 > k0 || v1 < k1)); bad; bad &= bad - 1) {
      const int src = __ffs(bad) - 1;
      const int b0 = __shfl_sync(0xFFFFFFFFu, v0, src), b1 = __shfl_sync(0xFFFFFFFFu, v1, src);
      const bool odd = odd_values<K>(a, w.at.seq, w.at.head, k0, min(b0, k1)) || odd_values<K>(a, w.at.seq, w.at.head, max(b1, k0), k1);
      if (!odd) continue;
      const float mr = __shfl_sync(0xFFFFFFFFu, m, src), f = __shfl_sync(0xFFFFFFFFu, inv, src);
      const uint16_t* q = static_cast<const uint16_t*>(a.query) + row * a.ld_q + static_cast<int64_t>(head) * a.head_dim;
      const uint16_t* qr = reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uintptr_t>(q), src));
      uint16_t* orow = reinterpret_cast<uint16_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uintptr_t>(out), src));
      float* prow = reinterpret_cast<float*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uintptr_t>(po), src));
      float o[(DP + 127) / 128][4];
      row_again<DP, K>(a, w.at.seq, w.at.head, qr, b0, b1, mr == -INFINITY ? 0.0f : mr, o);
#pragma unroll
      for (int i = 0; i < (DP + 127) / 128; ++i) {
        const int d = 4 * lane + 128 * i;
        if (d < a.head_dim) {
          if (whole)
            *reinterpret_cast<uint2*>(orow + d) = make_uint2(pack2(o[i][0] * f, o[i][1] * f, type), pack2(o[i][2] * f, o[i][3] * f, type));
          else
            *reinterpret_cast<float4*>(prow + d) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        }
      }
    }
    if (!whole && half == 0 && wtid == 0) w.note(a, work);
  }
}

// Tiled loads of the cache's pages: boxes of `rows` positions of one head (0: pages
// that no box of 8 positions divides, or no pages).
struct alignas(64) Maps {
  CUtensorMap k, v;
  int rows;
  Divisor row_boxes;  // boxes that a slab of a tile takes
};

// Box of 64 elements and `rows` slots of (head, page) to shared memory,
// completion counted on `bar` in bytes; elements past the head's end are zeros.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int d, int slot, int head, int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(d), "r"(slot), "r"(head), "r"(page), "r"(smem_u32(bar))
      : "memory");
}

template <int DP, int K>
__device__ __forceinline__ void producer_role(const AttnArgs& a, const Maps& maps, Shared<DP>& sm, uint8_t* ring, int tid) {
  using G = Geo<DP>;
  using T = Traits<K>;
  constexpr int BN = G::bn;
  constexpr int PR = DP * T::size / 16;      // 16-byte pieces of a position in the cache
  constexpr int PER = BN * PR / 128;         // of a tile, for each thread
  const int lane = tid & 31, warp = tid >> 5;
  const int pieces = a.head_dim * T::size / 16;
  const uint32_t ring_s = smem_u32(ring);
  RingPos load;
  uint32_t tiles = 0, groups = 0, tails = 0;
  // thread t looks up position t of the next tile
  int page = -1, slot = 0, head = 0;
  bool seen = false;
  struct View {
    int first, nt, lo, hi, seq, head, len;
  };
  Pieces<DP> ps(sm, a);
  auto view = [&] {
    const TileWalk<DP>& w = ps.at(0);
    if (!w.more()) return View{0, 0, 0, 0, 0, 0, 0};
    return View{w.ta * BN, w.tb - w.ta, w.tile.lo, w.tile.hi, w.at.seq, w.at.head, w.seq.len};
  };
  auto look_up = [&](const View& u, int j) {
    page = -1, slot = 0, head = u.head;
    const int pos = u.first + j * BN + tid;
    if (tid < BN && pos < u.len) page = page_of(a.q, u.seq, pos, slot);
    const bool counts = tid < BN && pos >= u.lo && pos < u.hi;
    seen = page >= 0 && counts;
    if (counts && page < 0) *reinterpret_cast<volatile int*>(&sm.holes) = 1;
  };
  // The looked-up tile, for all producers.
  auto post = [&] {
    if (tid < BN) {
      const uint32_t on = __ballot_sync(0xFFFFFFFFu, seen);
      sm.off[tiles & 3][tid] = seen ? page * a.page_stride + slot * a.slot_stride + head * a.head_stride : -1;
      sm.place[tiles & 3][tid] = make_int2(page, slot);
      if (lane == 0) sm.bits[tiles & 7][warp] = on;
    }
    named_bar(1, 128);
  };
  if (!ps.ready(0)) return;
  View u = view();
  look_up(u, 0);
  while (u.nt > 0) {
    const int nt = u.nt;
    ps.done();
    if (!ps.ready(0)) return;
    const View after = view();
#pragma unroll 1
    for (int j = 0; j < nt; ++j, ++tiles) {
      post();
      if (j + 1 < nt) look_up(u, j + 1);
      else if (after.nt > 0) look_up(after, 0);
      const int64_t* offs = sm.off[tiles & 3];
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++groups) {
        if (groups >= G::stages && !wait(sm, a, &sm.empty[load.s], load.ph ^ 1)) return;
        const uint32_t dst = ring_s + load.s * G::stage_bytes;
        if (maps.rows) {
          // The slots behind the sequence's end may hold anything: the values there become
          // zeros before the products see them.  What has no page is out of the tensor's bounds: zeros.
          const int held = u.len - (u.first + j * BN);
          uint64_t* bar = kv && held < BN ? &sm.tail : &sm.full[load.s];
          if (tid == 0) mbar_arrive_expect_tx(bar, G::stage_bytes);
          else if (bar != &sm.tail) mbar_arrive(bar);
          // lanes issue boxes one after the other, so the warps take turns
          const int box = lane * 4 + warp, slab = static_cast<int>(divide(box, maps.row_boxes)),
                    row = (box - slab * static_cast<int>(maps.row_boxes.d)) * maps.rows;
          if (slab < DP / 64) {
            const int2 at = sm.place[tiles & 3][row];
            load_box(dst + slab * (BN * 128) + row * 128, kv ? &maps.v : &maps.k, slab * 64, at.y, u.head,
                     at.x < 0 ? a.q.n_pages : at.x, bar);
          }
          if (bar == &sm.tail) {
            if (!wait(sm, a, bar, tails++ & 1)) return;
            if (tid < BN && tid >= held)
#pragma unroll 4
              for (int c = 0; c < DP / 8; ++c)
                *reinterpret_cast<uint4*>(ring + load.s * G::stage_bytes + (c / 8) * (BN * 128) + tid * 128 + (c & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            fence_async_smem();
            mbar_arrive(&sm.full[load.s]);
          }
        } else {
          // pages that no box of 8 positions divides: what does not count is zeros
          const uint8_t* base = static_cast<const uint8_t*>(kv ? a.v : a.k);
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int n = tid + 128 * i, row = n / PR, c = n % PR;
            const int64_t o = offs[row];
            const bool on = o >= 0 && c < pieces;
            cp_async16(dst + (c / 8) * (BN * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                       on ? static_cast<const void*>(base + o + c * 16) : a.query, on);
          }
          cp_commit();
          cp_wait<0>();
          fence_async_smem();
          mbar_arrive(&sm.full[load.s]);
        }
        load.next(G::stages);
      }
    }
    u = after;
  }
}

__device__ const uint4 zeros[16] = {};

// As above for e4m3 caches: codes wait in registers, half a tile ahead, and
// become 16-bit values on their way to shared memory.  A warp has a quarter of each tile's
// positions: it looks them up, a lane each, and copies them, as many lanes a position as
// it has 16-byte pieces; so the warps exchange nothing but which positions count.
// Bound by these warps' own instructions, so what can be done once a position or tile
// is: scales and addresses are made by the lane that looked a position up, one of
// zeros stands for what does not count, pages are asked for half a tile before
// their use.  2048 rows over 4096 positions of 8 heads of 128, queries of 64, in a graph:
// bf16 221 us, float16 206, 16-bit caches 190 and 194.  (bf16 codes turned bit by bit, which
// takes a NaN's code for 480, 213; with a look for such codes 237.)
template <int DP, int K>
__device__ __forceinline__ void dequant_role(const AttnArgs& a, Shared<DP>& sm, uint8_t* ring, int tid) {
  using G = Geo<DP>;
  using T = Traits<K>;
  constexpr int BN = G::bn, MINE = BN / 4, PR = DP / 16, STEP = 32 / PR, PER = MINE / STEP;
  const int lane = tid & 31, warp = tid >> 5;
  const int c = lane % PR, sub = lane / PR;  // the lane's piece, and its first position of the warp's
  const bool on = c < a.head_dim / 16;
  RingPos load;
  uint32_t tiles = 0, groups = 0;
  int64_t off = -1;  // of the position that this lane looked up (-1: not seen)
  float ks = 1.0f, vs = 1.0f;
  Pieces<DP> ps(sm, a);
  int page = -1, slot = 0, head = 0;
  bool counts = false;
  auto look_up = [&](int j) {  // tile j of the piece: asks for the pages
    const TileWalk<DP>& w = ps.at(0);
    const int pos = (w.ta + j) * BN + warp * MINE + lane;
    counts = lane < MINE && pos >= w.tile.lo && pos < w.tile.hi, head = w.at.head;
    if (counts) {
      const uint32_t i = divide(static_cast<uint32_t>(pos), a.q.page);
      slot = pos - static_cast<int>(i * a.q.page.d), page = a.q.table[w.at.seq * a.q.ld_table + i];
    }
  };
  auto look_at = [&] {  // when they have come
    off = -1, ks = vs = 1.0f;
    if (counts) {
      if (page < 0 || page >= a.q.n_pages) {
        *reinterpret_cast<volatile int*>(&sm.holes) = 1;
      } else {
        off = page * a.page_stride + slot * a.slot_stride + head * a.head_stride;
        const int64_t s = page * a.scale_page_stride + slot * a.scale_slot_stride + head * a.scale_head_stride;
        ks = a.k_scale[s], vs = a.v_scale[s];
      }
    }
  };
  auto fetch = [&](uint4 (&b)[PER], const void* base) {
    // of a position that does not count, zeros
    const uint64_t mine = off >= 0 ? reinterpret_cast<uint64_t>(base) + off : reinterpret_cast<uint64_t>(zeros);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint64_t at = __shfl_sync(0xFFFFFFFFu, mine, sub + STEP * i) + c * 16;
      if (on) b[i] = *reinterpret_cast<const uint4*>(at);
    }
  };
  auto store = [&](const uint4 (&b)[PER], float scale) {
    if (groups >= G::stages && !wait(sm, a, &sm.empty[load.s], load.ph ^ 1)) return false;
    uint8_t* dst = ring + load.s * G::stage_bytes + (c / 4) * (BN * 128);
    // a lane prepares its position's scale; the second product's code is there twice, so that no row asks
    const Dequant<T::f16> mine(scale);
    auto rows = [&](auto twice) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int at = sub + STEP * i, row = warp * MINE + at;
        const Dequant<T::f16> dq = mine.of(at, twice);
        // the second slab's lanes begin with their second half: its rows lie in the first one's banks
        const int p = (2 * c) & 7, odd = c >> 2 & 1;
        const uint32_t x[4] = {odd ? b[i].z : b[i].x, odd ? b[i].w : b[i].y, odd ? b[i].x : b[i].z, odd ? b[i].y : b[i].w};
        uint32_t v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          dq(x[k], v + 2 * k, twice);
        *reinterpret_cast<uint4*>(dst + row * 128 + (((p + odd) ^ (row & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<uint4*>(dst + row * 128 + (((p + 1 - odd) ^ (row & 7)) << 4)) = make_uint4(v[4], v[5], v[6], v[7]);
      }
    };
    if (mine.twice) rows(Bool<true>{});
    else rows(Bool<false>{});
    fence_async_smem();
    mbar_arrive(&sm.full[load.s]);
    load.next(G::stages);
    ++groups;
    return true;
  };
  auto tiles_of = [&] { return ps.at(0).more() ? ps.at(0).tb - ps.at(0).ta : 0; };
  uint4 kb[PER], vb[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) kb[i] = vb[i] = make_uint4(0, 0, 0, 0);  // stays behind a head's end
  if (!ps.ready(0)) return;
  int j = 0, nt = tiles_of();
  if (nt == 0) return;
  look_up(0);
  look_at();
  fetch(kb, a.k);
  for (;;) {
    fetch(vb, a.v);
    const float k_scale = ks, v_scale = vs;
    // which positions count, before the keys are handed over
    const uint32_t seen = __ballot_sync(0xFFFFFFFFu, off >= 0);
    if (lane == 0) {
      if (MINE == 32) sm.bits[tiles & 7][warp] = seen;
      else reinterpret_cast<uint16_t*>(sm.bits[tiles & 7])[warp] = static_cast<uint16_t>(seen);
    }
    ++tiles;
    if (++j == nt) {
      ps.done();
      if (!ps.ready(0)) return;
      j = 0, nt = tiles_of();
    }
    const bool more = nt > 0;
    if (more) look_up(j);
    if (!store(kb, k_scale)) return;
    if (more) {
      look_at();
      fetch(kb, a.k);
    }
    if (!store(vb, v_scale)) return;
    if (!more) return;
  }
}

template <int DP, int K>
__device__ __forceinline__ void mma_role(const AttnArgs& a, Shared<DP>& sm, uint32_t qs, uint32_t ring) {
  using G = Geo<DP>;
  using T = Traits<K>;
  constexpr int BN = G::bn;
  constexpr uint32_t id_z = idesc<T::f16>(BN, false), id_o = idesc<T::f16>(DP, true);
  const uint32_t tm = sm.tmem;
  RingPos p;                  // next tile to take, keys and values in turn
  uint32_t ph_p = 0, ph_q = 0;  // parities of p_ready (by half or buffer) and of q_full, a bit each
  uint32_t tile0 = 0;         // one half: parity of the piece's first tile, which names its buffer
  auto flip = [](uint32_t& ph, int i) {
    const uint32_t was = ph >> i & 1;
    ph ^= 1u << i;
    return was;
  };
  const bool lead = elect();
  // loops stay rolled: the code of eight products is fetched anew each time, of one it is at hand
  auto z_product = [&](int half, int buf, int stage) {
    uint32_t k0 = desc_lo(ring + stage * G::stage_bytes, 16), q0 = desc_lo(qs + half * G::q_bytes, 16);
    if (lead) {
#pragma unroll 1
      for (int c = 0; c < DP / 64; ++c, q0 += kHalf * 128 / 16, k0 += BN * 128 / 16)
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_ss(tm + buf * G::z_cols, q0 + k * 2, k0 + k * 2, id_z, c > 0 || k > 0);
      mma_commit(smem_u32(&sm.z_full[buf]));
    }
  };
  // the first half of the positions, then the second: their exponentials come one after the other
  auto o_product = [&](int half, int buf, int stage, bool more) {
    const uint32_t parity = flip(ph_p, buf);
    uint32_t v0 = desc_lo(ring + stage * G::stage_bytes, BN * 128), p0 = tm + buf * G::z_cols;
#pragma unroll 1
    for (int c = 0; c < 2; ++c, v0 += BN / 32 * 128, p0 += BN / 4) {
      if (!wait(sm, a, c ? &sm.p_ready[buf] : &sm.p_half[buf], parity)) return false;
      tc_fence_after();
      if (lead) {
#pragma unroll
        for (int k = 0; k < BN / 32; ++k)
          mma_ts(tm + G::o_col + (G::halves == 2 ? half * G::o_cols : 0), p0 + k * 8, v0 + k * 128, id_o, more || c > 0 || k > 0);
        if (c == 0) mma_commit(smem_u32(&sm.half_done[buf]));
      }
    }
    return true;
  };
  auto commit = [&](uint64_t* bar) {
    if (lead) mma_commit(smem_u32(bar));
  };
  auto take = [&](RingPos& r) {  // waits for the tile at r and steps on; its stage, or -1
    if (!wait(sm, a, &sm.full[r.s], r.ph)) return -1;
    const int s = r.s;
    r.next(G::stages);
    return s;
  };
  Pieces<DP> ps(sm, a);
#pragma unroll 1
  for (;; ps.done()) {
    if (!ps.ready(0) || !ps.at(0).more()) return;
    const int nt = ps.at(0).tb - ps.at(0).ta;
    if constexpr (G::halves == 2) {
      const int halves = ps.at(0).tile.rows > kHalf ? 2 : 1;
      int ks = take(p);
      if (ks < 0) return;
      for (int h = 0; h < halves; ++h) {
        if (!wait(sm, a, &sm.q_full[h], flip(ph_q, h))) return;
        tc_fence_after();
        z_product(h, h, ks);
      }
      commit(&sm.empty[ks]);
      for (int j = 0; j < nt; ++j) {
        const int vs = take(p);
        if (vs < 0) return;
        if (j + 1 < nt) ks = p.s;  // the next keys follow these values
        for (int h = 0; h < halves; ++h) {
          if (!o_product(h, h, vs, j > 0)) return;
          if (h == halves - 1) commit(&sm.empty[vs]);
          if (j + 1 < nt) {
            if (h == 0 && take(p) < 0) return;
            z_product(h, h, ks);
            if (h == halves - 1) commit(&sm.empty[ks]);
          } else {
            commit(&sm.o_full[h]);
          }
        }
      }
    } else {
      // tiles in the ring: k0 v0 k1 v1 ...; products: z0 z1 o0 z2 o1 ...
      if (!wait(sm, a, &sm.q_full[0], flip(ph_q, 0))) return;
      tc_fence_after();
      const uint32_t base = tile0;
      tile0 = (tile0 + nt) & 1;
      int ks = take(p);
      if (ks < 0) return;
      z_product(0, base & 1, ks);
      commit(&sm.empty[ks]);
      for (int j = 0; j < nt; ++j) {
        RingPos v = p;
        p.next(G::stages);
        if (j + 1 < nt) {
          ks = take(p);
          if (ks < 0) return;
          z_product(0, (base + j + 1) & 1, ks);
          commit(&sm.empty[ks]);
        }
        const int vs = take(v), buf = (base + j) & 1;
        if (vs < 0 || !o_product(0, buf, vs, j > 0)) return;
        commit(&sm.empty[vs]);
        commit(&sm.pv_done);
        if (j + 1 == nt) commit(&sm.o_full[0]);
      }
    }
  }
}

template <int DP, int K>
__global__ void __launch_bounds__(kThreads, 1) attention_tiles_kernel(const AttnArgs a, const __grid_constant__ Maps maps) {
  using G = Geo<DP>;
  extern __shared__ uint8_t raw[];
  __shared__ Shared<DP> sm;
  uint8_t* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t* ring = base + G::halves * G::q_bytes;
  const int tid = threadIdx.x, warp = tid >> 5;
  pdl_launch_dependents();
  if (warp == 12) tmem_alloc(smem_u32(&sm.tmem), 512);
  if (tid == kThreads - 1) {
    for (int i = 0; i < G::stages; ++i) mbar_init(&sm.full[i], 128), mbar_init(&sm.empty[i], 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(&sm.z_full[i], 1), mbar_init(&sm.half_done[i], 1), mbar_init(&sm.p_half[i], kHalf), mbar_init(&sm.p_ready[i], kHalf), mbar_init(&sm.o_full[i], 1),
          mbar_init(&sm.q_full[i], kHalf);
    mbar_init(&sm.pv_done, 1), mbar_init(&sm.tail, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&sm.piece_full[i], 1), mbar_init(&sm.piece_empty[i], 4 * G::halves + 4 + 1);
    sm.failed = sm.holes = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  tc_fence_before();
  const Work work = find_work<G::rows, G::bn, kThreads>(a, sm.plan);
  if (tid < 2) a.notes[2 * blockIdx.x + tid].count = 0;
  tc_fence_after();  // find_work's barriers lie between
  if (work.begin == work.end) {
    if (warp == 12) tmem_dealloc(sm.tmem, 512);
    return;
  }
  {
    // registers of the roles' 128 threads: 2 x 184 + 96 + 48 or 2 x 160 + 144 + 48 = 4 x 128
    constexpr bool e4m3 = Traits<K>::e4m3;
    if (warp < 8) {
      reg_up<e4m3 ? 160 : 184>();
      if (warp < 4 * G::halves) softmax_role<DP, K>(a, sm, base, work, warp >> 2, tid & 127);
    } else if (warp < 12) {
      if constexpr (e4m3) {
        reg_up<144>();
        dequant_role<DP, K>(a, sm, ring, tid - 256);
      } else {
        reg_down<96>();
        producer_role<DP, K>(a, maps, sm, ring, tid - 256);
      }
    } else {
      reg_down<48>();
      if (warp == 12) mma_role<DP, K>(a, sm, smem_u32(base), smem_u32(ring));
      else if (warp == 13) walk_role<DP>(a, sm, work);
    }
  }
  if (tid == 384 && *reinterpret_cast<volatile int*>(&sm.failed)) {
    // products in flight end before the memory they use is given back
    mma_commit(smem_u32(&sm.pv_done));
    const unsigned long long t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {}
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(sm.tmem, 512);
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(p) : nullptr;
  }();
  return fn;
}

// The tensor (elements, slots, heads, pages) of keys or values of a 16-bit
// cache.  False if the driver refuses it, or strides that it would refuse: tiles are
// then copied in pieces, as for pages that no box of 8 positions divides.
bool encode(CUtensorMap* map, const void* base, const AttnArgs& a, int rows, bool f16) {
  const EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.head_dim), a.q.page.d, static_cast<cuuint64_t>(a.kv_heads),
                              static_cast<cuuint64_t>(a.q.n_pages)};
  // a stride of 0 belongs to a dimension of 1 (or to places that are the same): any other does as well for the former
  const auto step = [](int64_t s, cuuint64_t n) { return static_cast<cuuint64_t>(n == 1 && s == 0 ? 16 : s); };
  const cuuint64_t strides[3] = {step(a.slot_stride, dims[1]), step(a.head_stride, dims[2]), step(a.page_stride, dims[3])};
  for (const cuuint64_t s : strides)
    if (s == 0 || s >= (1ull << 40)) return false;
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1}, one[4] = {1, 1, 1, 1};
  return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
            one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, int K>
cudaError_t launch(const AttnArgs& a, int num_sms, cudaStream_t st) {
  auto kernel = attention_tiles_kernel<DP, K>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(allowed, kernel, Geo<DP>::smem);
  if (e) return e;
  Maps maps = {};
  maps.row_boxes = divisor(1);
  if (!Traits<K>::e4m3 && a.q.n_pages > 0) {
    // the largest power of two that divides a page, up to a tile; a box starts on a swizzle's 1024 bytes from 8 on
    int rows = static_cast<int>(a.q.page.d & (0u - a.q.page.d));
    if (rows > Geo<DP>::bn) rows = Geo<DP>::bn;
    if (rows >= 8 && encode(&maps.k, a.k, a, rows, Traits<K>::f16) && encode(&maps.v, a.v, a, rows, Traits<K>::f16)) {
      maps.rows = rows;
      maps.row_boxes = divisor(static_cast<uint32_t>(Geo<DP>::bn / rows));
    }
  }
  kernel<<<num_sms, kThreads, Geo<DP>::smem, st>>>(a, maps);
  return cudaGetLastError();
}

template <int DP>
cudaError_t launch(const AttnArgs& a, Kind k, int num_sms, cudaStream_t st) {
  switch (k) {
    case kBf16: return launch<DP, kBf16>(a, num_sms, st);
    case kF16: return launch<DP, kF16>(a, num_sms, st);
    case kE4m3Bf16: return launch<DP, kE4m3Bf16>(a, num_sms, st);
    default: return launch<DP, kE4m3F16>(a, num_sms, st);
  }
}

}  // namespace

int tiles_rows(int head_dim) { return head_dim <= 64 ? Geo<64>::rows : head_dim <= 128 ? Geo<128>::rows : Geo<256>::rows; }
int tiles_keys(int head_dim) { return head_dim <= 64 ? Geo<64>::bn : head_dim <= 128 ? Geo<128>::bn : Geo<256>::bn; }
float tiles_lift(bool f16) { return f16 ? tile_lift<true>() : tile_lift<false>(); }

cudaError_t launch_tiles(const AttnArgs& a, Kind k, int num_sms, cudaStream_t st) {
  return a.head_dim <= 64    ? launch<64>(a, k, num_sms, st)
         : a.head_dim <= 128 ? launch<128>(a, k, num_sms, st)
                             : launch<256>(a, k, num_sms, st);
}

}  // namespace moe
