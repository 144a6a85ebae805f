// attention.cu -- attention of few rows over the paged cache, the join of units
// that several CTAs share, and the entry points (include/moe_cache.h).
//
// Mathematics: a row's softmax over its positions is taken in one pass with a
// running maximum m of z = q . k, sum l of 2^(c (z - m)) with c = scale * log2(e),
// and output o, all fp32; when m grows, l and o shrink by 2^(c (old - new)).  m is subtracted
// before the scale is multiplied on: exact near the maximum, however large z is (c z
// rounded before the subtraction is off by 2 from 2^25 on, by 128 from 2^31 on).
// Parts of the positions, of one warp, one CTA or several, join the same way.
//
// Layout: a unit's tile has 8 or 16 rows (attention.cuh).  A CTA of four warps takes 64
// positions at a time, each warp 16 of its own, with its own m, l and o, so
// that warps never wait for one another until the unit ends.  Each warp copies its
// positions' keys and values to a ring of stages in shared memory (cp.async, 16
// bytes a lane), several steps and units ahead.  Products are m16n8k16 tensor-core
// instructions with positions, then a head's elements, as M and rows as N, so that no
// half of them is empty for 8 rows (heads of few rows leave tcgen05's 128 idle, and the
// cache's bytes bound them).  The sum over a head's elements may run in any order, so
// each lane reads keys in whole 16-byte pieces and takes the query's elements in
// the same order; the outputs' order is free likewise, so values are read in 16-byte
// pieces of four positions and paired in registers.  Exponentials are turned over
// (movmatrix) between the products.  e4m3 codes become float16 values between shared
// memory and the product, a conversion for two; the keys' scales are multiplied on
// z, the values' on the exponentials, which makes a row's weights.  A weight is rounded to
// float16 in the row's own unit, a power of two that its largest weight so far has set and
// o follows: positions that a row does not see, or that weigh nothing, have no part in it.
//
// Bound: reading the cache.
#include <atomic>

#include <cuda_runtime.h>

#include "attention.cuh"

namespace moe {
int reportf(int code, const char* fmt, ...);

namespace {

// log2 of the factor that all exponentials carry: float16 holds fewer small
// values than large ones, so the largest exponential is 2^15 there.
// Weights of an e4m3 cache have units instead.
template <int K>
__host__ __device__ constexpr float exp_lift() {
  return K == kF16 ? 15.0f : 0.0f;
}
// The largest weight moves a row's unit so that it is 2^kUnitTop at most; smaller
// ones are rounded to 11 bits down to 2^-(14 + kUnitTop) of it, then to multiples of 2^-(24 + kUnitTop).
// The unit stays until a weight passes 2^kUnitMost, so that it seldom moves.
constexpr int kUnitTop = 10, kUnitMost = 14;
constexpr float kLowest = -3.402823466e38f;  // the maximum of no positions

constexpr int kRows = 16;     // rows of the larger tile
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;     // positions of a warp's step
constexpr int kBn = kWarps * kStep;
constexpr int kJoinRows = 4;  // of a unit that the warps join at once
constexpr size_t kCtlBytes = 256;

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DP, int K, int R>
struct Shape {
  using T = Traits<K>;
  static constexpr int row_bytes = DP * T::size;            // of one position in shared memory
  static constexpr int pieces = row_bytes / 16;             // 16-byte pieces of it
  static constexpr int ev = T::e4m3 && DP >= 128 ? 16 : 8;  // elements of a lane's piece of values
  static constexpr int vgroups = DP / (8 * ev);
  static constexpr int scale_bytes = T::e4m3 ? 2 * kStep * 4 : 0;
  static constexpr int stage_bytes = 2 * kStep * row_bytes + scale_bytes + 16;  // 16: which positions count
  // On an SM: as many warps as registers and two stages of each allow.  64 ragged e4m3
  // sequences with 8 rows of 128: two CTAs 138 us, three 123.
  static constexpr int ctas = DP <= 64 || (row_bytes <= 128 && R == 8) ? 3 : DP <= 128 ? 2 : 1;
  static constexpr bool q_shared = DP > 128 && R > 8;       // the query's fragments lie in shared memory
  static constexpr int join_bytes = kWarps * kJoinRows * DP * 4;
  static constexpr int q_bytes = q_shared ? DP / 16 * (R / 8) * 256 : 0;
  static constexpr int budget = (224 * 1024 / ctas - 5 * 1024 - join_bytes - q_bytes) / kWarps;
  static constexpr int fit = budget / stage_bytes;
  static constexpr int stages = fit > 8 ? 8 : fit;
  static constexpr int ring_bytes = stages * stage_bytes;   // of a warp
  static constexpr int smem = kWarps * ring_bytes + join_bytes + q_bytes;
  static_assert(stages >= 2, "ring");
};

// Swizzles that spread a phase's lanes over the banks: keys are read in pieces
// t = 0..3 of two neighbouring rows at a time, values in two pieces of every
// other row.
template <int RB>
__device__ __forceinline__ uint32_t key_at(int row, int piece) {
  return row * RB + ((RB >= 128 ? piece ^ ((row & 1) << 2) : piece) << 4);
}
template <int RB>
__device__ __forceinline__ uint32_t value_at(int row, int piece) {
  return row * RB + ((RB >= 128 ? piece ^ (row & 6) : piece) << 4);
}

__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// The codes in a word's low or high half as float16 values.
__device__ __forceinline__ uint32_t two_codes(uint32_t w, int high) {
  const __half2 v(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(high ? w >> 16 : w), __NV_E4M3));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// x, or the largest finite value for more; NaN stays.
__device__ __forceinline__ float finite(float x) {
  float y;
  asm("min.NaN.f32 %0, %1, 0f7F7FFFFF;" : "=f"(y) : "f"(x));
  return y;
}

// An 8 x 8 matrix of 16-bit values, two of row gi a lane, turned over.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// A lane's pieces of values of one group: positions 2t, 2t + 1, 2t + 8, 2t + 9.
template <int DP, int K, int R>
struct Values {
  using S = Shape<DP, K, R>;
  uint32_t w[4][S::ev == 16 || !Traits<K>::e4m3 ? 4 : 2];
  __device__ __forceinline__ void load(const uint8_t* v, int t, int gi, int h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 2 * t + (i & 1) + (i & 2) * 4;
      if constexpr (S::ev == 8 && Traits<K>::e4m3) {
        const uint2 u = *reinterpret_cast<const uint2*>(v + row * S::row_bytes + (gi + 8 * h) * 8);
        w[i][0] = u.x, w[i][1] = u.y;
      } else {
        const uint4 u = lds128(v + value_at<S::row_bytes>(row, gi + 8 * h));
        w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
      }
    }
  }
  // element j of the piece: the pairs of positions (2t, 2t + 1) and (2t + 8, 2t + 9);
  // of e4m3 codes the values without their scales
  __device__ __forceinline__ void pair(int j, uint32_t& b0, uint32_t& b1) const {
    if constexpr (Traits<K>::e4m3) {
      const uint32_t s = j & 2 ? 0x7362u : 0x5140u;  // elements j and j + 1 of both positions
      b0 = two_codes(bytes_of(w[0][j / 4], w[1][j / 4], s), j & 1);
      b1 = two_codes(bytes_of(w[2][j / 4], w[3][j / 4], s), j & 1);
    } else {
      const uint32_t s = j & 1 ? 0x7632u : 0x5410u;
      b0 = bytes_of(w[0][j / 2], w[1][j / 2], s);
      b1 = bytes_of(w[2][j / 2], w[3][j / 2], s);
    }
  }
};

template <int DP, int K, int R>
__global__ void __launch_bounds__(kThreads, Shape<DP, K, R>::ctas) attention_rows_kernel(const AttnArgs a) {
  using S = Shape<DP, K, R>;
  using RowWalk = Walk<R, kBn>;
  using T = Traits<K>;
  constexpr int RB = S::row_bytes, KS = DP / 16, MB = DP / 16, NB = R / 8, EV = S::ev;
  constexpr int half_type = T::f16 ? MOE_F16 : MOE_BF16;  // of the exponentials
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PlanSmem plan;
  __shared__ RowWalk walks[2][kWarps];       // of the pieces that are worked on, and of those that are loaded
  __shared__ float join_ml[kWarps][R][2];
  float* join_o = reinterpret_cast<float*>(smem + kWarps * S::ring_bytes);                     // [warp][kJoinRows][DP]
  uint2* q_frag = reinterpret_cast<uint2*>(smem + kWarps * S::ring_bytes + S::join_bytes);     // [KS][NB][lane]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gi = lane >> 2, t = lane & 3;
  pdl_launch_dependents();

  const Work work = find_work<R, kBn, kThreads>(a, plan);
  if (tid < 2) a.notes[2 * blockIdx.x + tid].count = 0;
  if (work.begin == work.end) return;
  RowWalk &w = walks[0][warp], &lw = walks[1][warp];
  if (lane < 2) walks[lane][warp].begin(a, work);

  uint8_t* ring = smem + warp * S::ring_bytes;
  const uint32_t ring_s = smem_u32(ring);
  const int pieces = a.head_dim * T::size / 16;
  if (pieces < S::pieces)  // elements past head_dim are zeros throughout
    for (int i = lane; i < S::stages * S::stage_bytes / 16; i += 32) reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
  __syncwarp();

  // The loading side runs stages ahead, into the next pieces.  Lane l copies for
  // position (l & 15) of a step; its page is looked up a step before.
  int l_pos = 0, l_left = 0, l_lo = 0, l_hi = 0, l_seq = 0, l_head = 0, page = -1, slot = 0;
  auto open = [&] {
    l_left = lw.more() ? lw.tb - lw.ta : 0;
    l_pos = lw.ta * kBn + warp * kStep + (lane & 15);
    l_lo = lw.tile.lo, l_hi = lw.tile.hi, l_seq = lw.at.seq, l_head = lw.at.head;
  };
  auto look_up = [&] { page = l_left > 0 && l_pos >= l_lo && l_pos < l_hi ? page_of(a.q, l_seq, l_pos, slot) : -1; };
  auto issue = [&](int stage) {
    if (l_left > 0) {
      const uint32_t base = ring_s + stage * S::stage_bytes;
      const bool on = page >= 0;
      const int64_t off = on ? page * a.page_stride + slot * a.slot_stride + l_head * a.head_stride : -1;
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, on) & 0xFFFFu;
      if constexpr (T::e4m3) {
        const float* s = (lane < 16 ? a.k_scale : a.v_scale) + l_head * a.scale_head_stride;
        cp_async4(base + 2 * kStep * RB + lane * 4,
                  on ? s + page * a.scale_page_stride + slot * a.scale_slot_stride : static_cast<const void*>(a.query), on);
      }
      if (lane == 0) *reinterpret_cast<uint32_t*>(ring + stage * S::stage_bytes + 2 * kStep * RB + S::scale_bytes) = mask;
#pragma unroll
      for (int i = 0; i < kStep * S::pieces / 32; ++i) {
        const int n = lane + 32 * i, row = n / S::pieces, c = n % S::pieces;
        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row);
        if (c < pieces) {
          // nothing is read for a position that does not count, but the address is one of memory
          const void* ka = o < 0 ? a.query : static_cast<const uint8_t*>(a.k) + o + c * 16;
          const void* va = o < 0 ? a.query : static_cast<const uint8_t*>(a.v) + o + c * 16;
          cp_async16(base + key_at<RB>(row, c), ka, o >= 0);
          cp_async16(base + kStep * RB + (S::ev == 8 && T::e4m3 ? row * RB + c * 16 : value_at<RB>(row, c)), va, o >= 0);
        }
      }
      l_pos += kBn;
      if (--l_left == 0) {
        lw.next(a);
        open();
      }
      look_up();
    }
    cp_commit();
  };
  open();
  look_up();
#pragma unroll 1
  for (int i = 0; i < S::stages - 1; ++i) issue(i);

  // A piece's query, in the order in which the keys are read.  For e4m3 caches
  // it becomes float16, a row times a power of two (q_scale takes it back) that brings its
  // largest magnitude to 2^13: exact but for elements below 2^-29 of that.
  uint32_t qb[S::q_shared ? 1 : KS][NB][2];
  float q_scale[NB][2];  // of rows 8 n + 2t and + 1
  auto q_row = [&](int n) {  // row 8 n + gi, NULL if there is none
    const int row0 = w.at.tile * R, r = gi + 8 * n;
    if (r >= w.tile.rows) return static_cast<const uint16_t*>(nullptr);
    const int token = static_cast<int>(divide(row0 + r, a.by_group)), g = row0 + r - token * a.group;
    return static_cast<const uint16_t*>(a.query) + (w.seq.first + token) * a.ld_q +
           static_cast<int64_t>(w.at.head * a.group + g) * a.head_dim;
  };
  auto q_at = [&](const uint16_t* q, int s) {
    const int d = T::e4m3 ? 16 * (t + 4 * (s / 4)) + 4 * (s % 4) : 8 * (t + 4 * (s / 2)) + 4 * (s % 2);
    return q && d < a.head_dim ? *reinterpret_cast<const uint2*>(q + d) : make_uint2(0, 0);
  };
  auto largest = [](uint32_t top, uint32_t u) {  // magnitudes' bits order them
    u &= 0x7FFF7FFFu;
    return max(top, max(u << 16, u & 0xFFFF0000u));
  };
  auto scale_of = [&](uint32_t top, float& back) {
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const int e = min(max(static_cast<int>(top >> 23) - 127, -100), 127) - 13;
    back = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  };
  auto scaled = [](uint32_t u, float f) { return pack2(bf16lo(u) * f, bf16hi(u) * f, MOE_F16); };
  auto spread = [&](int n, float back) {  // from the lanes that read a row to those that have it in z
    q_scale[n][0] = __shfl_sync(0xFFFFFFFFu, back, (2 * t) << 2), q_scale[n][1] = __shfl_sync(0xFFFFFFFFu, back, (2 * t + 1) << 2);
  };
  auto load_q = [&] {
    if constexpr (!S::q_shared) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const uint16_t* q = q_row(n);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint2 u = q_at(q, s);
          qb[s][n][0] = u.x, qb[s][n][1] = u.y;
        }
      }
    }
  };
  auto finish_q = [&] {
    const bool narrow = T::e4m3 && a.type == MOE_BF16;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float f = 1.0f, back = 1.0f;
      if constexpr (!S::q_shared) {
        if (narrow) {
          uint32_t top = 0;
#pragma unroll
          for (int s = 0; s < KS; ++s) top = largest(largest(top, qb[s][n][0]), qb[s][n][1]);
          f = scale_of(top, back);
#pragma unroll
          for (int s = 0; s < KS; ++s) qb[s][n][0] = scaled(qb[s][n][0], f), qb[s][n][1] = scaled(qb[s][n][1], f);
        }
      } else {  // registers are short: a warp brings a quarter of the fragments
        const uint16_t* q = q_row(n);
        if (narrow) {
          uint32_t top = 0;
#pragma unroll 4
          for (int s = 0; s < KS; ++s) {
            const uint2 u = q_at(q, s);
            top = largest(largest(top, u.x), u.y);
          }
          f = scale_of(top, back);
        }
#pragma unroll 1
        for (int s = warp; s < KS; s += kWarps) {
          uint2 u = q_at(q, s);
          if (narrow) u = make_uint2(scaled(u.x, f), scaled(u.y, f));
          q_frag[(s * NB + n) * 32 + lane] = u;
        }
      }
      if (T::e4m3) spread(n, back);
    }
  };
  if (w.more()) {  // for all warps alike: a CTA's places may be a unit's beginning alone
    load_q();
    finish_q();
  }
  if (S::q_shared) __syncthreads();

  int stage = 0;
  while (w.more()) {
    const int row0 = w.at.tile * R, rows = w.tile.rows, ta = w.ta, steps = w.tb - w.ta;
    // what the lane's rows 8 n + 2t and + 1 see
    int lo[NB][2], hi[NB][2];
    int tight_lo, tight_hi;  // what all of the tile's rows see
    {
      const int base = w.seq.len - w.seq.n;
      const int p0 = base + static_cast<int>(divide(row0, a.by_group));
      const int p1 = base + static_cast<int>(divide(row0 + rows - 1, a.by_group));
      tight_hi = sees_to(a, w.seq.len, p0), tight_lo = sees_from(a, p1);
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = 8 * n + 2 * t + c;
          const int p = base + static_cast<int>(divide(row0 + min(r, rows - 1), a.by_group));
          lo[n][c] = sees_from(a, p);
          hi[n][c] = r < rows ? sees_to(a, w.seq.len, p) : 0;
        }
    }
    float o[MB][NB][4], m[NB][2], l[NB][2];
    float unit[NB][2];  // e4m3: o counts weights in units of 2^unit, a whole number in [-126, 126]
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      m[n][0] = m[n][1] = kLowest, l[n][0] = l[n][1] = 0.0f;
      unit[n][0] = unit[n][1] = -126.0f;
#pragma unroll
      for (int j = 0; j < MB; ++j) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.0f;
    }

#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      cp_wait<S::stages - 2>();
      __syncwarp();
      issue(stage == 0 ? S::stages - 1 : stage - 1);
      const uint8_t* ks = ring + stage * S::stage_bytes;
      const uint8_t* vs = ks + kStep * RB;
      const uint32_t mask = *reinterpret_cast<const uint32_t*>(ks + 2 * kStep * RB + S::scale_bytes);
      const float* sc = reinterpret_cast<const float*>(ks + 2 * kStep * RB);
      if (++stage == S::stages) stage = 0;
      if (mask == 0) continue;

      // z: positions gi (values 0 and 1) and gi + 8, rows 8 n + 2t and + 1
      float z[NB][4];
#pragma unroll
      for (int n = 0; n < NB; ++n) z[n][0] = z[n][1] = z[n][2] = z[n][3] = 0.0f;
      auto product = [&](int s, const uint32_t (&k)[4]) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if constexpr (S::q_shared) {
            const uint2 u = q_frag[(s * NB + n) * 32 + lane];
            mma16816<T::f16>(z[n], k, u.x, u.y);
          } else {
            mma16816<T::f16>(z[n], k, qb[s][n][0], qb[s][n][1]);
          }
        }
      };
#pragma unroll
      for (int i = 0; i < S::pieces / 4; ++i) {
        const uint4 u0 = lds128(ks + key_at<RB>(gi, t + 4 * i)), u1 = lds128(ks + key_at<RB>(8 + gi, t + 4 * i));
        const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
        if constexpr (T::e4m3) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            product(4 * i + j, {two_codes(w0[j], 0), two_codes(w1[j], 0), two_codes(w0[j], 1), two_codes(w1[j], 1)});
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) product(2 * i + j, {w0[2 * j], w1[2 * j], w0[2 * j + 1], w1[2 * j + 1]});
        }
      }
      float vf[2];  // e4m3: the values' scales at positions gi and gi + 8
      if constexpr (T::e4m3) {
        const float k0 = sc[gi], k1 = sc[gi + 8];
        vf[0] = sc[kStep + gi], vf[1] = sc[kStep + gi + 8];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          // both factors at once: one of them alone may send z out of range; their product does only
          // where z is out of range too, or 0
          z[n][0] *= finite(q_scale[n][0] * k0), z[n][1] *= finite(q_scale[n][1] * k0);
          z[n][2] *= finite(q_scale[n][0] * k1), z[n][3] *= finite(q_scale[n][1] * k1);
        }
      }
      const int first = (ta + step) * kBn + warp * kStep;
      const bool edge = first < tight_lo || first + kStep > tight_hi || mask != 0xFFFFu;
      uint32_t seen = 0;  // bit 4 n + c: value c of block n is seen
      if (edge) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int k = gi + 8 * (c >> 1), pos = first + k;
            const bool see = (mask >> k & 1) && pos >= lo[n][c & 1] && pos < hi[n][c & 1];
            if (see) seen |= 1u << (4 * n + c);
            else z[n][c] = -INFINITY;
          }
      }
      // the running maximum, and what l and o shrink by when it grows
      auto largest_z = [&](int n, int c) {
        float x = fmaxf(z[n][c], z[n][2 + c]);
#pragma unroll
        for (int i = 4; i < 32; i *= 2) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, i));
        return x;
      };
      auto shrink_o = [&](int n, float f0, float f1) {
#pragma unroll
        for (int j = 0; j < MB; ++j) o[j][n][0] *= f0, o[j][n][1] *= f1, o[j][n][2] *= f0, o[j][n][3] *= f1;
      };
      bool moved = false;
      if constexpr (!T::e4m3) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) moved |= fmaxf(z[n][c], z[n][2 + c]) > m[n][c];
        if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            float shrink[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float x = largest_z(n, c);
              shrink[c] = 1.0f;
              if (x > m[n][c]) {
                shrink[c] = exp2_approx((m[n][c] - x) * a.scale_log2);
                m[n][c] = x;
              }
              l[n][c] *= shrink[c];
            }
            shrink_o(n, shrink[0], shrink[1]);
          }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            z[n][c] = exp2_approx(fmaf(z[n][c] - m[n][c & 1], a.scale_log2, exp_lift<K>()));
            l[n][c & 1] += z[n][c];
          }
      } else {
        // exponentials and weights as powers of two
        const float v_log2[2] = {log2_approx(vf[0]), log2_approx(vf[1])};
        float d[NB][4], w[NB][4];
        auto relate = [&] {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              d[n][c] = (z[n][c] - m[n][c & 1]) * a.scale_log2;
              w[n][c] = d[n][c] + (v_log2[c >> 1] - unit[n][c & 1]);
            }
        };
        relate();
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) moved |= d[n][c] > 0.0f || w[n][c] > static_cast<float>(kUnitMost);
        if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            float shrink[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float x = largest_z(n, c);
              float grown = 0.0f;  // m's growth in powers of two, of which the unit follows whole ones
              if (x > m[n][c]) {
                grown = fminf((x - m[n][c]) * a.scale_log2, 4096.0f);
                m[n][c] = x;
              }
              l[n][c] *= exp2_approx(-grown);
              float top = fmaxf((z[n][c] - m[n][c]) * a.scale_log2 + v_log2[0], (z[n][2 + c] - m[n][c]) * a.scale_log2 + v_log2[1]);
#pragma unroll
              for (int i = 4; i < 32; i *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
              const float was = unit[n][c] - floorf(grown), to = top > was + kUnitMost ? ceilf(top) - kUnitTop : was;
              unit[n][c] = fminf(fmaxf(to, -126.0f), 126.0f);
              shrink[c] = exp2_approx(floorf(grown) - grown) * exp2_approx(was - unit[n][c]);
            }
            shrink_o(n, shrink[0], shrink[1]);
          }
          relate();
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            l[n][c & 1] += exp2_approx(d[n][c]);
            z[n][c] = exp2_approx(w[n][c]);
          }
      }
      uint32_t pb[NB][2];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        // position by position for the next product's operand
        pb[n][0] = transposed(pack2(z[n][0], z[n][1], half_type));
        pb[n][1] = transposed(pack2(z[n][2], z[n][3], half_type));
      }

      bool odd = false;
      if (edge) {  // a value that some row must not see may be anything
        if constexpr (T::e4m3) odd = !(vf[0] < INFINITY) || !(vf[1] < INFINITY);
#pragma unroll
        for (int h = 0; h < S::vgroups; ++h) {
          Values<DP, K, R> v;
          v.load(vs, t, gi, h);
#pragma unroll
          for (int j = 0; j < EV; ++j) {
            uint32_t b0, b1;
            v.pair(j, b0, b1);
            odd |= odd_value<T::f16>(b0) || odd_value<T::f16>(b1);
          }
        }
        odd = __any_sync(0xFFFFFFFFu, odd);
      }
      if (!odd) {
#pragma unroll
        for (int h = 0; h < S::vgroups; ++h) {
          Values<DP, K, R> v;
          v.load(vs, t, gi, h);
#pragma unroll
          for (int j = 0; j < EV; j += 2) {
            uint32_t va[4];
            v.pair(j, va[0], va[2]);
            v.pair(j + 1, va[1], va[3]);
#pragma unroll
            for (int n = 0; n < NB; ++n) mma16816<T::f16>(o[(h * EV + j) / 2][n], va, pb[n][0], pb[n][1]);
          }
        }
      } else {
        // One position at a time, into the rows that see it: its values are in the
        // lanes of its pair, its exponentials in the lanes of its place in z.
#pragma unroll 1
        for (int k = 0; k < kStep; ++k) {
          const int from = ((k & 7) << 2) | t;
          const uint32_t who = __shfl_sync(0xFFFFFFFFu, seen, from) >> (2 * (k >> 3));
          float p[NB][2];
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) p[n][c] = __shfl_sync(0xFFFFFFFFu, k < 8 ? z[n][c] : z[n][2 + c], from);
#pragma unroll
          for (int h = 0; h < S::vgroups; ++h) {
            Values<DP, K, R> v;
            v.load(vs, t, gi, h);
#pragma unroll
            for (int j = 0; j < EV; ++j) {
              uint32_t b0, b1;
              v.pair(j, b0, b1);
              const uint32_t b = k < 8 ? b0 : b1, bits = k & 1 ? b >> 16 : b & 0xFFFFu;
              const float val = half_bits_to_f32(__shfl_sync(0xFFFFFFFFu, bits, (gi << 2) | ((k & 7) >> 1)), half_type);
#pragma unroll
              for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  if (who >> (4 * n + c) & 1) o[(h * EV + j) / 2][n][(j & 1) * 2 + c] += p[n][c] * val;
            }
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 4; i < 32; i *= 2) l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], i);
        if (gi == 0) join_ml[warp][8 * n + 2 * t + c][0] = m[n][c], join_ml[warp][8 * n + 2 * t + c][1] = l[n][c];
      }

    // The four warps' parts, a few rows at a time, while the next piece's query is
    // on its way.
    const bool whole = w.whole();
    const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (ta == w.tile.t0 ? 1 : 0);
    const int seq_first = w.seq.first, kv_head = w.at.head, d4 = a.head_dim / 4;
    if (!whole && tid == 0) w.note(a, work);
    w.next(a);
    const bool more = w.more();
    if (more) load_q();
    // of e4m3 caches a row's weights' unit, 1 otherwise
    auto unit_of = [&](int n, int c) { return T::e4m3 ? __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(unit[n][c])) << 23) : 1.0f; };
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kJoinRows) {
      // a lane has, of rows 8 n + 2t and + 1, the elements EV (gi + 8 h) + j
      if (((2 * t ^ r0) & 4) == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float* row = join_o + (warp * kJoinRows + ((2 * t + c) & 3)) * DP;
          const float u = NB > 1 && r0 >= 8 ? unit_of(NB - 1, c) : unit_of(0, c);
#pragma unroll
          for (int h = 0; h < S::vgroups; ++h)
#pragma unroll
            for (int j = 0; j < EV; j += 4) {
              const int b = (h * EV + j) / 2;
              float4 v = make_float4(o[b][0][c], o[b][0][2 + c], o[b + 1][0][c], o[b + 1][0][2 + c]);
              if (NB > 1 && r0 >= 8) v = make_float4(o[b][NB - 1][c], o[b][NB - 1][2 + c], o[b + 1][NB - 1][c], o[b + 1][NB - 1][2 + c]);
              *reinterpret_cast<float4*>(row + EV * (gi + 8 * h) + j) = make_float4(v.x * u, v.y * u, v.z * u, v.w * u);
            }
        }
      }
      __syncthreads();
      if (r0 + kJoinRows >= rows && more) finish_q();  // all warps are past the old one
#pragma unroll 1
      for (int i = tid; i < min(kJoinRows, rows - r0) * d4; i += kThreads) {
        const int rr = i / d4, d = (i - rr * d4) * 4, r = r0 + rr;
        float mw[kWarps], top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) mw[v] = join_ml[v][r][0], top = fmaxf(top, mw[v]);
        const float ref = top == -INFINITY ? 0.0f : top;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          const float f = exp2_approx((mw[v] - ref) * a.scale_log2);
          const float4 x = *reinterpret_cast<const float4*>(join_o + (v * kJoinRows + rr) * DP + d);
          sum += f * join_ml[v][r][1];
          acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
        }
        if (whole) {
          const int token = static_cast<int>(divide(row0 + r, a.by_group)), g = row0 + r - token * a.group;
          const int64_t row = seq_first + token;
          const int head = kv_head * a.group + g;
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          uint2 u;
          u.x = pack2(acc.x * inv, acc.y * inv, a.type), u.y = pack2(acc.z * inv, acc.w * inv, a.type);
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * a.ld_out + static_cast<int64_t>(head) * a.head_dim + d) = u;
          if (d == 0 && a.lse)
            a.lse[row * a.kv_heads * a.group + head] =
                sum == 0.0f ? -INFINITY : fmaf(top, a.scale, (log2f(sum) - exp_lift<K>()) * kLn2);
        } else {
          *reinterpret_cast<float4*>(a.part_o + (part * R + r) * a.head_dim + d) = acc;
          if (d == 0) a.part_ml[(part * R + r) * 2] = top, a.part_ml[(part * R + r) * 2 + 1] = sum;
        }
      }
      __syncthreads();  // the buffers are free again, the next query is there
    }
  }
  cp_wait<0>();
}

// ---- the join ---------------------------------------------------------------------

constexpr int kJoinThreads = 256;

// o, l and m of a group of four outputs.
struct Part {
  float m, l;
  float4 o;
  __device__ __forceinline__ void add(float m2, float l2, float4 o2, float scale_log2) {
    const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.0f : top;
    const float f = exp2_approx((m - ref) * scale_log2), f2 = exp2_approx((m2 - ref) * scale_log2);
    m = top, l = l * f + l2 * f2;
    o = make_float4(o.x * f + o2.x * f2, o.y * f + o2.y * f2, o.z * f + o2.z * f2, o.w * f + o2.w * f2);
  }
};

// A group's parts are shared by `lanes` threads of a warp, a power of two, as far
// as a block's share of the groups leaves threads for it (32 rows' parts of
// 128 CTAs: 32 lanes; 256 rows' parts of 5: one); neighbouring groups lie in
// neighbouring threads.
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttnArgs a, int tile_rows, int type, float lift) {
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d4 = a.head_dim / 4;
  for (int which = 0; which < 2; ++which) {
    const Note n = a.notes[2 * blockIdx.x + which];
    if (n.count == 0) continue;
    const int all = n.rows * d4, shares = n.count * gridDim.y, each = (all + shares - 1) / shares;
    int lanes = 1;
    while (lanes < 32 && lanes < n.count && 2 * lanes * each <= kJoinThreads) lanes *= 2;
    const int per_warp = 32 / lanes, item = lane & (per_warp - 1), first = lane / per_warp;
    const int from = ((blockIdx.x - n.c0) * gridDim.y + blockIdx.y) * each, to = min(all, from + each);
    for (int i0 = from + warp * per_warp; i0 < to; i0 += per_warp * (kJoinThreads / 32)) {
      const int i = i0 + item;
      const bool on = i < to;
      const int r = on ? i / d4 : 0, d = on ? (i - r * d4) * 4 : 0;
      Part p = {-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
      constexpr int kBatch = 4;  // parts read at once
      for (int c0 = first; c0 < n.count; c0 += lanes * kBatch) {
        float2 ml[kBatch];
        float4 o[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int c = c0 + b * lanes;
          ml[b] = make_float2(-INFINITY, 0.0f), o[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (on && c < n.count) {
            const int64_t at = (2 * static_cast<int64_t>(n.c0 + c) + (c == 0 ? 1 : 0)) * tile_rows + r;
            ml[b] = __ldg(reinterpret_cast<const float2*>(a.part_ml) + at);
            o[b] = __ldg(reinterpret_cast<const float4*>(a.part_o + at * a.head_dim + d));
          }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) p.add(ml[b].x, ml[b].y, o[b], a.scale_log2);
      }
      for (int s = per_warp; s < 32; s <<= 1) {
        const float m2 = __shfl_xor_sync(0xFFFFFFFFu, p.m, s), l2 = __shfl_xor_sync(0xFFFFFFFFu, p.l, s);
        const float4 o2 = make_float4(__shfl_xor_sync(0xFFFFFFFFu, p.o.x, s), __shfl_xor_sync(0xFFFFFFFFu, p.o.y, s),
                                      __shfl_xor_sync(0xFFFFFFFFu, p.o.z, s), __shfl_xor_sync(0xFFFFFFFFu, p.o.w, s));
        p.add(m2, l2, o2, a.scale_log2);
      }
      if (on && first == 0) {
        const int token = static_cast<int>(divide(n.row + r, a.by_group)), g = n.row + r - token * a.group;
        const int64_t row = n.first + token;
        const int head = n.head * a.group + g;
        const float inv = p.l == 0.0f ? 0.0f : 1.0f / p.l;
        uint2 u;
        u.x = pack2(p.o.x * inv, p.o.y * inv, type), u.y = pack2(p.o.z * inv, p.o.w * inv, type);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * a.ld_out + static_cast<int64_t>(head) * a.head_dim + d) = u;
        if (d == 0 && a.lse)
          a.lse[row * a.kv_heads * a.group + head] = p.l == 0.0f ? -INFINITY : fmaf(p.m, a.scale, (log2f(p.l) - lift) * kLn2);
      }
    }
  }
}

// ---- host --------------------------------------------------------------------------

// Rows of a sequence times query heads of a key head up to which tiles of 8 or 16
// rows are taken; more of them read the cache several times over, the tiles of 256 of
// attention_tc.cu once.  16 sequences of 8192 positions, 8 key heads of 128, in a graph:
//   rows            8      16     24     32     48
//   bf16, 8         94.7   180    263    343    460 us
//   bf16, 16        94.9   97.1   182    183    265
//   bf16, 256       106    106    107    107    109
//   e4m3, 8         65.5   118    170    216    315
//   e4m3, 16        82.0   88.2   152    156    224
//   e4m3, 256       135    135    137    137    138
// At 24 and 32 rows of e4m3 caches heads of 64 gain and lose with tiles of 16: 102 and 106
// us against 107 there, 14.4 and 14.8 against 17.4 and 18.1 over one sequence of 4000, but
// 118 and 122 against 109 over 64 of 2048, 40 and 42 against 37 over 64 of 300.  Heads of 256
// lose (212 and 218 against 146).
constexpr int kFewRows = 16;

// CTAs of the widest grid that a workspace serves, on an SM.
constexpr int kMaxCtas = 3;

struct Parts {
  size_t notes, ml, o, bytes;
};

Parts parts_of(int grid, int tile_rows, int head_dim) {
  Parts p;
  p.notes = kCtlBytes;
  p.ml = (p.notes + sizeof(Note) * 2 * grid + 255) / 256 * 256;
  p.o = (p.ml + sizeof(float) * 4 * grid * tile_rows + 255) / 256 * 256;
  p.bytes = p.o + sizeof(float) * 2 * static_cast<size_t>(grid) * tile_rows * head_dim;
  return p;
}

template <int DP, int K, int R>
cudaError_t launch_rows(const AttnArgs& a, int num_sms, int* grid, cudaStream_t st) {
  using S = Shape<DP, K, R>;
  static_assert(S::ctas <= kMaxCtas, "workspace");
  auto kernel = attention_rows_kernel<DP, K, R>;
  static std::atomic<uint64_t> allowed{0};  // devices
  const cudaError_t e = allow_smem(allowed, kernel, S::smem);
  if (e) return e;
  *grid = num_sms * S::ctas;
  kernel<<<*grid, kThreads, S::smem, st>>>(a);
  return cudaGetLastError();
}

template <int DP, int R>
cudaError_t launch_rows(const AttnArgs& a, Kind k, int num_sms, int* grid, cudaStream_t st) {
  switch (k) {
    case kBf16: return launch_rows<DP, kBf16, R>(a, num_sms, grid, st);
    case kF16: return launch_rows<DP, kF16, R>(a, num_sms, grid, st);
    default: return launch_rows<DP, kE4m3F16, R>(a, num_sms, grid, st);  // for both types of q
  }
}

template <int R>
cudaError_t launch_rows(const AttnArgs& a, Kind k, int num_sms, int* grid, cudaStream_t st) {
  return a.head_dim <= 64    ? launch_rows<64, R>(a, k, num_sms, grid, st)
         : a.head_dim <= 128 ? launch_rows<128, R>(a, k, num_sms, grid, st)
                             : launch_rows<256, R>(a, k, num_sms, grid, st);
}

bool heads_ok(int32_t q_heads, int32_t kv_heads) {
  return kv_heads >= 1 && kv_heads <= 1024 && q_heads >= 1 && q_heads <= 4096 && q_heads % kv_heads == 0 &&
         q_heads / kv_heads <= 128;
}

// Whether 32 bits count the places of a line of such tiles, whatever the device values are
// (attention.cuh): all rows in as many row tiles as sequences can make of them, each as
// long as the page table.
bool counts(const moe_sequences& s, int32_t cap, int32_t kv_heads, int group, int tile_rows, int tile_keys) {
  const int64_t units = (static_cast<int64_t>(s.rows) * group / tile_rows + s.n_seqs) * kv_heads;
  return units * (cap / tile_keys + 1 + kUnitCost) <= 0x7FFFFFFF;
}

// The current device's SMs, asked for once a device.
cudaError_t sm_count(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (!e && dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return e;
  if (!e) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (!e && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

size_t workspace_bytes_for(int sms, int head_dim) {
  const size_t few = parts_of(sms * kMaxCtas, kRows, head_dim).bytes, many = parts_of(sms, tiles_rows(head_dim), head_dim).bytes;
  return few > many ? few : many;
}

}  // namespace

cudaError_t launch_join(const AttnArgs& a, int grid, int tile_rows, bool f16, float lift, cudaStream_t st) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid, tile_rows > kRows ? 16 : 1), c.blockDim = dim3(kJoinThreads), c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at, c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, attention_join_kernel, a, tile_rows, static_cast<int>(f16 ? MOE_F16 : MOE_BF16), lift);
}

}  // namespace moe

extern "C" size_t moe_attention_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  using namespace moe;
  int sms = 0;
  if (!heads_ok(q_heads, kv_heads) || head_dim < 16 || head_dim > 256 || head_dim % 16 || sm_count(&sms)) return 0;
  return workspace_bytes_for(sms, head_dim);
}

extern "C" int moe_attention_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
  using namespace moe;
  if (!workspace || workspace_bytes < kCtlBytes)
    return reportf(MOE_ERR_ARG, "moe_attention_workspace_init: workspace is NULL or smaller than %zu bytes", kCtlBytes);
  if (reinterpret_cast<uintptr_t>(workspace) % 256)
    return reportf(MOE_ERR_ALIGN, "moe_attention_workspace_init: workspace is not 256-byte aligned");
  const cudaError_t e = cudaMemsetAsync(workspace, 0, kCtlBytes, static_cast<cudaStream_t>(stream));
  if (e) return reportf(MOE_ERR_CUDA, "moe_attention_workspace_init: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  return MOE_OK;
}

extern "C" int moe_attention(const moe_attention_args* args, const moe_kv_cache* cache, const moe_sequences* seqs,
                             void* workspace, size_t workspace_bytes, void* stream) {
  using namespace moe;
  if (!args) return reportf(MOE_ERR_ARG, "moe_attention: args is NULL");
  const moe_attention_args& g = *args;
  AttnArgs a = {};
  const int rc = check_cache("moe_attention", cache, seqs, &a.q);
  if (rc) return rc;
  const moe_kv_cache& c = *cache;
  if (g.q_type != MOE_BF16 && g.q_type != MOE_F16)
    return reportf(MOE_ERR_ARG, "moe_attention: q has an unknown type %d", g.q_type);
  if (c.type != MOE_E4M3 && c.type != g.q_type)
    return reportf(MOE_ERR_UNSUPPORTED, "moe_attention: q is of type %d, the cache of %d", g.q_type, c.type);
  if (!heads_ok(g.q_heads, c.kv_heads))
    return reportf(MOE_ERR_ARG, "moe_attention: q_heads=%d must be at most 4096, a multiple of kv_heads=%d and at most 128 times it",
                   g.q_heads, c.kv_heads);
  if ((g.causal != 0 && g.causal != 1) || g.window < 0)
    return reportf(MOE_ERR_ARG, "moe_attention: causal=%d must be 0 or 1, window=%d not negative", g.causal, g.window);
  if (!(g.scale > 0.0f) || g.scale > 3.0e38f / 1.5f)
    return reportf(MOE_ERR_ARG, "moe_attention: scale must be positive and below 2^127");
  if (seqs->rows == 0 || seqs->n_seqs == 0) return MOE_OK;
  const int group = g.q_heads / c.kv_heads;
  if (static_cast<int64_t>(seqs->rows) * group > (1 << 30))
    return reportf(MOE_ERR_ARG, "moe_attention: %d rows of %d query heads a key head are more than 2^30", seqs->rows, group);
  const int64_t most = static_cast<int64_t>(seqs->max_rows) * group;
  const int few_rows = most > 8 ? 16 : 8;
  const bool many = most > kFewRows || !counts(*seqs, a.q.cap, c.kv_heads, group, few_rows, kBn);
  const int tile_rows = many ? tiles_rows(c.head_dim) : few_rows;
  if (many && !counts(*seqs, a.q.cap, c.kv_heads, group, tile_rows, tiles_keys(c.head_dim)))
    return reportf(MOE_ERR_UNSUPPORTED,
                   "moe_attention: %d rows of %d heads in %d sequences of up to %d positions are 2^31 places of work or more", seqs->rows,
                   g.q_heads, seqs->n_seqs, a.q.cap);
  if (!g.q || !g.out || !workspace) return reportf(MOE_ERR_ARG, "moe_attention: q, out or workspace is NULL");
  const int64_t width = static_cast<int64_t>(g.q_heads) * c.head_dim;
  if (g.ld_q < width || g.ld_out < width || g.ld_q % 8 || g.ld_out % 8)
    return reportf(MOE_ERR_ARG, "moe_attention: ld_q=%lld and ld_out=%lld must be multiples of 8, at least %lld",
                   static_cast<long long>(g.ld_q), static_cast<long long>(g.ld_out), static_cast<long long>(width));
  if ((reinterpret_cast<uintptr_t>(g.q) | reinterpret_cast<uintptr_t>(g.out)) % 16 || reinterpret_cast<uintptr_t>(g.lse) % 4 ||
      reinterpret_cast<uintptr_t>(workspace) % 256)
    return reportf(MOE_ERR_ALIGN, "moe_attention: q or out is not 16-byte aligned, lse not 4, or workspace not 256");
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e) return reportf(MOE_ERR_CUDA, "moe_attention: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  const size_t need = workspace_bytes_for(sms, c.head_dim);
  if (workspace_bytes < need)
    return reportf(MOE_ERR_ARG, "moe_attention: these heads need %zu bytes of workspace, got %zu", need, workspace_bytes);

  a.query = g.q, a.out = g.out, a.lse = g.lse, a.ld_q = g.ld_q, a.ld_out = g.ld_out;
  const int size = c.type == MOE_E4M3 ? 1 : 2;
  a.k = c.k, a.v = c.v, a.k_scale = c.k_scale, a.v_scale = c.v_scale;
  a.page_stride = c.page_stride * size, a.slot_stride = c.slot_stride * size, a.head_stride = c.head_stride * size;
  a.scale_page_stride = c.scale_page_stride, a.scale_slot_stride = c.scale_slot_stride, a.scale_head_stride = c.scale_head_stride;
  a.head_dim = c.head_dim, a.kv_heads = c.kv_heads, a.group = group, a.causal = g.causal, a.window = g.window, a.type = g.q_type;
  a.scale = g.scale, a.scale_log2 = g.scale * 1.4426950408889634f;
  a.by_group = divisor(static_cast<uint32_t>(group));
  const Kind kind = c.type == MOE_BF16 ? kBf16 : c.type == MOE_F16 ? kF16 : g.q_type == MOE_BF16 ? kE4m3Bf16 : kE4m3F16;
  const bool f16 = g.q_type == MOE_F16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  const Parts p = parts_of(many ? sms : sms * kMaxCtas, tile_rows, c.head_dim);
  a.ctl = reinterpret_cast<unsigned*>(base);
  a.notes = reinterpret_cast<Note*>(base + p.notes);
  a.part_ml = reinterpret_cast<float*>(base + p.ml), a.part_o = reinterpret_cast<float*>(base + p.o);
  int grid = sms;
  e = many              ? launch_tiles(a, kind, sms, st)
      : tile_rows == 16 ? launch_rows<16>(a, kind, sms, &grid, st)
                        : launch_rows<8>(a, kind, sms, &grid, st);
  if (!e)
    e = launch_join(a, grid, tile_rows, f16, many ? tiles_lift(f16) : kind == kF16 ? exp_lift<kF16>() : 0.0f, st);
  if (e) return reportf(MOE_ERR_CUDA, "moe_attention: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  return MOE_OK;
}

extern "C" int moe_attention_check(void* workspace, void* stream) {
  using namespace moe;
  if (!workspace) return reportf(MOE_ERR_ARG, "moe_attention_check: workspace is NULL");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned bits = 0;
  cudaError_t e = cudaMemcpyAsync(&bits, workspace, sizeof bits, cudaMemcpyDeviceToHost, st);
  if (!e) e = cudaStreamSynchronize(st);
  if (!e && bits) {
    e = cudaMemsetAsync(workspace, 0, kCtlBytes, st);
    if (!e) e = cudaStreamSynchronize(st);
  }
  if (e) return reportf(MOE_ERR_CUDA, "moe_attention_check: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  if (bits & kErrTimeout) return reportf(MOE_ERR_TIMEOUT, "moe_attention_check: a bounded device-side wait ran out (bits 0x%x)", bits);
  if (bits) return reportf(MOE_ERR_ARG, "moe_attention_check: the starts of a call fell (bits 0x%x)", bits);
  return MOE_OK;
}
