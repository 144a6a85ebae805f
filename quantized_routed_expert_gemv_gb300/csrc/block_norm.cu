// block_norm.cu -- the block boundary (moe_block_norm): post-norm, gate,
// scaled residual and the next block's pre-norm in one pass over the rows.
//
// Mathematics: r = y * rsqrt(mean(y^2) + eps) * w_post, h' = s h + g r,
// x = h' * rsqrt(mean(h'^2) + eps) * w_pre.  The two means need the whole
// row, so a row's values stay in registers between them: y and h are read
// once, h' and x written once, nothing in between goes to memory.
//
// Bound: memory traffic for many rows (about 11 operations per value against
// 8 to 12 bytes), the latency of one load and two reductions for few.  Two
// kernels: block_norm_kernel takes one row per block (or per warp);
// block_norm_stream_kernel keeps one block on each SM whose teams of threads
// load their next rows while they work on one, with the weights at hand.
// Measured: 8192 rows of 7168, fp32 y and bf16 h, h' and x, 92 to 94 us (6.2 to
// 6.4 TB/s, 92 to 94% of the measured copy rate); one such row 3.5 us a call in a
// graph, 128 of them 4.0.
// That is the streaming kernel's form, both norms and all of y, h, h' and x with a
// gate of every channel or none.  Many rows of another form take a row a block,
// whose loads, sums and stores follow one another (bytes at the copy rate in
// brackets): 8192 x 7168 without the post-norm, bf16 y, 95 us (69), without y 86
// (52); 4096 x 4096, bf16 y, with a gate of every token 42.7 (19.8), of every
// element 46.1 (24.7), where the streaming form takes 26.6; rows of 16384 values,
// 4096 of them, 181 (99).  8192 rows of 2000 bf16 values take 24.3 us (19.3), rows
// of 1999 in 2000, a width that 8 does not divide, 61.8, of 2000 in 2001, off 16
// bytes, 68.9.
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "elem.cuh"

namespace moe {
int reportf(int code, const char* fmt, ...);

namespace {

constexpr int kMaxHidden = 16384;
// Values per SM from which streaming pays: bf16 rows of 512, 2432 of them 4.8
// us against 4.0 a row a block, 4864 5.9 against 6.9; of 2048, 608 4.7 against
// 4.0, 2432 8.2 against 12.0; fp32 y, rows of 7168, 304 6.6 against 5.5, 608
// 8.8 against 9.7.
constexpr int kStreamValues = 16384;
constexpr int kStreamThreads = 896;  // of a streaming block: 72 registers each
constexpr int kStreamHidden = 8192;  // widest row of a team (512 threads of 16 values)
constexpr int kMaxTeams = 14;        // one named barrier each

// Sum over the row's threads, the same value in all of them.  A block of 32
// threads per row needs no barrier.  `red` has one slot per warp.
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (blockDim.x == 32) return v;
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  float s = static_cast<int>(threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

// Operands whose rows start on 16-byte boundaries, by bit.
enum : int { kY = 1, kH = 2, kGate = 4, kWPost = 8, kWPre = 16, kHOut = 32, kXOut = 64, kAll = 127 };

// Eight values as loaded, converted only when they are used, so that loads
// are issued together whatever their types.  Of an operand whose rows do not
// start on 16 bytes a warp loads its 256 values one by one, neighbouring
// lanes neighbouring values (w[i] = value 32 i + lane), and exchanges them
// through shared memory afterwards (settle).
struct Raw {
  uint32_t w[8];  // 16-bit types: two values a word once settled

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0;
  }
  // Elements [j, j + 8) of the row that starts at element `row`, zeros past H.
  __device__ __forceinline__ void load(const void* p, bool wide, bool aligned, int64_t row, int j, int H) {
    if (aligned) {
      if (j + 8 <= H) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + (row + j) * (wide ? 4 : 2));
        const uint4 a = q[0];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        if (wide) {
          const uint4 b = q[1];
          w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        }
      } else {
        zero();
        if (wide) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (j + i < H) w[i] = static_cast<const uint32_t*>(p)[row + j + i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (j + i < H) w[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[row + j + i]) << (16 * (i & 1));
        }
      }
    } else {
      const int k = j - 7 * static_cast<int>(threadIdx.x & 31);  // the warp's first value + lane
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] = 0;
        if (k + 32 * i < H)
          w[i] = wide ? static_cast<const uint32_t*>(p)[row + k + 32 * i] : static_cast<const uint16_t*>(p)[row + k + 32 * i];
      }
    }
  }
  __device__ __forceinline__ void settle(uint32_t* buf, bool wide, bool aligned) {
    if (aligned) return;
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) buf[32 * i + lane] = w[i];
    __syncwarp();
    const uint4 a = reinterpret_cast<const uint4*>(buf)[2 * lane], b = reinterpret_cast<const uint4*>(buf)[2 * lane + 1];
    if (wide) {
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      w[0] = a.x | a.y << 16, w[1] = a.z | a.w << 16, w[2] = b.x | b.y << 16, w[3] = b.z | b.w << 16;
    }
  }
  __device__ __forceinline__ void get(int type, float (&v)[8]) const {
    if (type == MOE_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
      unpack8(make_uint4(w[0], w[1], w[2], w[3]), type, v);
    }
  }
};

__device__ __forceinline__ void store_chunk(void* p, int type, bool aligned, int64_t row, int j, int H, const float (&v)[8],
                                            uint32_t* buf) {
  if (aligned) {
    if (j + 8 <= H) {
      store8(p, type, row + j, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i < H) store_elem(p, type, row + j + i, v[i]);
    }
  } else {
    const int lane = threadIdx.x & 31, k = j - 7 * lane;
    __syncwarp();
    float4* to = reinterpret_cast<float4*>(buf) + 2 * lane;
    to[0] = make_float4(v[0], v[1], v[2], v[3]);
    to[1] = make_float4(v[4], v[5], v[6], v[7]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + 32 * i < H) store_elem(p, type, row + k + 32 * i, __uint_as_float(buf[32 * i + lane]));
  }
}

__device__ __forceinline__ void scale_by(float (&v)[8], float s, float add, const Raw& raw, int type) {
  float w[8];
  raw.get(type, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= s * (add + w[i]);
}

// blockDim = (threads per row, rows per block); more than one row per block
// only with 32 threads per row.  A thread holds NC chunks of 8 values.
// Y32, H32: y and h are 32-bit.  MIXED: the operands' types and alignments
// (`aligned`) are looked at one by one.
template <int NC, bool Y32, bool H32, bool MIXED>
__global__ void __launch_bounds__(NC == 1 ? 1024 : 512) block_norm_kernel(const moe_block_norm_args a, int aligned) {
  __shared__ float red[2][32];
  __shared__ __align__(16) uint32_t exchange[MIXED ? (NC == 1 ? 32 : 16) : 1][256];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= a.rows) return;
  const int H = a.hidden;
  const bool y32 = MIXED ? a.y_type == MOE_F32 : Y32, h32 = MIXED ? a.h_type == MOE_F32 : H32;
  const int yt = Y32 ? MOE_F32 : a.y_type, ht = H32 ? MOE_F32 : a.h_type;
  auto ok = [&](int bit) { return !MIXED || (aligned & bit); };
  uint32_t* buf = MIXED ? exchange[(threadIdx.y * blockDim.x + threadIdx.x) >> 5] : nullptr;
  auto at = [&](int c) { return static_cast<int>(c * blockDim.x + threadIdx.x) * 8; };
  Raw y[NC], h[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (a.y) y[c].load(a.y, y32, ok(kY), t * a.ld_y, at(c), H);
    else y[c].zero();
    if (a.h) h[c].load(a.h, h32, ok(kH), t * a.ld_h, at(c), H);
    else h[c].zero();
  }
  // narrow rows: the weights come with the row; wide ones: from L1 when they are used
  Raw wp[NC], wn[NC], gt[NC];
  const bool w32 = a.w_type == MOE_F32, g32 = a.gate_type == MOE_F32;
  const bool has_wp = a.post_norm && a.w_post, has_wn = a.pre_norm && a.w_pre, has_g = a.y && a.gate && a.ld_gate_col;
  auto load_w = [&](int c) {
    wp[c].zero();
    if (has_wp) wp[c].load(a.w_post, w32, ok(kWPost), 0, at(c), H);
    if (has_g) gt[c].load(a.gate, g32, ok(kGate), t * a.ld_gate_row, at(c), H);
  };
  auto load_wn = [&](int c) {
    wn[c].zero();
    if (has_wn) wn[c].load(a.w_pre, w32, ok(kWPre), 0, at(c), H);
  };
  if constexpr (NC == 1) load_w(0), load_wn(0);
  float g1 = 1.0f;
  if (a.y && a.gate && !a.ld_gate_col) g1 = load_elem(a.gate, a.gate_type, t * a.ld_gate_row);
  float v[NC][8];
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (a.y) y[c].settle(buf, y32, ok(kY));
    y[c].get(yt, v[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
  }
  const float inv_h = 1.0f / static_cast<float>(H);
  float rs = 1.0f;
  if (a.post_norm) rs = rsqrtf(row_sum(ss, red[0]) * inv_h + a.eps);
  ss = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if constexpr (NC > 1) load_w(c);
    if (a.y) {
      if (a.post_norm) {
        if (has_wp) wp[c].settle(buf, w32, ok(kWPost));
        scale_by(v[c], rs, a.w_add, wp[c], a.w_type);
      }
      if (has_g) {
        gt[c].settle(buf, g32, ok(kGate));
        scale_by(v[c], 1.0f, 0.0f, gt[c], a.gate_type);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= g1;
      }
    }
    if (a.h) {
      float hv[8];
      h[c].settle(buf, h32, ok(kH));
      h[c].get(ht, hv);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(a.residual_scale, hv[i], v[c][i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at(c) + i < H) ss = fmaf(v[c][i], v[c][i], ss);
    if (a.h_out) store_chunk(a.h_out, a.h_type, ok(kHOut), t * a.ld_h_out, at(c), H, v[c], buf);
  }
  if (!a.x_out) return;
  rs = 1.0f;
  if (a.pre_norm) rs = rsqrtf(row_sum(ss, red[1]) * inv_h + a.eps);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (a.pre_norm) {
      if constexpr (NC > 1) load_wn(c);
      if (has_wn) wn[c].settle(buf, w32, ok(kWPre));
      scale_by(v[c], rs, a.w_add, wn[c], a.w_type);
    }
    store_chunk(a.x_out, a.x_type, ok(kXOut), t * a.ld_x_out, at(c), H, v[c], buf);
  }
}

// The whole boundary (y and h, both norms, both outputs, at most a gate of
// every channel) of rows of a multiple of 8 values, for many rows.  One block
// of several teams per SM; a team takes rows by itself, 16 values a thread in
// two chunks of 8, and loads its next row while it works on one.  The weights
// lie in shared memory as fp32, the gate in the post-norm's, in two planes of
// 16 bytes a chunk; the arithmetic goes in pairs.  With the other kernel's
// some 60 instructions a value and weights read from L1 between the sums,
// issue and latency were the bound, not memory.  With fp32 h a thread's 72
// registers spill (28 bytes of stores, 92 with fp32 y too): 8192 x 7168 123 us
// from bf16 y and 140 from fp32, 84 and 87% of the copy rate.  Widths whose teams
// leave much of the 896 threads idle are slower: 4096 x 8192 (one team of 512)
// 69.4 us, 71% of that rate.
template <bool Y32, bool H32>
__global__ void __launch_bounds__(kStreamThreads, 1)
    block_norm_stream_kernel(const moe_block_norm_args a, int team_threads) {
  extern __shared__ __align__(16) float4 w4[];  // [post, pre][plane][chunk]
  __shared__ float red[kMaxTeams][4][16];       // by row parity and sum: a barrier lies between two uses of one
  const int H = a.hidden, chunks = 2 * team_threads;
  const int team = threadIdx.x / team_threads, tt = threadIdx.x - team * team_threads, teams = blockDim.x / team_threads;
  for (int c = threadIdx.x; c < 2 * chunks; c += blockDim.x) {
    // half-chunk c: elements [4 c, 4 c + 4) in plane c % 2 at chunk c / 2
    float p[4], n[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = 4 * c + i;
      p[i] = n[i] = 0.0f;
      if (k < H) {
        p[i] = a.w_add + (a.w_post ? load_elem(a.w_post, a.w_type, k) : 0.0f);
        if (a.gate) p[i] *= load_elem(a.gate, a.gate_type, k);
        n[i] = a.w_add + (a.w_pre ? load_elem(a.w_pre, a.w_type, k) : 0.0f);
      }
    }
    const int at = (c & 1) * chunks + (c >> 1);
    w4[at] = make_float4(p[0], p[1], p[2], p[3]);
    w4[2 * chunks + at] = make_float4(n[0], n[1], n[2], n[3]);
  }
  __syncthreads();

  const float inv_h = 1.0f / static_cast<float>(H), eps = a.eps;
  const int warp = tt >> 5, warps = team_threads >> 5, lane = tt & 31;
  float* const mine = &red[team][0][0];
  auto sum_row = [&](float v, int which) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) mine[which * 16 + warp] = v;
    named_bar(1 + team, team_threads);
    v = (lane & 15) < warps ? mine[which * 16 + (lane & 15)] : 0.0f;
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  };
  auto pairs = [](const uint4& lo, const uint4& hi, bool wide, int type, float2 (&v)[4]) {
    if (wide) {
      v[0] = make_float2(__uint_as_float(lo.x), __uint_as_float(lo.y));
      v[1] = make_float2(__uint_as_float(lo.z), __uint_as_float(lo.w));
      v[2] = make_float2(__uint_as_float(hi.x), __uint_as_float(hi.y));
      v[3] = make_float2(__uint_as_float(hi.z), __uint_as_float(hi.w));
    } else {
      float f[8];
      unpack8(lo, type, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
  };
  auto scaled = [&](float2 (&v)[4], float rs, const float4* w) {
    const float4 lo = w[0], hi = w[chunks];
    const float2 q = make_float2(rs, rs);
    v[0] = __fmul2_rn(__fmul2_rn(v[0], q), make_float2(lo.x, lo.y));
    v[1] = __fmul2_rn(__fmul2_rn(v[1], q), make_float2(lo.z, lo.w));
    v[2] = __fmul2_rn(__fmul2_rn(v[2], q), make_float2(hi.x, hi.y));
    v[3] = __fmul2_rn(__fmul2_rn(v[3], q), make_float2(hi.z, hi.w));
  };
  auto squares = [](const float2 (&v)[2][4]) {
    float2 q = __fmul2_rn(v[0][0], v[0][0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) q = __ffma2_rn(v[i >> 2][i & 3], v[i >> 2][i & 3], q);
    return q.x + q.y;
  };
  auto store = [&](char* p, bool wide, int type, const float2 (&v)[4]) {
    uint4* q = reinterpret_cast<uint4*>(p);
    if (wide) {
      q[0] = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
      q[1] = make_uint4(__float_as_uint(v[2].x), __float_as_uint(v[2].y), __float_as_uint(v[3].x), __float_as_uint(v[3].y));
    } else {
      q[0] = make_uint4(pack2(v[0].x, v[0].y, type), pack2(v[1].x, v[1].y, type), pack2(v[2].x, v[2].y, type),
                        pack2(v[3].x, v[3].y, type));
    }
  };

  // a team's threads cover chunk 0 wholly (H > 8 * team_threads), chunk 1 in part
  constexpr int YE = Y32 ? 4 : 2, HE = H32 ? 4 : 2;
  const int xe = elem_size(a.x_type), apart = team_threads * 8;
  const bool two = tt * 8 + apart < H;
  const int stride = static_cast<int>(gridDim.x) * teams;
  int64_t t = static_cast<int64_t>(blockIdx.x) * teams + team;
  if (t >= a.rows) return;
  const char* py = static_cast<const char*>(a.y) + (t * a.ld_y + tt * 8) * YE;
  const char* ph = static_cast<const char*>(a.h) + (t * a.ld_h + tt * 8) * HE;
  char* po = static_cast<char*>(a.h_out) + (t * a.ld_h_out + tt * 8) * HE;
  char* px = static_cast<char*>(a.x_out) + (t * a.ld_x_out + tt * 8) * xe;
  const float4* const wp = w4 + tt;
  const float4* const wn = w4 + 2 * chunks + tt;
  uint4 y[2][2], h[2][2];
  auto fetch = [&]() {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    y[0][0] = *reinterpret_cast<const uint4*>(py);
    if (Y32) y[0][1] = *reinterpret_cast<const uint4*>(py + 16);
    h[0][0] = *reinterpret_cast<const uint4*>(ph);
    if (H32) h[0][1] = *reinterpret_cast<const uint4*>(ph + 16);
    y[1][0] = two ? *reinterpret_cast<const uint4*>(py + apart * YE) : zero;
    if (Y32) y[1][1] = two ? *reinterpret_cast<const uint4*>(py + apart * YE + 16) : zero;
    h[1][0] = two ? *reinterpret_cast<const uint4*>(ph + apart * HE) : zero;
    if (H32) h[1][1] = two ? *reinterpret_cast<const uint4*>(ph + apart * HE + 16) : zero;
  };
  fetch();
  const float2 rscale = make_float2(a.residual_scale, a.residual_scale);
  for (int odd = 0;; odd ^= 2) {
    // places past the row hold zeros, so they add nothing to the sums
    float2 v[2][4];
    pairs(y[0][0], y[0][1], Y32, a.y_type, v[0]);
    pairs(y[1][0], y[1][1], Y32, a.y_type, v[1]);
    const float rs = rsqrtf(sum_row(squares(v), odd) * inv_h + eps);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float2 hv[4];
      scaled(v[c], rs, wp + c * team_threads);
      pairs(h[c][0], h[c][1], H32, a.h_type, hv);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] = __ffma2_rn(rscale, hv[i], v[c][i]);
    }
    t += stride;
    const bool more = t < a.rows;
    if (more) {
      py += stride * a.ld_y * YE;
      ph += stride * a.ld_h * HE;
      fetch();
    }
    store(po, H32, a.h_type, v[0]);
    if (two) store(po + apart * HE, H32, a.h_type, v[1]);
    const float rx = rsqrtf(sum_row(squares(v), odd + 1) * inv_h + eps);
    scaled(v[0], rx, wn);
    scaled(v[1], rx, wn + team_threads);
    store(px, a.x_type == MOE_F32, a.x_type, v[0]);
    if (two) store(px + apart * xe, a.x_type == MOE_F32, a.x_type, v[1]);
    if (!more) return;
    po += stride * a.ld_h_out * HE;
    px += stride * a.ld_x_out * xe;
  }
}

template <int NC>
cudaError_t launch_rows(const moe_block_norm_args& a, int aligned, dim3 grid, dim3 block, cudaStream_t st) {
  const bool y32 = a.y_type == MOE_F32, h32 = a.h_type == MOE_F32;
  if (aligned != kAll) block_norm_kernel<NC, false, false, true><<<grid, block, 0, st>>>(a, aligned);
  else if (y32 && h32) block_norm_kernel<NC, true, true, false><<<grid, block, 0, st>>>(a, aligned);
  else if (y32) block_norm_kernel<NC, true, false, false><<<grid, block, 0, st>>>(a, aligned);
  else if (h32) block_norm_kernel<NC, false, true, false><<<grid, block, 0, st>>>(a, aligned);
  else block_norm_kernel<NC, false, false, false><<<grid, block, 0, st>>>(a, aligned);
  return cudaGetLastError();
}

template <bool Y32, bool H32>
cudaError_t launch_stream(const moe_block_norm_args& a, int num_sms, cudaStream_t st) {
  const int threads = (a.hidden + 511) / 512 * 32;  // of a team: 16 values each
  const int fit = kStreamThreads / threads, teams = fit < kMaxTeams ? fit : kMaxTeams;
  const int smem = 2 * threads * 16 * static_cast<int>(sizeof(float));
  auto kernel = block_norm_stream_kernel<Y32, H32>;
  // the widest rows' size whatever this call's: the attribute is the process's,
  // and another thread's call may lie between this line and the launch
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             2 * kStreamHidden * static_cast<int>(sizeof(float)));
  if (e) return e;
  const int64_t blocks = (static_cast<int64_t>(a.rows) + teams - 1) / teams;
  kernel<<<static_cast<unsigned>(blocks < num_sms ? blocks : num_sms), threads * teams, smem, st>>>(
      a, threads);
  return cudaGetLastError();
}

bool vec_ok(const void* p, int type, int64_t ld) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * elem_size(type) % 16 == 0);
}

int check_matrix(const char* name, const void* p, int type, int64_t ld, int32_t hidden) {
  if (!elem_type_ok(type)) return reportf(MOE_ERR_ARG, "moe_block_norm: %s has an unknown type %d", name, type);
  if (reinterpret_cast<uintptr_t>(p) % elem_size(type))
    return reportf(MOE_ERR_ALIGN, "moe_block_norm: %s is not aligned to its elements", name);
  if (ld < hidden)
    return reportf(MOE_ERR_ARG, "moe_block_norm: %s has rows of %d values %lld apart", name, hidden,
                   static_cast<long long>(ld));
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int moe_block_norm(const moe_block_norm_args* args, void* stream) {
  using namespace moe;
  if (!args) return reportf(MOE_ERR_ARG, "moe_block_norm: args is NULL");
  const moe_block_norm_args a = *args;
  if (a.rows < 0) return reportf(MOE_ERR_ARG, "moe_block_norm: rows=%d is negative", a.rows);
  if (a.rows == 0) return MOE_OK;  // whatever the buffers: empty ones may be NULL
  if (a.hidden < 1 || a.hidden > kMaxHidden)
    return reportf(MOE_ERR_ARG, "moe_block_norm: hidden=%d must be in [1, %d]", a.hidden, kMaxHidden);
  if (!a.y && !a.h) return reportf(MOE_ERR_ARG, "moe_block_norm: y and h are both NULL");
  if (!a.h_out && !a.x_out) return reportf(MOE_ERR_ARG, "moe_block_norm: h_out and x_out are both NULL");
  if ((a.post_norm != 0 && a.post_norm != 1) || (a.pre_norm != 0 && a.pre_norm != 1))
    return reportf(MOE_ERR_ARG, "moe_block_norm: post_norm=%d and pre_norm=%d must be 0 or 1", a.post_norm, a.pre_norm);
  if (!(a.eps > 0.0f)) return reportf(MOE_ERR_ARG, "moe_block_norm: eps must be positive");
  if (a.w_add != 0.0f && a.w_add != 1.0f) return reportf(MOE_ERR_ARG, "moe_block_norm: w_add must be 0 or 1");
  int rc;
  if (a.y && (rc = check_matrix("y", a.y, a.y_type, a.ld_y, a.hidden))) return rc;
  if (a.h && (rc = check_matrix("h", a.h, a.h_type, a.ld_h, a.hidden))) return rc;
  if (a.h_out && (rc = check_matrix("h_out", a.h_out, a.h_type, a.ld_h_out, a.hidden))) return rc;
  if (a.x_out && (rc = check_matrix("x_out", a.x_out, a.x_type, a.ld_x_out, a.hidden))) return rc;
  if (a.w_post && (rc = check_matrix("w_post", a.w_post, a.w_type, a.hidden, a.hidden))) return rc;
  if (a.w_pre && (rc = check_matrix("w_pre", a.w_pre, a.w_type, a.hidden, a.hidden))) return rc;
  if (a.gate) {
    if ((rc = check_matrix("gate", a.gate, a.gate_type, a.hidden, a.hidden))) return rc;
    if ((a.ld_gate_col != 0 && a.ld_gate_col != 1) || a.ld_gate_row < 0)
      return reportf(MOE_ERR_ARG, "moe_block_norm: ld_gate_col=%lld must be 0 or 1, ld_gate_row=%lld not negative",
                     static_cast<long long>(a.ld_gate_col), static_cast<long long>(a.ld_gate_row));
  }

  const int aligned = kAll & ~((vec_ok(a.y, a.y_type, a.ld_y) ? 0 : kY) | (vec_ok(a.h, a.h_type, a.ld_h) ? 0 : kH) |
                               (vec_ok(a.h_out, a.h_type, a.ld_h_out) ? 0 : kHOut) |
                               (vec_ok(a.x_out, a.x_type, a.ld_x_out) ? 0 : kXOut) |
                               (vec_ok(a.w_post, a.w_type, 0) ? 0 : kWPost) | (vec_ok(a.w_pre, a.w_type, 0) ? 0 : kWPre) |
                               (!a.ld_gate_col || vec_ok(a.gate, a.gate_type, a.ld_gate_row) ? 0 : kGate));
  const int chunks = (a.hidden + 7) / 8;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (!e) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e) return reportf(MOE_ERR_CUDA, "moe_block_norm: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  if (aligned == kAll && a.hidden % 8 == 0 && a.hidden > 256 && a.hidden <= kStreamHidden && a.y && a.h && a.h_out && a.x_out &&
      a.post_norm && a.pre_norm && (!a.gate || (a.ld_gate_col && !a.ld_gate_row)) &&
      static_cast<int64_t>(a.rows) * a.hidden >= static_cast<int64_t>(kStreamValues) * sms) {
    const bool y32 = a.y_type == MOE_F32, h32 = a.h_type == MOE_F32;
    e = y32 && h32 ? launch_stream<true, true>(a, sms, st)
        : y32      ? launch_stream<true, false>(a, sms, st)
        : h32      ? launch_stream<false, true>(a, sms, st)
                   : launch_stream<false, false>(a, sms, st);
  } else {
    // A warp a row up to 256 values, else a block.  While there are fewer rows
    // than SMs, one chunk a thread up to 1024 threads: the weights then come
    // with the row instead of after each sum (one row of 7168: 4.1 -> 3.5 us).
    const int nc = chunks <= 512 || (chunks <= 1024 && a.rows <= sms) ? 1 : chunks <= 1024 ? 2 : 4;
    const dim3 block = chunks <= 32 ? dim3(32, 4) : dim3(((chunks + nc - 1) / nc + 31) / 32 * 32);
    const dim3 grid((static_cast<unsigned>(a.rows) + block.y - 1) / block.y);
    e = nc == 1   ? launch_rows<1>(a, aligned, grid, block, st)
        : nc == 2 ? launch_rows<2>(a, aligned, grid, block, st)
                  : launch_rows<4>(a, aligned, grid, block, st);
  }
  if (e != cudaSuccess) return reportf(MOE_ERR_CUDA, "moe_block_norm: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  return MOE_OK;
}
