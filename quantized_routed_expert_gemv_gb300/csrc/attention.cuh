// attention.cuh -- how attention over the paged cache is cut into work, shared
// by its kernels (attention.cu, attention_tc.cu).
//
// A unit is a tile of `tile_rows` rows of one key head of one sequence, a row
// being one token's query head of the head's group (row r: token r / group,
// head r % group); it has the key tiles of `bn` positions that its rows may
// see, one at least, and kUnitCost places more, for the time that it takes to begin and to
// end.  All units, ordered by sequence, head and row
// tile, make one line of T places, which is cut into equal parts, one a CTA:
// CTA c of G (G cut to T) has tiles T c / G to T (c + 1) / G.  So the work is
// even whatever the lengths, which the kernels alone know; neighbours share a head's
// keys in L2; and the cut, hence the order of every sum, depends on the sequences and
// the number of SMs only.
//
// A unit that lies in one CTA is finished there.  Of one that is cut, each CTA
// leaves its rows' maximum, sum and unnormalised output (fp32) in the
// workspace, in slot 0 if it continues the unit, in slot 1 if it begins it,
// with a note on who shares it, and the join kernel, launched behind, adds them up: each
// CTA's block there does an equal share of the unit's outputs.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "cache.cuh"
#include "common.cuh"

namespace moe {

constexpr float kLn2 = 0.69314718055994531f;

// How the cache's elements and the query's type meet.
enum Kind { kBf16, kF16, kE4m3Bf16, kE4m3F16 };
template <int K>
struct Traits {
  static constexpr bool f16 = K == kF16 || K == kE4m3F16, e4m3 = K == kE4m3Bf16 || K == kE4m3F16;
  static constexpr int size = e4m3 ? 1 : 2;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The bytes s of {a, b} (0..3 of a, 4..7 of b), lowest first.
__device__ __forceinline__ uint32_t bytes_of(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }

// What turns a head's e4m3 codes into 16-bit values: made by each lane of a warp
// from a scale of its own, taken from lane to lane by of().  `twice`: some lane's scale
// needs a second product.
template <bool B>
struct Bool {
  static constexpr bool value = B;
};

template <bool F16>
struct Dequant;

// bf16: the hardware's conversion to float16 (a NaN's code becomes a NaN), then the
// scale in fp32: exact, as a code has 4 significant bits.
template <>
struct Dequant<false> {
  float s;
  static constexpr bool twice = false;
  Dequant() = default;
  __device__ __forceinline__ explicit Dequant(float scale) : s(scale) {}
  template <bool TWICE>
  __device__ __forceinline__ Dequant of(int lane, Bool<TWICE>) const {
    return Dequant(__shfl_sync(0xFFFFFFFFu, s, lane));
  }
  // four codes to four values
  template <bool TWICE>
  __device__ __forceinline__ void operator()(uint32_t x, uint32_t* out, Bool<TWICE>) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __nv_fp8x2_storage_t two = static_cast<__nv_fp8x2_storage_t>(x >> 16 * i);
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
      out[i] = pack2(f.x * s, f.y * s, MOE_BF16);
    }
  }
};

// f16: the hardware's conversion, then the scale; one beyond float16's powers
// of two is multiplied on in two steps (the first one exact, the second one cut to
// where any code but 0 is infinite).
template <>
struct Dequant<true> {
  __half2 m, more;
  bool twice;
  Dequant() = default;
  __device__ __forceinline__ explicit Dequant(float s) {
    twice = __any_sync(0xFFFFFFFFu, s > 32768.0f || s < 6.103515625e-05f);
    const float c = fminf(fmaxf(s, 6.103515625e-05f), 32768.0f);
    m = __float2half2_rn(s == s ? c : s);
    more = __float2half2_rn(fminf(s / c, 32768.0f));
  }
  template <bool TWICE>
  __device__ __forceinline__ Dequant of(int lane, Bool<TWICE>) const {
    Dequant d;
    d.m = __shfl_sync(0xFFFFFFFFu, m, lane);
    if (TWICE) d.more = __shfl_sync(0xFFFFFFFFu, more, lane);
    return d;
  }
  template <bool TWICE>
  __device__ __forceinline__ void operator()(uint32_t x, uint32_t* out, Bool<TWICE>) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __nv_fp8x2_storage_t two = static_cast<__nv_fp8x2_storage_t>(x >> 16 * i);
      __half2 v = __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)), m);
      if (TWICE) v = __hmul2(v, more);
      out[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
};

// Whether one of two 16-bit values is an infinity or a NaN.
template <bool F16>
__device__ __forceinline__ bool odd_value(uint32_t x) {
  constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
  return (x & e) == e || ((x >> 16) & e) == e;
}

struct AttnArgs {
  Seqs q;
  const void* query;
  void* out;
  float* lse;
  int64_t ld_q, ld_out;
  const void *k, *v;  // the cache
  const float *k_scale, *v_scale;
  int64_t page_stride, slot_stride, head_stride;                 // bytes
  int64_t scale_page_stride, scale_slot_stride, scale_head_stride;  // floats
  int head_dim, kv_heads, group, causal, window;
  int type;           // of the query and the output
  float scale, scale_log2;  // scale, and scale * log2(e)
  Divisor by_group;
  unsigned* ctl;    // [0] error bits
  struct Note* notes;  // [G][2]
  float* part_ml;   // [G][2][tile_rows][2]: maximum of q . k, sum
  float* part_o;    // [G][2][tile_rows][head_dim]
};

// Who shares the unit of a slot.
struct Note {
  int c0, count;      // CTAs c0 .. c0 + count - 1 (0: the slot is not used)
  int row, rows;      // the unit's first row of the sequence, and its rows
  int first, head;    // the sequence's first row in the call's tensors, key head
};

// A unit's beginning and end cost about as much as these key tiles, of 64 positions or 128.
// 0, 1 and 3 of them, in a graph: 64 e4m3 sequences of 256 to 16384 positions with 8 rows 154,
// 137, 123 us; 16 ragged sequences of up to 2048 with up to 300 tokens 150, 99, 79;
// 2048 rows over 4096 195, 192, 190; only 16 windows of 1024 positions are not (18.0, 16.3, 16.9).
constexpr int kUnitCost = 3;

// What a row tile sees: positions [lo, hi) over all of its rows.
struct Tile {
  int rows;    // rows in the tile
  int lo, hi;
  int t0, t1;  // key tiles
};

// The positions that the token at position `pos` sees are [lo, hi).
__device__ __forceinline__ int sees_from(const AttnArgs& a, int pos) {
  return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
}
__device__ __forceinline__ int sees_to(const AttnArgs& a, int len, int pos) {
  return a.causal ? max(0, min(len, pos + 1)) : len;
}

template <int R, int BN>
__device__ __forceinline__ Tile tile_of(const AttnArgs& a, const Seq& s, int r) {
  Tile t;
  const int first = r * R, all = s.n * a.group;
  t.rows = min(R, all - first);
  const int base = s.len - s.n;
  t.lo = sees_from(a, base + static_cast<int>(divide(first, a.by_group)));
  t.hi = sees_to(a, s.len, base + static_cast<int>(divide(first + t.rows - 1, a.by_group)));
  t.t0 = t.lo / BN;
  t.t1 = max(t.t0 + 1, (t.hi + BN - 1) / BN);
  return t;
}

template <int R>
__device__ __forceinline__ int row_tiles(const AttnArgs& a, const Seq& s) {
  return (s.n * a.group + R - 1) / R;
}

// Place in the line: unit (seq, head, tile) and a place in it: key tiles follow
// its first kUnitCost ones.
struct Place {
  int seq, head, tile, at;
};

// Key tiles of one head of the sequences of this warp's lanes (all lanes;
// n = 0 for a lane without one): one row tile a lane by itself, more by the
// whole warp.
template <int R, int BN>
__device__ __forceinline__ int head_cost(const AttnArgs& a, const Seq& s) {
  const int nt = row_tiles<R>(a, s), lane = threadIdx.x & 31;
  int cost = 0;
  if (nt == 1) {
    const Tile t = tile_of<R, BN>(a, s, 0);
    cost = t.t1 - t.t0 + kUnitCost;
  }
#pragma unroll 1
  for (uint32_t many = __ballot_sync(0xFFFFFFFFu, nt > 1); many; many &= many - 1) {
    const int l = __ffs(many) - 1;
    Seq o;
    o.first = 0, o.n = __shfl_sync(0xFFFFFFFFu, s.n, l), o.len = __shfl_sync(0xFFFFFFFFu, s.len, l);
    const int tiles = row_tiles<R>(a, o);
    int sum = 0;
#pragma unroll 1
    for (int r = lane; r < tiles; r += 32) {
      const Tile t = tile_of<R, BN>(a, o, r);
      sum += t.t1 - t.t0 + kUnitCost;
    }
    sum = __reduce_add_sync(0xFFFFFFFFu, sum);
    if (lane == l) cost = sum;
  }
  return cost;
}

__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

struct PlanSmem {
  int tiles[32];                  // of each warp's sequences
  int chunk[kMaxSeqs / 128];      // of THREADS sequences at a time
  int off;                        // where the CTA's first tile lies in its head's tiles
  Place at;
  Seq seq;
};

// A CTA's part of the line.  The host refuses calls that might have 2^31 tiles.
struct Work {
  int total, begin, end;  // tiles in all; this CTA's (none: begin = end)
  int each, more;         // the first `more` CTAs have one tile more than `each`
  Place at;               // of the first tile
  Seq seq;
  __device__ __forceinline__ int cut(int c) const { return each * c + min(c, more); }
  __device__ __forceinline__ int cta_of(int x) const {  // the CTA that has tile x
    const int wide = more * (each + 1);
    return x < wide ? static_cast<uint32_t>(x) / (each + 1u) : more + static_cast<uint32_t>(x - wide) / each;
  }
};

// Moves to the next unit (a sequence without rows has none).  The sequence's
// values are loaded again where it changes.
template <int R>
__device__ __forceinline__ void next_unit(const AttnArgs& a, Place& p, Seq& s) {
  p.at = 0;
  if (++p.tile < row_tiles<R>(a, s)) return;
  p.tile = 0;
  if (++p.head < a.kv_heads) return;
  p.head = 0;
  do {
    if (++p.seq >= a.q.n) return;
    s = load_seq(a.q, p.seq);
  } while (s.n == 0);
}

// All of a CTA's threads (THREADS, a multiple of 128) find its part of the line.
// Starts that fall would let sequences share rows, so that their tiles have no
// bound that the host could have checked: no CTA has a part then.
// It runs once a CTA, from instructions that come from afar, so its time goes by
// its length: few and narrow operations (with 64-bit ones and divisions for
// every cut it took 6500 clocks instead of 4000 in front of 128 rows over 32768).
template <int R, int BN, int THREADS>
__device__ __forceinline__ Work find_work(const AttnArgs& a, PlanSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = (a.q.n + THREADS - 1) / THREADS;
  Work w;
  w.total = 0;
  int cost, incl;  // tiles of a head of this thread's sequence, and of the chunk's sequences up to it
  Seq mine;
  int ch = 0, before = 0;
  bool again = false, falls = false;
#pragma unroll 1
  for (;;) {
    mine = {0, 0, 0};
    bool fall = false;
    if (ch * THREADS + tid < a.q.n) mine = load_seq(a.q, ch * THREADS + tid, fall);
    cost = head_cost<R, BN>(a, mine);
    incl = warp_scan(cost * a.kv_heads);
    if (lane == 31) sm.tiles[warp] = incl;
    falls |= __syncthreads_or(fall) != 0;
    const int v = lane < THREADS / 32 ? sm.tiles[lane] : 0;
    const int all = __reduce_add_sync(0xFFFFFFFFu, v);
    incl += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? v : 0);
    if (again) break;
    if (chunks > 1 && tid == 0) sm.chunk[ch] = all;
    w.total += all;
    if (chunks > 1) __syncthreads();
    if (++ch < chunks) continue;
    // its first and last tile
    const int grid = gridDim.x, ctas = grid < w.total ? grid : w.total, c = blockIdx.x;
    w.begin = w.end = 0;
    if (falls) {
      if (c == 0 && tid == 0) latch_error(a.ctl, kErrRange);
      return w;
    }
    if (c >= ctas) return w;
    w.each = static_cast<uint32_t>(w.total) / static_cast<uint32_t>(ctas), w.more = w.total - w.each * ctas;
    w.begin = w.cut(c), w.end = w.cut(c + 1);
    if (chunks == 1) break;
    for (ch = 0; ch + 1 < chunks && before + sm.chunk[ch] <= w.begin; ++ch) before += sm.chunk[ch];
    again = true;
  }
  if (chunks == 1) ch = 0;
  const int from = before + incl - cost * a.kv_heads;
  if (from <= w.begin && w.begin < before + incl) {
    const int off = w.begin - from, head = static_cast<uint32_t>(off) / static_cast<uint32_t>(cost);
    sm.at.seq = ch * THREADS + tid, sm.at.head = head, sm.at.tile = 0, sm.at.at = sm.off = off - head * cost;
    sm.seq = mine;
  }
  __syncthreads();
  const int tiles = row_tiles<R>(a, sm.seq);
  if (tiles > 1) {  // the row tile, 32 of them at a time
    if (warp == 0) {
      const Seq s = sm.seq;
      int rem = sm.off;
#pragma unroll 1
      for (int r0 = 0; r0 < tiles; r0 += 32) {
        int n = 0;
        if (r0 + lane < tiles) {
          const Tile t = tile_of<R, BN>(a, s, r0 + lane);
          n = t.t1 - t.t0 + kUnitCost;
        }
        const int up_to = warp_scan(n);
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, up_to > rem);
        if (past) {
          if (lane == __ffs(past) - 1) sm.at.tile = r0 + lane, sm.at.at = rem - (up_to - n);
          break;
        }
        rem -= __shfl_sync(0xFFFFFFFFu, up_to, 31);
      }
    }
    __syncthreads();
  }
  w.at = sm.at, w.seq = sm.seq;
  return w;
}

// One CTA's pieces of units, in order.  Each warp has one (or two) in shared memory,
// which its first lane moves on: registers are short.
template <int R, int BN>
struct Walk {
  Place at;
  Seq seq;
  Tile tile;
  int x, end;  // places of the line: the piece's first, the CTA's last
  int length;  // places of the piece
  int ta, tb;  // its key tiles
  __device__ __forceinline__ void begin(const AttnArgs& a, const Work& work) {
    at = work.at, seq = work.seq, x = work.begin, end = work.end;
    if (!cut(a)) step(a);
  }
  // The piece at x; false if it has no key tiles.
  __device__ __forceinline__ bool cut(const AttnArgs& a) {
    tile = tile_of<R, BN>(a, seq, at.tile);
    length = min(tile.t1 - tile.t0 + kUnitCost - at.at, end - x);
    ta = tile.t0 + max(at.at - kUnitCost, 0);
    tb = tile.t0 + at.at + length - kUnitCost;
    return tb > ta;
  }
  __device__ __forceinline__ bool more() const { return x < end; }
  __device__ __forceinline__ bool whole() const { return ta == tile.t0 && tb == tile.t1; }
  // all lanes of the warp
  __device__ __forceinline__ void next(const AttnArgs& a) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) step(a);
    __syncwarp();
  }
  // all lanes: a copy, and a copy one piece ahead
  __device__ __forceinline__ void become(const Walk& o) {
    __syncwarp();
    static_assert(sizeof(Walk) % 4 == 0 && sizeof(Walk) <= 128, "a word a lane");
    if ((threadIdx.x & 31) < sizeof(Walk) / 4)
      reinterpret_cast<int*>(this)[threadIdx.x & 31] = reinterpret_cast<const int*>(&o)[threadIdx.x & 31];
    __syncwarp();
  }
  __device__ __forceinline__ void follow(const AttnArgs& a, const Walk& o) {
    become(o);
    next(a);
  }
  __device__ __forceinline__ void step(const AttnArgs& a) {
    while (x < end) {
      x += length;
      next_unit<R>(a, at, seq);
      if (x >= end || cut(a)) return;
    }
  }
  // Who shares a piece that is not whole, for the join.
  __device__ __forceinline__ void note(const AttnArgs& a, const Work& work) const {
    const int first = x - at.at + kUnitCost;  // the place of the unit's first key tile
    Note n;
    n.c0 = work.cta_of(first), n.count = work.cta_of(first + tile.t1 - tile.t0 - 1) - n.c0 + 1;
    n.row = at.tile * R, n.rows = tile.rows, n.first = seq.first, n.head = at.head;
    a.notes[2 * blockIdx.x + (ta == tile.t0 ? 1 : 0)] = n;
  }
};

// Lets a kernel have `bytes` of dynamic shared memory, once a device (`allowed`: a
// bit each; a second thread may do it again, with the same value).
template <class F>
cudaError_t allow_smem(std::atomic<uint64_t>& allowed, F* kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e || (dev < 64 && allowed.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (!e && dev < 64) allowed.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

cudaError_t launch_tiles(const AttnArgs& a, Kind k, int num_sms, cudaStream_t st);
int tiles_rows(int head_dim);   // rows of launch_tiles' tiles
int tiles_keys(int head_dim);   // their positions
float tiles_lift(bool f16);     // its exponentials' factor, in powers of two
cudaError_t launch_join(const AttnArgs& a, int grid, int tile_rows, bool f16, float lift, cudaStream_t st);

}  // namespace moe
