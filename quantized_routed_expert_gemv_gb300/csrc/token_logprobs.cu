// token_logprobs.cu -- log probabilities, ranks, entropy and top tokens of
// rows of logits (moe_token_logprobs), in one pass over the logits.
//
// Mathematics, in powers of two: with u = scale * log2(e) and a reference r
// near the row's largest u l,
//     S = sum_v 2^(u l_v - r),  A = sum_v (u l_v - r) 2^(u l_v - r)
//     lse = ln 2 (r + log2 S),  entropy = ln 2 (log2 S - A / S),
//     logprob_t = ln 2 (u l_t - r - log2 S).
// One fma gives u l - r with a single rounding.  Every thread keeps its own
// (r, S, A) in fp32 and moves r only when a logit lies more than kRefSlack
// powers of two above it, so the usual step has no rescaling.
//
// r is a rounded product itself, so the term of the logit that it came from is
// 2^(u l - r), up to 2^64 where |r| < 2^31 and without bound above.  So from
// |u l| = 2^31 on nothing is summed: values there are 128 powers of two and
// more from their neighbours, whatever the type.  Those below -2^31 (masks such
// as -1e10 or the type's lowest value) add 0, and a row whose largest is that
// far from 0 has all of its probability on the logits equal to it, which are
// counted instead.
//
// No sum overflows: a term is at most 2^88 (kRefSlack and a residual of 2^3
// below |r| = 2^28, 2^64 above, where r moves with every larger logit), there
// are at most 2^24 of them, and A has a factor of 2^14 at most.
//
// Top tokens: a thread's running maximum is the best of the group of tokens
// that thread visited.  Any token of the row's top n lies in one of the n
// groups whose best tokens come first: the best of each group before its own
// comes before it too.  So the pass keeps one value per thread, and afterwards
// only winning groups are read again, for the tokens that do not come after
// the n-th group's best, or after a lower value that n groups reach.
//
// A row is read by one block, or by a cluster of up to 8 blocks, each a
// contiguous part, when there are too few rows for the SMs; the parts meet in
// the first block's shared memory and are joined in rank order, so results do
// not depend on timing.
//
// Bound: for many long rows memory, and the latency of a row's end, which the
// pass of the SM's other blocks covers in part: 4096 rows of 131072 bf16 with 5
// alternatives 171 to 174 us, 6.2 to 6.3 TB/s, 91 to 92% of the measured copy
// rate.  Reading alone goes faster than copying: 2048 rows of 131072 fp32
// without targets or alternatives 155 us, 6.9 TB/s, 102% of that rate, so some
// 10% are left there.  For shorter rows the rows' ends: 4096 rows of 32000 54 us,
// of 4000 24.  For few rows the chain of steps: one row of 131072 with 20
// alternatives 8.5 to 9.9 us.  Tried: blocks of 512 threads 215 us, warps of
// their own for the rows' ends 224.
// The instances for 8 targets of 16-bit logits spill at 64 registers, 216 to 372
// bytes of stores a thread without the ring, 36 to 80 with it; those for 2 and 4
// targets without it 16 to 96.  4096 rows of 65536 with 8 targets and 20 alternatives take 235 us,
// where one target and 5 take 97.
#include <climits>
#include <cmath>
#include <cstdint>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "elem.cuh"

namespace moe {
int reportf(int code, const char* fmt, ...);

namespace {

namespace cg = cooperative_groups;

// chunks of 8 logits a thread loads at once
__host__ __device__ constexpr int batch_of(int type) { return type == MOE_F32 ? 2 : 4; }
constexpr int kBatchBytes = 64;        // of a thread
// Batches a thread has in shared memory where it copies through there: one in
// use, two on their way.  A thread copies for itself, so the pass has no
// barrier; registers have room for one batch on its way.
constexpr int kRing = 3;
constexpr int kMaxTop = 32;
constexpr int kMaxTargets = 8;
constexpr int kMaxSplit = 8;
constexpr int kSplitThreads = 256;     // of blocks that may read parts of a row
constexpr int kSmallVocab = 56 * 1024, kRingVocab = 12 * 1024;  // launch_type's
constexpr int64_t kPartBytes = 32 * 1024;  // of a row, at least, in a part
constexpr int kCand = 1024;            // candidate buffer of the top selection
constexpr float kRefSlack = 80.0f;     // powers of two a logit may lie above the reference
constexpr float kUnset = 3.402823466e38f;
constexpr float kSlackBelow = 268435456.0f;  // 2^28: |r| from which r moves with every larger logit
constexpr float kFar = 2147483648.0f;  // 2^31: |u l| from which logits are not summed
constexpr float kLn2 = 0.6931471805599453f;

struct Key {  // order: value descending, id ascending; id < 0: none
  float v;
  int id;
};

__device__ __forceinline__ bool before(const Key& a, const Key& b) { return a.v > b.v || (a.v == b.v && a.id < b.id); }

// What a block knows of its part of a row.
struct Part {
  float r, S, A, best;
  int cnt[kMaxTargets];
  Key top[kMaxTop];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max that returns NaN if either is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Smallest value above v: x > v iff x >= next_up(v) (NaN for NaN and +inf).
__device__ __forceinline__ float next_up(float v) {
  const uint32_t u = __float_as_uint(v);
  if (v == 0.0f) return __uint_as_float(1u);
  if (v != v) return v;  // NaN stays NaN
  return __uint_as_float(v > 0.0f ? u + 1 : u - 1);
}
__device__ __forceinline__ uint32_t next_up16(uint32_t bits, uint32_t inf) {
  if ((bits & 0x7FFFu) == 0) return 1u;
  if ((bits & 0x7FFFu) > inf) return bits;  // NaN stays NaN
  return bits & 0x8000u ? bits - 1 : bits + 1;
}

// A thread's running sums; nr is minus the reference, twice, and `limit` the
// logit above which the reference has to move (nr unset: what adds at all).
struct Sums {
  float2 nr = {-kUnset, -kUnset}, S = {0.0f, 0.0f}, A = {0.0f, 0.0f};
  float limit;
  __device__ __forceinline__ explicit Sums(float u) : limit(-kFar / u) {}

  // Makes room for logits up to m.
  __device__ __forceinline__ void reach(float m, float u) {
    if (m > limit) {
      const float z = m * u;
      const float d = nr.x == -kUnset ? -1e4f : max_nan(-nr.x - z, -1e4f);
      const float e = ex2(d);
      A.x = fmaf(S.x, d, A.x) * e, A.y = fmaf(S.y, d, A.y) * e;
      S.x *= e, S.y *= e;
      nr = make_float2(-z, -z);
      // rounded down: to nearest, the next float above a large m could pass
      limit = fabsf(z) < kSlackBelow ? __fadd_rd(m, kRefSlack / u) : m;
    }
  }
  // Two logits (already bounded below unless CLAMP); uu is u twice.
  template <bool CLAMP>
  __device__ __forceinline__ void add(float2 l, float2 uu) {
    float2 d = __ffma2_rn(l, uu, nr);
    if (CLAMP) d.x = max_nan(d.x, -200.0f), d.y = max_nan(d.y, -200.0f);
    const float2 e = make_float2(ex2(d.x), ex2(d.y));
    S = __fadd2_rn(S, e);
    A = __ffma2_rn(e, d, A);
  }
};

// Masks of two 16-bit halves that are not below thr's, and the equal ones.
template <int TYPE>
__device__ __forceinline__ uint32_t ge_mask(uint32_t w, uint32_t thr) {
  if constexpr (TYPE == MOE_BF16)
    return __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&thr));
  else
    return __hge2_mask(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&thr));
}

// Joins the (r, S, A) of a warp's lanes in every lane: moved to the largest
// reference, then summed in a fixed order.  Lanes without a sum have r unset
// and S = 0.
__device__ __forceinline__ void join_warp(float& r, float& S, float& A) {
  const int b = __float_as_int(r == kUnset ? -INFINITY : r);
  const int key = __reduce_max_sync(0xFFFFFFFFu, b ^ ((b >> 31) & 0x7FFFFFFF));
  const float top = __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF));
  const float d = r == kUnset ? -1e4f : max_nan(r - top, -1e4f), e = exp2f(d);
  A = fmaf(S, d, A) * e;
  S *= e;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    S += __shfl_xor_sync(0xFFFFFFFFu, S, o);
    A += __shfl_xor_sync(0xFFFFFFFFu, A, o);
  }
  r = top == -INFINITY ? kUnset : top;
}

__device__ __forceinline__ float max_warp(float v) {
  const int b = __float_as_int(v);
  const int key = __reduce_max_sync(0xFFFFFFFFu, b ^ ((b >> 31) & 0x7FFFFFFF));
  return __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF));
}

// Calls emit(place, i) for the keys among the first n of keys[0..m): a key's
// place is the number of keys before it.  A warp takes four keys at a time
// (32 alternatives in 4096 rows of 32000: 116 us with one, 102 with four; 5
// alternatives 52.2 and 52.9).
template <int kWarps, class Emit>
__device__ __forceinline__ void place_keys(const Key* keys, int m, int n, Emit emit) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = 4 * (threadIdx.x >> 5); i < m; i += 4 * kWarps) {
    Key k[4];
    int c[4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = keys[min(i + j, m - 1)];
#pragma unroll 1
    for (int q = lane; q < m; q += 32) {
      const Key o = keys[q];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] += before(o, k[j]);
    }
    int place = n;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = __reduce_add_sync(0xFFFFFFFFu, c[j]);
      if (lane == j) place = c[j];
    }
    if (lane < 4 && i + lane < m && place < n) emit(place, i + lane);
  }
}

// The row's logits on a grid of 16-byte aligned addresses: chunk c holds
// elements [8 c - off, 8 c - off + 8).  Chunks [w0, w1) lie wholly in the row;
// the elements before and after them, at most 14, are its edges.
template <int TYPE>
struct Row {
  static constexpr int ES = TYPE == MOE_F32 ? 4 : 2;
  const char* p;
  int off, vocab, w0, w1;
  __device__ __forceinline__ Row(const moe_token_logprobs_args& a, int64_t t) {
    p = static_cast<const char*>(a.logits) + t * a.ld_logits * ES;
    off = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / ES);
    vocab = a.vocab;
    w0 = off ? 1 : 0;
    w1 = max(w0, (vocab + off) / 8);
  }
  __device__ __forceinline__ const uint4* chunk(int c) const {
    return reinterpret_cast<const uint4*>(p + (static_cast<int64_t>(c) * 8 - off) * ES);
  }
  __device__ __forceinline__ void load(int c, float (&v)[8]) const { load8(chunk(c), TYPE, 0, v); }
  __device__ __forceinline__ float at(int j) const { return load_elem(p, TYPE, j); }
  // The i-th edge element's index, or -1.
  __device__ __forceinline__ int edge(int i) const {
    const int head = min(vocab, 8 * w0 - off);
    if (i < head) return i;
    const int j = i - head + max(head, 8 * w1 - off);
    return j < vocab ? j : -1;
  }
};

template <int THREADS>
struct Picks {                 // of the top selection
  Key group[THREADS];          // groups at or above the cut: best token ...
  int owner[THREADS];          // ... and thread
  Key cand[kCand];
};

template <int THREADS, bool RING>
union Shared {
  Picks<THREADS> picks;
};
template <int THREADS>
union Shared<THREADS, true> {
  Picks<THREADS> picks;                             // after the pass
  uint4 ring[kRing][kBatchBytes / 16][THREADS];     // the pass: batches of the threads
};

template <int THREADS, bool RING>
struct Smem {
  static constexpr int kWarps = THREADS / 32;
  Shared<THREADS, RING> u;
  Part parts[THREADS == kSplitThreads ? kMaxSplit : 1];  // the cluster's first block: one per part
  Part mine;
  float team[32];              // best value of each team of THREADS / 32 threads
  float cut;                   // value no group of the top n lies below
  int ngroup, ncand;
  Key sel[kMaxTop];            // the n first groups
  int sel_owner[kMaxTop];
  Key last, best[kWarps];
  float r[kWarps], S[kWarps], A[kWarps];
  int cnt[kWarps][kMaxTargets];
};

// The first n tokens of this block's part to part.top.
template <int TYPE, int THREADS, bool RING>
__device__ __forceinline__ void select_top(const Row<TYPE>& row, Smem<THREADS, RING>& sm, int n, int c0, int c1,
                                           float best, int best_b, float edge_v, int edge_j) {
  constexpr int kBatch = batch_of(TYPE), kThreads = THREADS, kWarps = THREADS / 32;
  Picks<THREADS>& pk = sm.u.picks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // a value that n groups reach: the n-th largest of 32 teams' best
  constexpr int kTeam = kThreads / 32;
  float h = best;
#pragma unroll
  for (int o = kTeam / 2; o; o >>= 1) h = fmaxf(h, __shfl_xor_sync(0xFFFFFFFFu, h, o));
  if (tid % kTeam == 0) sm.team[tid / kTeam] = h;
  if (tid == 0) sm.ngroup = sm.ncand = 0, sm.cut = -INFINITY;
  if (tid < kMaxTop) sm.mine.top[tid].v = -INFINITY, sm.mine.top[tid].id = -1;
  __syncthreads();
  if (warp == 0) {
    const float v = sm.team[lane];
    int place = 0;
#pragma unroll 8
    for (int q = 0; q < 32; ++q) {
      const float w = __shfl_sync(0xFFFFFFFFu, v, q);
      place += w > v || (w == v && q < lane);
    }
    if (place == n - 1) sm.cut = v;
  }
  __syncthreads();
  // Groups that reach it.  Where these are little more than n, all of their
  // tokens that reach it are candidates: that spares looking for the groups'
  // tokens and their order (4096 rows of 8192 bf16 with 5 alternatives 30.4 us
  // without, 26.3 with; of 131072 176 and 171).  Else the n-th group's best is
  // the bound, and fewer groups are read again.
  int slot = -1;
  if (best > -INFINITY && best >= sm.cut) {
    slot = atomicAdd(&sm.ngroup, 1);
    pk.owner[slot] = tid;
  }
  __syncthreads();
  const int m = sm.ngroup;
  int winners = m;
  const int* owner = pk.owner;
  Key cut = {sm.cut, INT_MAX};
  if (m > n + n / 2 + 4) {
    if (slot >= 0) {
      // the token: the first place of that value in the batch it was seen in
      int id = -1;
#pragma unroll
      for (int i = kBatch - 1; i >= 0; --i) {
        const int c = best_b + i * kThreads + tid;
        if (c < c1) {
          float v[8];
          row.load(c, v);
#pragma unroll
          for (int k = 7; k >= 0; --k)
            if (v[k] == best) id = 8 * c - row.off + k;
        }
      }
      pk.group[slot].v = best, pk.group[slot].id = id;
    }
    __syncthreads();
    place_keys<kWarps>(pk.group, m, n, [&](int place, int i) {
      sm.sel[place] = pk.group[i], sm.sel_owner[place] = pk.owner[i];
    });
    __syncthreads();
    cut = sm.sel[n - 1];  // there are more than n
    owner = sm.sel_owner;
    winners = n;
  }
  auto push = [&](float v, int id) {
    const Key k = {v, id};
    if (v > -INFINITY && !before(cut, k)) {
      const int s = atomicAdd(&sm.ncand, 1);
      if (s < kCand) pk.cand[s] = k;
    }
  };
  if (edge_j >= 0) push(edge_v, edge_j);
  // chunk k of winner g is item g * chunks + k, one thread each
  const int chunks = (c1 - c0 + kThreads - 1) / kThreads, items = winners * chunks;
#pragma unroll 1
  for (int e = tid; e < items; e += kThreads) {
    const int g = e / chunks, c = c0 + owner[g] + (e - g * chunks) * kThreads;
    if (c < c1) {
      float v[8];
      row.load(c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) push(v[i], 8 * c - row.off + i);
    }
  }
  __syncthreads();
  const int nc = sm.ncand;
  if (nc <= kCand) {
    place_keys<THREADS / 32>(pk.cand, nc, n, [&](int place, int i) { sm.mine.top[place] = pk.cand[i]; });
    return;
  }
  // many tokens in few groups: one round over the winning groups per place
  if (tid == 0) sm.last.v = INFINITY, sm.last.id = -1;
  __syncthreads();
  for (int r = 0; r < n; ++r) {
    const Key last = sm.last;
    Key b = {-INFINITY, -1};
    auto look = [&](float v, int id) {
      const Key k = {v, id};
      if (v > -INFINITY && before(last, k) && (b.id < 0 || before(k, b))) b = k;
    };
    if (edge_j >= 0) look(edge_v, edge_j);
    for (int e = tid; e < items; e += kThreads) {
      const int g = e / chunks, c = c0 + owner[g] + (e - g * chunks) * kThreads;
      if (c < c1) {
        float v[8];
        row.load(c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) look(v[i], 8 * c - row.off + i);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const Key k = {__shfl_xor_sync(0xFFFFFFFFu, b.v, o), __shfl_xor_sync(0xFFFFFFFFu, b.id, o)};
      if (k.id >= 0 && (b.id < 0 || before(k, b))) b = k;
    }
    if (lane == 0) sm.best[warp] = b;
    __syncthreads();
    if (tid == 0) {
      Key w = {-INFINITY, -1};
      for (int q = 0; q < kWarps; ++q)
        if (sm.best[q].id >= 0 && (w.id < 0 || before(sm.best[q], w))) w = sm.best[q];
      sm.mine.top[r] = w;
      if (w.id >= 0) sm.last = w;
    }
    __syncthreads();
  }
}

// NT: targets whose ranks are counted, rounded up to 0, 1, 2, 4 or 8.
template <int TYPE, int NT, int THREADS, bool RING>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    token_logprobs_kernel(const moe_token_logprobs_args a, int parts) {
  extern __shared__ uint4 dyn_smem[];
  constexpr int kThreads = THREADS, kWarps = THREADS / 32;
  using Sm = Smem<THREADS, RING>;
  Sm& sm = *reinterpret_cast<Sm*>(dyn_smem);
  constexpr bool F32 = TYPE == MOE_F32;
  constexpr int kBatch = batch_of(TYPE);
  constexpr int NG = NT > 0 ? NT : 1;
  cg::cluster_group cluster = cg::this_cluster();
  const int split = THREADS == kSplitThreads ? parts : 1;
  const int rank = split > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  if (split > 1) cluster.barrier_arrive();  // paired with the wait before the parts meet
  const int64_t t = blockIdx.x / split;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Row<TYPE> row(a, t);
  const float u = a.scale * 1.4426950408889634f;
  const int per = (row.w1 - row.w0 + split - 1) / split;
  const int c0 = min(row.w1, row.w0 + rank * per), c1 = min(row.w1, c0 + per);

  // Raw logits of a batch: chunk i at c + i * kThreads, -inf outside the part.
  // The batches before the last are whole for every thread.
  constexpr int Q = F32 ? 2 : 1, kStep = kBatch * kThreads;
  using Batch = uint4[kBatch][Q];
  static_assert(sizeof(Batch) == kBatchBytes && !(RING && F32), "a batch in the ring, of 16-bit logits");
  constexpr uint32_t fill = F32 ? 0xFF800000u : TYPE == MOE_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
  auto fetch = [&](Batch& raw, int cb) {
    const uint4* p = row.chunk(cb + tid);
    if (cb + kStep <= c1) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int q = 0; q < Q; ++q) raw[i][q] = __ldg(p + i * kThreads * Q + q);
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int q = 0; q < Q; ++q)
          raw[i][q] =
              cb + tid + i * kThreads < c1 ? __ldg(p + i * kThreads * Q + q) : make_uint4(fill, fill, fill, fill);
    }
  };
  auto copy = [&](int slot, int cb) {  // the same into the ring
    if constexpr (RING) {
      const uint4* p = row.chunk(cb + tid);
      uint4* const to = &sm.u.ring[slot][0][tid];
      auto one = [&](int i) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(
                         __cvta_generic_to_shared(to + i * kThreads))),
                     "l"(p + i * kThreads)
                     : "memory");
      };
      if (cb + kStep <= c1) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) one(i);
      } else if (cb < c1) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (cb + tid + i * kThreads < c1) one(i);
          else to[i * kThreads] = make_uint4(fill, fill, fill, fill);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  Batch even;
  if constexpr (RING) {
    for (int i = 0; i < kRing - 1; ++i) copy(i, c0 + i * kStep);
  } else {
    fetch(even, c0);
  }

  // the first block's first warp writes the row's answers: its targets' logits
  int my_target = -1;
  float my_logit = 0.0f;
  if (rank == 0 && tid < a.n_targets) {
    my_target = a.targets[t * a.n_targets + tid];
    if (my_target >= a.vocab) my_target = -1;
    if (my_target >= 0) my_logit = row.at(my_target);
  }
  // ranks: chunk c counts logits >= lo if it lies before the target's chunk,
  // else >= hi (the next value); the target's own chunk is completed below
  int tj[NG], tc[NG];
  float xt[NG];
  uint32_t lo[NG], hi[NG], cnt[NG];
  if constexpr (NT > 0) {
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      tj[g] = g < a.n_targets ? a.targets[t * a.n_targets + g] : -1;
      const bool in = tj[g] >= 0 && tj[g] < a.vocab;
      if (!in) tj[g] = -1;
      xt[g] = in ? row.at(tj[g]) : NAN;
      tc[g] = in ? (tj[g] + row.off) / 8 : -1;
      cnt[g] = 0;
      if constexpr (F32) {
        lo[g] = __float_as_uint(xt[g]);
        hi[g] = __float_as_uint(next_up(xt[g]));
      } else {
        const uint32_t nan = TYPE == MOE_BF16 ? 0x7FC0u : 0x7E00u;
        const uint32_t b = in ? reinterpret_cast<const uint16_t*>(row.p)[tj[g]] : nan;
        const uint32_t n = next_up16(b, TYPE == MOE_BF16 ? 0x7F80u : 0x7C00u);
        lo[g] = b * 0x10001u;
        hi[g] = n * 0x10001u;
      }
    }
  }

  // Read early, used after the pass, in the first part: the row's edges, one
  // thread each, and the logits before a target in its own chunk, eight
  // threads each.
  int edge_j = -1, fix_g = -1;
  float edge_v = -INFINITY, fix_v = NAN;
  if (rank == 0) {
    if (tid < 16) edge_j = row.edge(tid);
    if (edge_j >= 0) edge_v = row.at(edge_j);
    if constexpr (NT > 0) {
#pragma unroll
      for (int g = 0; g < NT; ++g) {
        const int j = 8 * tc[g] - row.off + (lane & 7);
        if (warp == g % kWarps && lane >> 3 == g / kWarps && tc[g] >= row.w0 && tc[g] < row.w1 && j < tj[g])
          fix_g = g, fix_v = row.at(j);
      }
    }
  }

  Sums sums(u);
  float best = -INFINITY;
  int best_c = -1;
  // bf16 logits are bounded below before they are widened, so that a value far
  // under the reference gives 0 * finite in A
  const float bound = __bfloat162float(__float2bfloat16_rn(fmaxf(-1.2676506e30f / u, -3.3895314e38f)));
  const __nv_bfloat162 bound2 = __float2bfloat162_rn(bound);
  const float2 uu = make_float2(u, u);
  // a batch whose first chunk is cb; this thread's are cb + tid + i * kThreads
  auto process = [&](const Batch& cur, int cb) {
    float m;
    if constexpr (F32) {
      m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          m = fmaxf(m, fmaxf(__uint_as_float(cur[i][q].x), __uint_as_float(cur[i][q].y)));
          m = fmaxf(m, fmaxf(__uint_as_float(cur[i][q].z), __uint_as_float(cur[i][q].w)));
        }
    } else if constexpr (TYPE == MOE_BF16) {
      __nv_bfloat162 w = *reinterpret_cast<const __nv_bfloat162*>(&cur[0][0].x);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(&cur[i][0]);
        w = __hmax2(w, __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3])));
      }
      m = fmaxf(__low2float(w), __high2float(w));
    } else {
      __half2 w = *reinterpret_cast<const __half2*>(&cur[0][0].x);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const __half2* v = reinterpret_cast<const __half2*>(&cur[i][0]);
        w = __hmax2(w, __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3])));
      }
      m = fmaxf(__low2float(w), __high2float(w));
    }
    best_c = m > best ? cb : best_c;
    best = fmaxf(best, m);
    sums.reach(m, u);
    // sums first: the targets' logits of a short row may still be on their way
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const uint32_t w[4] = {cur[i][q].x, cur[i][q].y, cur[i][q].z, cur[i][q].w};
        if constexpr (F32) {
          sums.add<true>(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), uu);
          sums.add<true>(make_float2(__uint_as_float(w[2]), __uint_as_float(w[3])), uu);
        } else {
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            if constexpr (TYPE == MOE_BF16) {
              const __nv_bfloat162 v = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w[z]), bound2);
              const uint32_t x = *reinterpret_cast<const uint32_t*>(&v);
              sums.add<false>(make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)), uu);
            } else {
              sums.add<true>(__half22float2(*reinterpret_cast<const __half2*>(&w[z])), uu);
            }
          }
        }
      }
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      // logits not below the target's in a batch before its chunk, above
      // it in one after; the batch of its chunk counts as one after, and
      // its equals in the chunks before are added
      const uint32_t thr = cb + kStep <= tc[g] ? lo[g] : hi[g];
      uint32_t q = 0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&cur[i][0]);
#pragma unroll
        for (int z = 0; z < 4 * Q; ++z) {
          if constexpr (F32) q += __uint_as_float(w[z]) >= __uint_as_float(thr);
          else q += ge_mask<TYPE>(w[z], thr);
        }
      }
      if (cb <= tc[g] && tc[g] < cb + kStep) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&cur[i][0]);
          if (cb + tid + i * kThreads < min(tc[g], c1)) {
#pragma unroll
            for (int z = 0; z < 4 * Q; ++z) {
              if constexpr (F32) q += __uint_as_float(w[z]) == xt[g];
              else q += ge_mask<TYPE>(w[z], lo[g]) & ~ge_mask<TYPE>(w[z], hi[g]);
            }
          }
        }
      }
      cnt[g] += q;
    }
  };
  int cb = c0;
  if constexpr (RING) {
    int slot = 0;
#pragma unroll 1
    for (; cb < c1; cb += kStep) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
      Batch cur;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) cur[i][0] = sm.u.ring[slot][i][tid];
      // into the slot before this one, whose batch the last turn has read
      copy(slot == 0 ? kRing - 1 : slot - 1, cb + (kRing - 1) * kStep);
      process(cur, cb);
      slot = slot == kRing - 1 ? 0 : slot + 1;
    }
  } else {
    Batch odd;
#pragma unroll 1
    while (cb < c1) {
      if (cb + kStep < c1) fetch(odd, cb + kStep);
      process(even, cb);
      cb += kStep;
      if (cb >= c1) break;
      if (cb + kStep < c1) fetch(even, cb + kStep);
      process(odd, cb);
      cb += kStep;
    }
  }

  if (edge_j >= 0) {
    sums.reach(edge_v, u);
    sums.add<true>(make_float2(edge_v, -INFINITY), uu);
  }
#pragma unroll
  for (int g = 0; g < NT; ++g) {
    if constexpr (!F32) {
      // cnt is the sum of masks: 65535 low - 65536 high counts, modulo 2^32
      const uint32_t low = (0u - cnt[g]) & 0xFFFFu;
      cnt[g] = low + (((65535u * low - cnt[g]) >> 16) & 0xFFFFu);
    }
    // the last batch's places outside the part hold -inf, which counts
    // before a target that is -inf itself
    if (xt[g] == -INFINITY && c0 < c1 && cb <= tc[g])
      for (int k = cb - kStep + tid; k < cb; k += kThreads) cnt[g] -= k >= c1 ? 8 : 0;
    if (edge_j >= 0) cnt[g] += edge_v > xt[g] || (edge_v == xt[g] && edge_j < tj[g]);
    cnt[g] += fix_g == g && fix_v == xt[g];
  }

  // join the block's sums in a fixed order
  float r = -sums.nr.x, S = sums.S.x + sums.S.y, A = sums.A.x + sums.A.y;
  join_warp(r, S, A);
  if (lane == 0) sm.r[warp] = r, sm.S[warp] = S, sm.A[warp] = A;
  if constexpr (NT > 0) {
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      const uint32_t s = __reduce_add_sync(0xFFFFFFFFu, cnt[g]);
      if (lane == 0) sm.cnt[warp][g] = static_cast<int>(s);
    }
  }
  const int n = a.top_n;
  float top_v = max_warp(fmaxf(best, edge_v));
  if (lane == 0) sm.best[warp].v = top_v;
  __syncthreads();
  if (warp == kWarps - 1) {
    // while the other warps begin the selection
    r = kUnset, S = 0.0f, A = 0.0f, top_v = -INFINITY;
    if (lane < kWarps) r = sm.r[lane], S = sm.S[lane], A = sm.A[lane], top_v = sm.best[lane].v;
    join_warp(r, S, A);
    top_v = max_warp(top_v);
    if (lane == 0) sm.mine.r = r, sm.mine.S = S, sm.mine.A = A, sm.mine.best = top_v;
    if (lane < NT) {
      int q = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) q += sm.cnt[w][lane];
      sm.mine.cnt[lane] = q;
    }
  }
  if (n > 0) select_top<TYPE, THREADS, RING>(row, sm, n, c0, c1, best, best_c, edge_v, edge_j);
  __syncthreads();

  // the parts meet in the first block
  Part* all = &sm.mine;
  if (split > 1) {
    constexpr int words = sizeof(Part) / 4;
    static_assert(words <= kSplitThreads && kMaxSplit * kMaxTop <= kSplitThreads, "one word, one token a thread");
    uint32_t* to = reinterpret_cast<uint32_t*>(cluster.map_shared_rank(&sm.parts[rank], 0));
    cluster.barrier_wait();  // the first block has started
    if (tid < words) to[tid] = reinterpret_cast<const uint32_t*>(&sm.mine)[tid];
    if (tid == 0) sm.ncand = 0;
    cluster.sync();
    if (rank != 0) return;
    all = sm.parts;
    if (n > 0) {
      // a token that n of the lists' tokens do not come after: the last of
      // the lists' c-th, with c parts = n or a little more; only those tokens
      // are ranked (searches of all lists for every token took 1 us more)
      const int c = (n + split - 1) / split - 1;
      Key cut = all[0].top[c];
#pragma unroll
      for (int q = 1; q < kMaxSplit; ++q) {
        const Key k = all[q < split ? q : 0].top[c];
        if (before(cut, k)) cut = k;
      }
      Picks<THREADS>& pk = sm.u.picks;
      if (tid < split * kMaxTop && tid % kMaxTop < n) {
        const Key k = all[tid / kMaxTop].top[tid % kMaxTop];
        if (k.id >= 0 && !before(cut, k)) pk.cand[atomicAdd(&sm.ncand, 1)] = k;
      }
      if (tid < kMaxTop) sm.mine.top[tid].v = -INFINITY, sm.mine.top[tid].id = -1;
      __syncthreads();
      place_keys<kWarps>(pk.cand, sm.ncand, n, [&](int place, int i) { sm.mine.top[place] = pk.cand[i]; });
      __syncthreads();
    }
  }
  r = kUnset, S = 0.0f, A = 0.0f, top_v = -INFINITY;
  if (lane < split) r = all[lane].r, S = all[lane].S, A = all[lane].A, top_v = all[lane].best;
  join_warp(r, S, A);
  top_v = max_warp(top_v);
  const bool empty = (S == 0.0f && top_v == -INFINITY) || top_v * a.scale == -INFINITY;
  // all probability on the largest logits: count them
  const bool flat = !empty && top_v > -INFINITY && top_v < INFINITY &&
                    (S == 0.0f || fabsf(top_v * u) >= kFar);
  bool bad = top_v == INFINITY || top_v * a.scale == INFINITY || (!flat && S != S);
  __syncthreads();
  if (flat) {
    int eq = 0, nan = 0;
    auto look = [&](float v) { eq += v == top_v, nan |= v != v; };
    if (edge_j >= 0) look(edge_v);
#pragma unroll 2
    for (int c = row.w0 + tid; c < row.w1; c += kThreads) {
      float v[8];
      row.load(c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) look(v[k]);
    }
    eq = __reduce_add_sync(0xFFFFFFFFu, eq);
    nan = __reduce_add_sync(0xFFFFFFFFu, nan);
    if (lane == 0) sm.cnt[warp][0] = eq, sm.cnt[warp][1] = nan;
    __syncthreads();
    eq = nan = 0;
    for (int w = 0; w < kWarps; ++w) eq += sm.cnt[w][0], nan += sm.cnt[w][1];
    S = static_cast<float>(eq);
    A = 0.0f;
    bad = bad || nan;
  }
  if (warp != 0) return;

  const float log2_s = log2f(S);
  const float lse = flat ? fmaf(top_v, a.scale, kLn2 * log2_s) : kLn2 * (r + log2_s);
  auto logprob = [&](float x) {
    if (bad) return NAN;
    if (empty || x * a.scale == -INFINITY) return -INFINITY;
    if (flat) return x == top_v ? -kLn2 * log2_s : (x - top_v) * a.scale - kLn2 * log2_s;
    const float d = fmaf(x, u, -r);
    return d == -INFINITY ? x * a.scale - lse : kLn2 * (d - log2_s);
  };
  if (lane == 0) {
    if (a.lse) a.lse[t] = bad ? NAN : empty ? -INFINITY : lse;
    if (a.entropy) a.entropy[t] = bad ? NAN : empty ? 0.0f : kLn2 * (log2_s - A / S);
  }
  if (lane < a.n_targets) {
    const int64_t i = t * a.n_targets + lane;
    const bool in = my_target >= 0;
    if (a.target_logprobs) a.target_logprobs[i] = in ? logprob(my_logit) : -INFINITY;
    if constexpr (NT > 0) {
      int q = 0;
      for (int w = 0; w < split; ++w) q += all[w].cnt[lane];
      if (a.target_ranks) a.target_ranks[i] = in ? q + 1 : 0;
    }
  }
  if (lane < n) {
    Key k = sm.mine.top[lane];
    if (k.id >= 0 && k.v * a.scale == -INFINITY) k.id = -1;
    if (a.top_ids) a.top_ids[t * n + lane] = k.id;
    if (a.top_logprobs) a.top_logprobs[t * n + lane] = k.id >= 0 ? logprob(k.v) : -INFINITY;
  }
}

template <int TYPE, int NT, int THREADS, bool RING>
cudaError_t launch(const moe_token_logprobs_args& a, int split, cudaStream_t st) {
  auto kernel = token_logprobs_kernel<TYPE, NT, THREADS, RING>;
  const int parts = THREADS == kSplitThreads ? split : 1;  // as the kernel has it
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * parts);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = sizeof(Smem<THREADS, RING>);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = parts;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cfg.dynamicSmemBytes > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, cfg.dynamicSmemBytes);
    if (e) return e;
  }
  return cudaLaunchKernelEx(&cfg, kernel, a, parts);
}

template <int TYPE, int THREADS, bool RING>
cudaError_t launch_nt(const moe_token_logprobs_args& a, int split, cudaStream_t st) {
  const int nt = a.target_ranks ? a.n_targets : 0;
  if (nt == 0) return launch<TYPE, 0, THREADS, RING>(a, split, st);
  if (nt == 1) return launch<TYPE, 1, THREADS, RING>(a, split, st);
  if (nt == 2) return launch<TYPE, 2, THREADS, RING>(a, split, st);
  if (nt <= 4) return launch<TYPE, 4, THREADS, RING>(a, split, st);
  return launch<TYPE, kMaxTargets, THREADS, RING>(a, split, st);
}

template <int TYPE>
cudaError_t launch_type(const moe_token_logprobs_args& a, int split, int sms, cudaStream_t st) {
  // Measured in graphs over inputs larger than the L2, bf16, one target, 5
  // alternatives where not said.
  // Blocks of 128 threads have shorter ends and leave an SM more rows to cover
  // them with, while a winning group, twice as long, costs more to read again:
  // 4096 rows of 4000 23.6 us against 44.3 with 256 threads, of 8192 29.6 / 44.9,
  // of 32000 53.8 / 67.5, of 50001 80.7 / 92.6, of 65536 98.3 / 97.0, of 131072
  // 206 / 174; 600 rows of 32000, a wave of the larger blocks, 12.7 / 13.9.
  // Copies through shared memory: 4096 rows of 131072 174 us against 189 into
  // registers, of 65536 97 / 109, of 65536 with 8 targets and 20 alternatives 235 /
  // 318, of 20000 (128 threads) 41.6 / 43.5, of 8192 28.5 / 29.6, of 4000 24.7 /
  // 23.6.
  // fp32 rows keep to registers: 2048 of 131072 without targets or alternatives
  // take 155 us, through shared memory 244 to 267 whatever the order of the
  // copies, which is not explained.
  const bool many = a.rows > 4 * sms, small = many && a.vocab <= kSmallVocab;
  if constexpr (TYPE == MOE_F32) {
    return small ? launch_nt<TYPE, 128, false>(a, split, st) : launch_nt<TYPE, kSplitThreads, false>(a, split, st);
  } else {
    if (small && a.vocab >= kRingVocab) return launch_nt<TYPE, 128, true>(a, split, st);
    if (small) return launch_nt<TYPE, 128, false>(a, split, st);
    if (many) return launch_nt<TYPE, kSplitThreads, true>(a, split, st);
    return launch_nt<TYPE, kSplitThreads, false>(a, split, st);
  }
}

}  // namespace
}  // namespace moe

extern "C" int moe_token_logprobs(const moe_token_logprobs_args* args, void* stream) {
  using namespace moe;
  if (!args) return reportf(MOE_ERR_ARG, "moe_token_logprobs: args is NULL");
  moe_token_logprobs_args a = *args;
  if (a.rows < 0) return reportf(MOE_ERR_ARG, "moe_token_logprobs: rows=%d is negative", a.rows);
  if (a.rows == 0) return MOE_OK;  // whatever the buffers: empty ones may be NULL
  if (a.rows > (1 << 27)) return reportf(MOE_ERR_ARG, "moe_token_logprobs: rows=%d is above 2^27", a.rows);
  if (a.vocab < 1 || a.vocab > (1 << 24))  // a thread's counts of a row fit 16 bits
    return reportf(MOE_ERR_ARG, "moe_token_logprobs: vocab=%d must be in [1, 2^24]", a.vocab);
  if (!elem_type_ok(a.logits_type))
    return reportf(MOE_ERR_ARG, "moe_token_logprobs: logits have an unknown type %d", a.logits_type);
  if (!a.logits) return reportf(MOE_ERR_ARG, "moe_token_logprobs: logits is NULL");
  if (a.ld_logits < a.vocab)
    return reportf(MOE_ERR_ARG, "moe_token_logprobs: logits have rows of %d values %lld apart", a.vocab,
                   static_cast<long long>(a.ld_logits));
  if (a.n_targets < 0 || a.n_targets > kMaxTargets)
    return reportf(MOE_ERR_ARG, "moe_token_logprobs: n_targets=%d must be in [0, %d]", a.n_targets, kMaxTargets);
  if (a.top_n < 0 || a.top_n > kMaxTop)
    return reportf(MOE_ERR_ARG, "moe_token_logprobs: top_n=%d must be in [0, %d]", a.top_n, kMaxTop);
  if (a.n_targets > 0 && !a.targets) return reportf(MOE_ERR_ARG, "moe_token_logprobs: targets is NULL");
  if (!(a.scale >= 5.4210109e-20f && a.scale <= 1.8446744e19f))
    return reportf(MOE_ERR_ARG, "moe_token_logprobs: scale must be in [2^-64, 2^64]");
  const uintptr_t words = reinterpret_cast<uintptr_t>(a.targets) | reinterpret_cast<uintptr_t>(a.target_logprobs) |
                          reinterpret_cast<uintptr_t>(a.target_ranks) | reinterpret_cast<uintptr_t>(a.entropy) |
                          reinterpret_cast<uintptr_t>(a.lse) | reinterpret_cast<uintptr_t>(a.top_ids) |
                          reinterpret_cast<uintptr_t>(a.top_logprobs);
  if (words % 4 || reinterpret_cast<uintptr_t>(a.logits) % elem_size(a.logits_type))
    return reportf(MOE_ERR_ALIGN, "moe_token_logprobs: a pointer is not aligned to its elements");

  if (!a.top_ids && !a.top_logprobs) a.top_n = 0;

  // Long rows, and few of them, are read in parts.  Parts of at least 32 KB of
  // rows of 128 KB, up to two blocks an SM: 152 rows of 131072 bf16 14.2 us in 2
  // parts, 15.2 whole (when rows' ends took longer: now 12.5 in 2); 152 rows of
  // 32000 (64 KB) would take 8.6 in 2 parts, 7.8 whole.  Parts down to 16 KB of
  // rows of 96 KB while they leave SMs idle: one row of 50001 bf16 7.8 us in 4
  // parts, 9.0 whole; 32 of them 8.0 / 9.3; but 150 of them 10.1 in 2, 9.5 whole.
  int dev = 0, sms = 0, split = 1;
  cudaError_t e = cudaGetDevice(&dev);
  if (!e) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e) return reportf(MOE_ERR_CUDA, "moe_token_logprobs: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  const int64_t row_bytes = static_cast<int64_t>(a.vocab) * elem_size(a.logits_type);
  for (; split < kMaxSplit; split *= 2) {
    const int64_t part = row_bytes / (2 * split), blocks = static_cast<int64_t>(a.rows) * split;
    const bool wide = row_bytes >= 4 * kPartBytes && part >= kPartBytes && blocks <= sms;
    const bool few = row_bytes >= 3 * kPartBytes && part >= kPartBytes / 2 && blocks <= sms / 2;
    if (!wide && !few) break;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.logits_type == MOE_BF16)
    e = launch_type<MOE_BF16>(a, split, sms, st);
  else if (a.logits_type == MOE_F16)
    e = launch_type<MOE_F16>(a, split, sms, st);
  else
    e = launch_type<MOE_F32>(a, split, sms, st);
  if (e != cudaSuccess)
    return reportf(MOE_ERR_CUDA, "moe_token_logprobs: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  return MOE_OK;
}
