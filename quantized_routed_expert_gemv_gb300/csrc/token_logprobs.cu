// token_logprobs.cu -- log probabilities, ranks, entropy and top tokens of
// rows of logits (moe_token_logprobs), in one pass over the logits.
//
// Mathematics, with u = scale * log2(e) and a reference R near the row's
// maximum:
//     S = sum_v 2^(u (l_v - R)),  A = sum_v u (l_v - R) 2^(u (l_v - R))
//     lse = scale R + ln S,  entropy = ln S - ln 2 * A / S,
//     logprob_t = scale (l_t - R) - ln S.
// Every thread keeps its own (R, S, A) and moves R only when a logit lies
// more than 2^kRefSlack above it, so the usual step has no rescaling; S, A
// and the differences stay in fp32.  Differences are clamped at -200 (in
// powers of two), where 2^d is 0, so -inf and the type's lowest value add 0
// to A instead of 0 * -inf.
//
// Top tokens: a thread's running maximum (and the chunk it was first seen
// in) is the best of the group of tokens that thread visited.  Any token of
// the row's top n lies in one of the n groups whose best come first, since
// the best of every group that precedes its own group's precedes it too.  So
// the pass keeps one value per thread, and afterwards only the n winning
// groups are read again (from cache) for tokens that do not come after the
// n-th best.
//
// A row is read by one block, or by a cluster of up to 8 blocks, each a
// contiguous part, when there are too few rows for the SMs; the parts are
// joined through distributed shared memory in rank order, so results do not
// depend on timing.
#include <cmath>
#include <cstdint>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "elem.cuh"

namespace moe {
int reportf(int code, const char* fmt, ...);

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kMaxTargets = 8;
constexpr int kMaxSplit = 8;
constexpr int kCand = 1024;            // candidate buffer of the top selection
constexpr float kRefSlack = 80.0f;     // powers of two a logit may lie above the reference
constexpr float kLn2 = 0.6931471805599453f;

struct Key {  // order: value descending, id ascending; id < 0: none
  float v;
  int id;
};

__device__ __forceinline__ bool before(float av, int ai, float bv, int bi) {
  return av > bv || (av == bv && ai < bi);
}

// What one block knows of its part of a row, read by the cluster's first
// block.
struct Part {
  float R, S, A;
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

// Smallest float above v (v itself for NaN and +inf -> NaN): x > v iff x >= next_up(v).
__device__ __forceinline__ float next_up(float v) {
  const uint32_t u = __float_as_uint(v);
  if (v == 0.0f) return __uint_as_float(1u);
  return __uint_as_float(v > 0.0f ? u + 1 : u - 1);
}

// The row's logits as chunks of 8 on a grid of 16-byte aligned addresses:
// chunk c holds elements [8 c - off, 8 c - off + 8) of the row.  Elements
// outside the row read as -inf.
template <int TYPE>
struct Row {
  const void* p;
  int off, vocab, chunks;
  __device__ __forceinline__ Row(const moe_token_logprobs_args& a, int64_t t) {
    constexpr int ES = TYPE == MOE_F32 ? 4 : 2;
    p = static_cast<const char*>(a.logits) + t * a.ld_logits * ES;
    off = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / ES);
    vocab = a.vocab;
    chunks = static_cast<int>((static_cast<int64_t>(vocab) + off + 7) / 8);
  }
  __device__ __forceinline__ bool whole(int c) const { return 8 * c >= off && vocab - 8 >= 8 * c - off; }
  __device__ __forceinline__ void load(int c, float (&v)[8]) const {
    const int j = 8 * c - off;
    if (whole(c)) {
      load8(p, TYPE, j, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = j + i >= 0 && j + i < vocab ? load_elem(p, TYPE, j + i) : -INFINITY;
    }
  }
};

__device__ __forceinline__ void merge(float& R, float& S, float& A, float r, float s, float a, float u) {
  if (s == 0.0f) return;
  if (S == 0.0f) {
    R = r, S = s, A = a;
    return;
  }
  const float m = fmaxf(R, r);
  const float d0 = max_nan((R - m) * u, -1e4f), d1 = max_nan((r - m) * u, -1e4f);
  const float e0 = exp2f(d0), e1 = exp2f(d1);
  A = (A + S * d0) * e0 + (a + s * d1) * e1;
  S = S * e0 + s * e1;
  R = m;
}

// One warp: the n first keys of the 32 * PER keys its lanes hold, in order,
// to out[0..n).
template <int PER>
__device__ __forceinline__ void warp_select(Key (&k)[PER], int n, Key* out) {
  const int lane = threadIdx.x & 31;
  for (int r = 0; r < n; ++r) {
    Key b = {-INFINITY, -1};
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (k[i].id >= 0 && (b.id < 0 || before(k[i].v, k[i].id, b.v, b.id))) b = k[i];
    Key w = b;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float v = __shfl_xor_sync(0xFFFFFFFFu, w.v, o);
      const int id = __shfl_xor_sync(0xFFFFFFFFu, w.id, o);
      if (id >= 0 && (w.id < 0 || before(v, id, w.v, w.id))) w.v = v, w.id = id;
    }
    if (lane == 0) out[r] = w;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (w.id >= 0 && k[i].id == w.id) k[i].id = -1;
  }
}

struct Smem {
  Key group[kThreads];   // each thread's first-ranked token
  int owner[kMaxTop];    // threads whose groups win
  Key sel[kMaxTop];
  Key cand[kCand];
  int ncand;
  Key last, best[kWarps];
  float R[kWarps], S[kWarps], A[kWarps];
  int cnt[kWarps][kMaxTargets];
  Part part;
};

// NT: number of targets whose ranks are counted, rounded up to 0, 1 or 8.
template <int TYPE, int NT>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const moe_token_logprobs_args a, int split) {
  __shared__ Smem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = split > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int64_t t = blockIdx.x / split;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Row<TYPE> row(a, t);
  const float u = a.scale * 1.4426950408889634f;
  const int per = (row.chunks + split - 1) / split;
  const int c0 = rank * per, c1 = min(row.chunks, c0 + per);

  float xt[NT > 0 ? NT : 1];
  int ct[NT > 0 ? NT : 1], it[NT > 0 ? NT : 1], cnt[NT > 0 ? NT : 1];
  if constexpr (NT > 0) {
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      it[g] = g < a.n_targets ? a.targets[t * a.n_targets + g] : -1;
      const bool in = it[g] >= 0 && it[g] < a.vocab;
      xt[g] = in ? load_elem(row.p, TYPE, it[g]) : NAN;
      ct[g] = in ? (it[g] + row.off) / 8 : -1;
      cnt[g] = 0;
    }
  }

  // the pass
  float R = -3.402823466e38f, S = 0.0f, A = 0.0f, best = -INFINITY;
  int best_c = -1;
  for (int c = c0 + tid; c < c1; c += kThreads) {
    float v[8];
    row.load(c, v);
    float m = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, v[i]);
    if (m > best) best = m, best_c = c;
    if ((m - R) * u > kRefSlack) {
      const float d = max_nan((R - m) * u, -1e4f), e = exp2f(d);
      A = (A + S * d) * e;
      S *= e;
      R = m;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = max_nan((v[i] - R) * u, -200.0f);
      const float e = ex2(d);
      S += e;
      A = fmaf(e, d, A);
    }
    if constexpr (NT > 0) {
      const bool whole = row.whole(c);
#pragma unroll
      for (int g = 0; g < NT; ++g) {
        if (whole && c != ct[g]) {
          const float thr = c < ct[g] ? xt[g] : next_up(xt[g]);
#pragma unroll
          for (int i = 0; i < 8; ++i) cnt[g] += v[i] >= thr;
        } else {
          const int j = 8 * c - row.off;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            cnt[g] += j + i >= 0 && j + i < a.vocab && (v[i] > xt[g] || (v[i] == xt[g] && j + i < it[g]));
        }
      }
    }
  }

  // join the block's sums in a fixed order
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float r = __shfl_down_sync(0xFFFFFFFFu, R, o), s = __shfl_down_sync(0xFFFFFFFFu, S, o),
                b = __shfl_down_sync(0xFFFFFFFFu, A, o);
    merge(R, S, A, r, s, b, u);
  }
  if (lane == 0) sm.R[warp] = R, sm.S[warp] = S, sm.A[warp] = A;
  if constexpr (NT > 0) {
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      const int s = __reduce_add_sync(0xFFFFFFFFu, cnt[g]);
      if (lane == 0) sm.cnt[warp][g] = s;
    }
  }
  const int n = a.top_n;
  if (n > 0) {
    // the id of the thread's best: the first place of that value in its chunk
    int id = -1;
    if (best_c >= 0) {
      float v[8];
      row.load(best_c, v);
      const int j = 8 * best_c - row.off;
#pragma unroll
      for (int i = 7; i >= 0; --i)
        if (v[i] == best) id = j + i;
    }
    sm.group[tid].v = best, sm.group[tid].id = id;
  }
  if (tid == 0) sm.ncand = 0;
  __syncthreads();
  if (warp == 0) {
    float r = -3.402823466e38f, s = 0.0f, b = 0.0f;
    if (lane < kWarps) r = sm.R[lane], s = sm.S[lane], b = sm.A[lane];
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) {
      const float r2 = __shfl_down_sync(0xFFFFFFFFu, r, o), s2 = __shfl_down_sync(0xFFFFFFFFu, s, o),
                  b2 = __shfl_down_sync(0xFFFFFFFFu, b, o);
      merge(r, s, b, r2, s2, b2, u);
    }
    if (lane == 0) sm.part.R = r, sm.part.S = s, sm.part.A = b;
    if (lane < NT) {
      int q = 0;
      for (int w = 0; w < kWarps; ++w) q += sm.cnt[w][lane];
      sm.part.cnt[lane] = q;
    }
  }
  if (n > 0) {
    if (warp == 0) {
      Key k[kWarps];
#pragma unroll
      for (int i = 0; i < kWarps; ++i) k[i] = sm.group[32 * i + lane];
      warp_select<kWarps>(k, n, sm.sel);
    }
    __syncthreads();
    if (tid < n) sm.owner[tid] = -1;
    __syncthreads();
    {
      const Key mine = sm.group[tid];
      if (mine.id >= 0)
        for (int r = 0; r < n; ++r)
          if (sm.sel[r].id == mine.id) sm.owner[r] = tid;
    }
    __syncthreads();
    // the winning groups' tokens that do not come after the n-th group's best
    const Key thr = sm.sel[n - 1];
    for (int r = warp; r < n; r += kWarps) {
      const int o = sm.owner[r];
      if (o < 0) continue;
      for (int c = c0 + o + lane * kThreads; c < c1; c += 32 * kThreads) {
        float v[8];
        row.load(c, v);
        const int j = 8 * c - row.off;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (v[i] > -INFINITY && (thr.id < 0 || !before(thr.v, thr.id, v[i], j + i))) {
            const int s = atomicAdd(&sm.ncand, 1);
            if (s < kCand) sm.cand[s].v = v[i], sm.cand[s].id = j + i;
          }
        }
      }
    }
    __syncthreads();
    const int m = sm.ncand;
    if (m <= kCand) {
      // a candidate's place is the number of candidates before it
      for (int i = tid; i < n; i += kThreads) sm.part.top[i].v = -INFINITY, sm.part.top[i].id = -1;
      __syncthreads();
      for (int i = tid; i < m; i += kThreads) {
        const Key k = sm.cand[i];
        int place = 0;
        for (int q = 0; q < m; ++q) place += before(sm.cand[q].v, sm.cand[q].id, k.v, k.id);
        if (place < n) sm.part.top[place] = k;
      }
    } else {
      // many tokens of few groups: one round over the winning groups per place
      if (tid == 0) sm.last.v = INFINITY, sm.last.id = -1;
      __syncthreads();
      for (int r = 0; r < n; ++r) {
        const Key last = sm.last;
        Key b = {-INFINITY, -1};
        for (int q = warp; q < n; q += kWarps) {
          const int o = sm.owner[q];
          if (o < 0) continue;
          for (int c = c0 + o + lane * kThreads; c < c1; c += 32 * kThreads) {
            float v[8];
            row.load(c, v);
            const int j = 8 * c - row.off;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (v[i] > -INFINITY && before(last.v, last.id, v[i], j + i) &&
                  (b.id < 0 || before(v[i], j + i, b.v, b.id)))
                b.v = v[i], b.id = j + i;
          }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const float v = __shfl_xor_sync(0xFFFFFFFFu, b.v, o);
          const int id = __shfl_xor_sync(0xFFFFFFFFu, b.id, o);
          if (id >= 0 && (b.id < 0 || before(v, id, b.v, b.id))) b.v = v, b.id = id;
        }
        if (lane == 0) sm.best[warp] = b;
        __syncthreads();
        if (tid == 0) {
          Key w = {-INFINITY, -1};
          for (int q = 0; q < kWarps; ++q)
            if (sm.best[q].id >= 0 && (w.id < 0 || before(sm.best[q].v, sm.best[q].id, w.v, w.id))) w = sm.best[q];
          sm.part.top[r] = w;
          if (w.id >= 0) sm.last = w;
        }
        __syncthreads();
      }
    }
  }
  __syncthreads();

  // join the parts of the row
  if (split > 1) {
    cluster.sync();
    if (rank == 0 && warp == 0) {
      float r = sm.part.R, s = sm.part.S, b = sm.part.A;
      for (int q = 1; q < split; ++q) {
        const Part* o = cluster.map_shared_rank(&sm.part, q);
        merge(r, s, b, o->R, o->S, o->A, u);
      }
      int q_cnt = 0;
      if (lane < NT)
        for (int q = 0; q < split; ++q) q_cnt += cluster.map_shared_rank(&sm.part, q)->cnt[lane];
      Key k[kMaxSplit];
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q) {
        k[q].v = -INFINITY, k[q].id = -1;
        if (q < split && lane < n) k[q] = cluster.map_shared_rank(&sm.part, q)->top[lane];
      }
      __syncwarp();
      if (lane == 0) sm.part.R = r, sm.part.S = s, sm.part.A = b;
      if (lane < NT) sm.part.cnt[lane] = q_cnt;
      warp_select<kMaxSplit>(k, n, sm.part.top);
      __syncwarp();
    }
    cluster.sync();
    if (rank != 0) return;
  }

  if (warp != 0) return;
  R = sm.part.R, S = sm.part.S, A = sm.part.A;
  const float ln_s = logf(S);
  // no probability anywhere: only -inf, or logits that overflow to it
  const bool empty = S == 0.0f || R * a.scale == -INFINITY;
  const bool bad = S != S || R == INFINITY;
  auto logprob = [&](float x) {
    if (bad) return NAN;
    return empty || x * a.scale == -INFINITY ? -INFINITY : (x - R) * a.scale - ln_s;
  };
  if (lane == 0) {
    if (a.lse) a.lse[t] = bad ? NAN : empty ? -INFINITY : fmaf(R, a.scale, ln_s);
    if (a.entropy) a.entropy[t] = bad ? NAN : empty ? 0.0f : ln_s - kLn2 * (A / S);
  }
  if (lane < a.n_targets) {
    const int64_t i = t * a.n_targets + lane;
    const int id = a.targets[i];
    const bool in = id >= 0 && id < a.vocab;
    if (a.target_logprobs) a.target_logprobs[i] = in ? logprob(load_elem(row.p, TYPE, id)) : -INFINITY;
    if constexpr (NT > 0) {
      if (a.target_ranks) a.target_ranks[i] = in ? sm.part.cnt[lane] + 1 : 0;
    }
  }
  if (lane < n) {
    Key k = sm.part.top[lane];
    if (k.id >= 0 && k.v * a.scale == -INFINITY) k.id = -1;
    if (a.top_ids) a.top_ids[t * n + lane] = k.id;
    if (a.top_logprobs) a.top_logprobs[t * n + lane] = k.id >= 0 ? logprob(k.v) : -INFINITY;
  }
}

template <int TYPE>
cudaError_t launch_type(const moe_token_logprobs_args& a, int split, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * split);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = split;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const int nt = a.target_ranks ? a.n_targets : 0;
  if (nt == 0) return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<TYPE, 0>, a, split);
  if (nt == 1) return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<TYPE, 1>, a, split);
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<TYPE, kMaxTargets>, a, split);
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
  if (a.vocab < 1 || a.vocab > (1 << 30))
    return reportf(MOE_ERR_ARG, "moe_token_logprobs: vocab=%d must be in [1, 2^30]", a.vocab);
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
  if (!(a.scale > 0.0f) || std::isinf(a.scale))
    return reportf(MOE_ERR_ARG, "moe_token_logprobs: scale must be positive and finite");
  const uintptr_t words = reinterpret_cast<uintptr_t>(a.targets) | reinterpret_cast<uintptr_t>(a.target_logprobs) |
                          reinterpret_cast<uintptr_t>(a.target_ranks) | reinterpret_cast<uintptr_t>(a.entropy) |
                          reinterpret_cast<uintptr_t>(a.lse) | reinterpret_cast<uintptr_t>(a.top_ids) |
                          reinterpret_cast<uintptr_t>(a.top_logprobs);
  if (words % 4 || reinterpret_cast<uintptr_t>(a.logits) % elem_size(a.logits_type))
    return reportf(MOE_ERR_ALIGN, "moe_token_logprobs: a pointer is not aligned to its elements");

  if (!a.top_ids && !a.top_logprobs) a.top_n = 0;

  // Few rows: enough blocks for the SMs, while a part keeps some work.
  int split = 1;
  while (split < kMaxSplit && a.rows * split < 152 && a.vocab / split >= 8 * kThreads) split *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.logits_type == MOE_BF16)
    e = launch_type<MOE_BF16>(a, split, st);
  else if (a.logits_type == MOE_F16)
    e = launch_type<MOE_F16>(a, split, st);
  else
    e = launch_type<MOE_F32>(a, split, st);
  if (e != cudaSuccess)
    return reportf(MOE_ERR_CUDA, "moe_token_logprobs: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  return MOE_OK;
}
