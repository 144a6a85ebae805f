// cache.cu -- writing rows of keys and values into the paged cache and reading
// them back (include/moe_cache.h).
//
// Mathematics: per token and head of an e4m3 cache the scale is the smallest
// power of two s >= 2^-126 with max |x| <= 448 s, the codes are x / s rounded to
// nearest even: the division is exact, so is code * s.
//
// Bound: memory; each value is read once and written once.  A unit is one head
// of one row's keys or values, worked on by the fewest threads (a power of two)
// that hold 16 of them, so an e4m3 unit is stored in whole 16-byte pieces and
// its largest magnitude is a few shuffles away.  Which sequence a row belongs to
// is found by the warp: 32 starts are compared at a time.
#include <cuda_runtime.h>

#include "cache.cuh"

namespace moe {
int reportf(int code, const char* fmt, ...);

int check_cache(const char* name, const moe_kv_cache* cache, const moe_sequences* seqs, Seqs* q) {
  if (!cache || !seqs) return reportf(MOE_ERR_ARG, "%s: cache or seqs is NULL", name);
  const moe_kv_cache& c = *cache;
  const moe_sequences& s = *seqs;
  if (s.n_seqs < 0 || s.n_seqs > kMaxSeqs || s.rows < 0 || s.rows > kMaxSeqRows)
    return reportf(MOE_ERR_ARG, "%s: n_seqs=%d must be in [0, %d], rows=%d in [0, %d]", name, s.n_seqs, kMaxSeqs, s.rows,
                   kMaxSeqRows);
  if (c.type != MOE_BF16 && c.type != MOE_F16 && c.type != MOE_E4M3)
    return reportf(MOE_ERR_ARG, "%s: the cache has an unknown type %d", name, c.type);
  if (c.head_dim < 16 || c.head_dim > 256 || c.head_dim % 16)
    return reportf(MOE_ERR_ARG, "%s: head_dim=%d must be a multiple of 16 in [16, 256]", name, c.head_dim);
  if (c.kv_heads < 1 || c.kv_heads > 1024 || c.page_size < 1 || c.page_size > (1 << 20) || c.n_pages < 0)
    return reportf(MOE_ERR_ARG, "%s: kv_heads=%d must be in [1, 1024], page_size=%d in [1, 2^20], n_pages=%d not negative",
                   name, c.kv_heads, c.page_size, c.n_pages);
  const int per16 = c.type == MOE_E4M3 ? 16 : 8;
  if (c.page_stride < 0 || c.slot_stride < 0 || c.head_stride < 0 || c.page_stride % per16 || c.slot_stride % per16 ||
      c.head_stride % per16)
    return reportf(MOE_ERR_ARG, "%s: strides %lld, %lld and %lld must be multiples of %d, not negative", name,
                   static_cast<long long>(c.page_stride), static_cast<long long>(c.slot_stride),
                   static_cast<long long>(c.head_stride), per16);
  if (s.max_rows < 0) return reportf(MOE_ERR_ARG, "%s: max_rows=%d is negative", name, s.max_rows);
  if (s.n_seqs && s.rows) {
    if (s.table_width < 0 || s.ld_table < s.table_width)
      return reportf(MOE_ERR_ARG, "%s: table_width=%d must be in [0, ld_table=%lld]", name, s.table_width,
                     static_cast<long long>(s.ld_table));
    if (!s.starts || !s.kv_lens || (s.table_width && !s.page_table))
      return reportf(MOE_ERR_ARG, "%s: starts, kv_lens or page_table is NULL", name);
    if ((reinterpret_cast<uintptr_t>(s.starts) | reinterpret_cast<uintptr_t>(s.kv_lens) |
         reinterpret_cast<uintptr_t>(s.page_table)) % 4)
      return reportf(MOE_ERR_ALIGN, "%s: starts, kv_lens or page_table is misaligned", name);
    if (c.n_pages && (!c.k || !c.v)) return reportf(MOE_ERR_ARG, "%s: the cache's k or v is NULL", name);
    if ((reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) % 16)
      return reportf(MOE_ERR_ALIGN, "%s: the cache's k or v is not 16-byte aligned", name);
    if (c.type == MOE_E4M3) {
      if (c.n_pages && (!c.k_scale || !c.v_scale)) return reportf(MOE_ERR_ARG, "%s: k_scale or v_scale is NULL", name);
      if ((reinterpret_cast<uintptr_t>(c.k_scale) | reinterpret_cast<uintptr_t>(c.v_scale)) % 4)
        return reportf(MOE_ERR_ALIGN, "%s: k_scale or v_scale is misaligned", name);
      if (c.scale_page_stride < 0 || c.scale_slot_stride < 0 || c.scale_head_stride < 0)
        return reportf(MOE_ERR_ARG, "%s: a stride of the scales is negative", name);
    }
  }
  const int64_t cap = static_cast<int64_t>(s.table_width) * c.page_size;
  q->starts = s.starts, q->kv_lens = s.kv_lens, q->table = s.page_table, q->ld_table = s.ld_table;
  q->n = s.n_seqs, q->rows = s.rows, q->cap = static_cast<int32_t>(cap < kMaxPositions ? cap : kMaxPositions);
  q->page = divisor(static_cast<uint32_t>(c.page_size)), q->n_pages = c.n_pages;
  return MOE_OK;
}

namespace {

constexpr int kThreads = 256;

struct MoveArgs {
  moe_kv_cache c;
  Seqs q;
  void *k, *v;  // the rows' keys and values
  int64_t ld_k, ld_v;
  int type, tpu_log2, vec;  // threads of a unit; vec: rows on 16-byte (1) or 32-byte (2) boundaries
  Divisor heads;
};

// The last sequence that starts at or before row t, for the warp's first row
// (all lanes): the number of starts[1 ..] at or before it.
__device__ __forceinline__ int find_seq(const Seqs& q, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, span = q.n;  // the answer is in [lo, lo + span)
  while (span > 1) {
    const int step = (span + 31) / 32, i = lo + (lane + 1) * step;  // starts[i] <= t: the answer is i or more
    const bool past = i < lo + span && q.starts[i] <= t;
    const int c = __popc(__ballot_sync(0xFFFFFFFFu, past));
    span = min(step, lo + span - (lo + c * step));
    lo += c * step;
  }
  return lo;
}

__device__ __forceinline__ int next_seq(const Seqs& q, int s, int t) {
  while (s + 1 < q.n && q.starts[s + 1] <= t) ++s;
  return s;
}

// A thread's place: its row, head and first value; whether the row has one
// (in a sequence), and the cache's page and slot for it (-1: missing).
struct Place {
  int row, head, d, page, slot;
  bool in, held;
};

__device__ __forceinline__ Place place_of(const MoveArgs& a) {
  Place p;
  const uint32_t tpu = 1u << a.tpu_log2, unit = (blockIdx.x * kThreads + threadIdx.x) >> a.tpu_log2;
  p.row = static_cast<int>(divide(unit, a.heads));
  p.head = static_cast<int>(unit - p.row * a.heads.d);
  p.d = static_cast<int>(threadIdx.x & (tpu - 1)) * 16;
  const int warp_unit = (blockIdx.x * kThreads + (threadIdx.x & ~31u)) >> a.tpu_log2;
  const int first_row = static_cast<int>(divide(warp_unit, a.heads)), lane = threadIdx.x & 31;
  p.in = p.held = false, p.page = -1, p.slot = 0;
  Seq q = {0, 0, 0};
  int s = 0;
  if (a.q.n <= 32 && __all_sync(0xFFFFFFFFu, p.row == first_row)) {
    // few sequences, one row: a lane has a sequence, so one read instead of three in turn
    // (8192 rows of 8 heads of 128 17.0 -> 16.4 us, 32614 read back 41 -> 39)
    const Seq mine = lane < a.q.n ? load_seq(a.q, lane) : Seq{0x7FFFFFFF, 0, 0};
    const int start = lane < a.q.n ? a.q.starts[lane] : 0x7FFFFFFF;
    s = max(__popc(__ballot_sync(0xFFFFFFFFu, start <= p.row)) - 1, 0);
    q.first = __shfl_sync(0xFFFFFFFFu, mine.first, s), q.n = __shfl_sync(0xFFFFFFFFu, mine.n, s);
    q.len = __shfl_sync(0xFFFFFFFFu, mine.len, s);
  } else {
    const int s0 = find_seq(a.q, first_row);
    if (p.row < a.q.rows) {
      s = next_seq(a.q, s0, p.row);
      q = load_seq(a.q, s);
    }
  }
  if (p.row < a.q.rows && p.row >= q.first && p.row < q.first + q.n) {
    p.in = true;
    const int pos = q.len - q.n + (p.row - q.first);
    if (pos >= 0) p.page = page_of(a.q, s, pos, p.slot);
    p.held = p.page >= 0;
  }
  if (p.d >= a.c.head_dim) p.in = p.held = false;
  return p;
}

__device__ __forceinline__ int64_t cache_at(const moe_kv_cache& c, const Place& p) {
  return p.page * c.page_stride + p.slot * c.slot_stride + p.head * c.head_stride + p.d;
}
__device__ __forceinline__ int64_t scale_at(const moe_kv_cache& c, const Place& p) {
  return p.page * c.scale_page_stride + p.slot * c.scale_slot_stride + p.head * c.scale_head_stride;
}

// 16 values of a row, keys or values.
__device__ __forceinline__ int64_t row_at(const MoveArgs& a, int row, int head, int d, int64_t ld) {
  return row * ld + static_cast<int64_t>(head) * a.c.head_dim + d;
}

struct Sixteen {
  float x[16];
  __device__ __forceinline__ void load(const MoveArgs& a, const void* src, int64_t at) {
    if (a.vec == 2 && a.type != MOE_F32) {
      uint32_t w[8];
      load32(static_cast<const uint16_t*>(src) + at, w);
      float lo[8], hi[8];
      unpack8(make_uint4(w[0], w[1], w[2], w[3]), a.type, lo);
      unpack8(make_uint4(w[4], w[5], w[6], w[7]), a.type, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = lo[i], x[8 + i] = hi[i];
    } else if (a.vec) {
      float lo[8], hi[8];
      load8(src, a.type, at, lo);
      load8(src, a.type, at + 8, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = lo[i], x[8 + i] = hi[i];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = load_elem(src, a.type, at + i);
    }
  }
  __device__ __forceinline__ void store(const MoveArgs& a, void* dst, int64_t at) const {
    if (a.vec == 2 && a.type != MOE_F32) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack2(x[2 * i], x[2 * i + 1], a.type);
      store32(static_cast<uint16_t*>(dst) + at, w);
    } else if (a.vec) {
      store_half(dst, a.type, at, 0);
      store_half(dst, a.type, at + 8, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) store_elem(dst, a.type, at + i, x[i]);
    }
  }
  __device__ __forceinline__ void store_half(void* dst, int type, int64_t at, int from) const {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = from ? x[8 + i] : x[i];
    store8(dst, type, at, v);
  }
};

// blockIdx.y: 0 keys, 1 values.  What is written is read while the way to its
// slot is found, which takes three reads one after the other.
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const MoveArgs a) {
  const bool values = blockIdx.y != 0;
  const uint32_t unit = (blockIdx.x * kThreads + threadIdx.x) >> a.tpu_log2;
  const int row = static_cast<int>(divide(unit, a.heads)), head = static_cast<int>(unit - row * a.heads.d);
  const int d = static_cast<int>(threadIdx.x & ((1u << a.tpu_log2) - 1)) * 16;
  Sixteen s;
#pragma unroll
  for (int i = 0; i < 16; ++i) s.x[i] = 0.0f;
  if (row < a.q.rows && d < a.c.head_dim) s.load(a, values ? a.v : a.k, row_at(a, row, head, d, values ? a.ld_v : a.ld_k));
  const Place p = place_of(a);
  void* dst = values ? a.c.v : a.c.k;
  if (a.c.type != MOE_E4M3) {
    if (p.held) {
      const int64_t at = cache_at(a.c, p);
      s.store_half(dst, a.c.type, at, 0);
      s.store_half(dst, a.c.type, at + 8, 8);
    }
    return;
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(s.x[i]) & 0x7FFFFFFFu);
  for (int o = (1 << a.tpu_log2) >> 1; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (!p.held) return;
  float inv;
  const float scale = block_scale(m, inv);
  uint4 w = make_uint4(e4m3x4(s.x[0] * inv, s.x[1] * inv, s.x[2] * inv, s.x[3] * inv),
                       e4m3x4(s.x[4] * inv, s.x[5] * inv, s.x[6] * inv, s.x[7] * inv),
                       e4m3x4(s.x[8] * inv, s.x[9] * inv, s.x[10] * inv, s.x[11] * inv),
                       e4m3x4(s.x[12] * inv, s.x[13] * inv, s.x[14] * inv, s.x[15] * inv));
  if (inv == 0.0f) w = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  *reinterpret_cast<uint4*>(static_cast<uint8_t*>(dst) + cache_at(a.c, p)) = w;
  if (p.d == 0) (values ? a.c.v_scale : a.c.k_scale)[scale_at(a.c, p)] = scale;
}

// A thread has 16 keys and the 16 values beside them, which share the way to their slot.
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const MoveArgs a) {
  const Place p = place_of(a);
  if (!p.in) return;
  Sixteen v[2];
  if (p.held && a.c.type == MOE_E4M3) {
    uint4 w[2];
    float scale[2];
    const int64_t at = cache_at(a.c, p), sat = scale_at(a.c, p);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      w[kv] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv ? a.c.v : a.c.k) + at);
      scale[kv] = (kv ? a.c.v_scale : a.c.k_scale)[sat];
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t u[4] = {w[kv].x, w[kv].y, w[kv].z, w[kv].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __nv_fp8x2_storage_t two = static_cast<__nv_fp8x2_storage_t>(u[i / 2] >> (16 * (i & 1)));
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
        v[kv].x[2 * i] = f.x * scale[kv], v[kv].x[2 * i + 1] = f.y * scale[kv];
      }
    }
  } else if (p.held) {
    const int64_t at = cache_at(a.c, p);
    float lo[2][8], hi[2][8];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      load8(kv ? a.c.v : a.c.k, a.c.type, at, lo[kv]);
      load8(kv ? a.c.v : a.c.k, a.c.type, at + 8, hi[kv]);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[kv].x[i] = lo[kv][i], v[kv].x[8 + i] = hi[kv][i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[0].x[i] = v[1].x[i] = 0.0f;
  }
  v[0].store(a, a.k, row_at(a, p.row, p.head, p.d, a.ld_k));
  v[1].store(a, a.v, row_at(a, p.row, p.head, p.d, a.ld_v));
}

int move(const char* name, bool write, const moe_kv_cache* cache, const moe_sequences* seqs, void* k, int64_t ld_k, void* v,
         int64_t ld_v, int32_t type, void* stream) {
  MoveArgs a;
  const int rc = check_cache(name, cache, seqs, &a.q);
  if (rc) return rc;
  if (!elem_type_ok(type)) return reportf(MOE_ERR_ARG, "%s: the rows have an unknown type %d", name, type);
  if (seqs->rows == 0 || seqs->n_seqs == 0) return MOE_OK;
  if (write && (cache->n_pages == 0 || seqs->table_width == 0)) return MOE_OK;  // every page is missing
  if (!k || !v) return reportf(MOE_ERR_ARG, "%s: k or v is NULL", name);
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  if (ld_k < width || ld_v < width)
    return reportf(MOE_ERR_ARG, "%s: rows of %lld values are %lld and %lld apart", name, static_cast<long long>(width),
                   static_cast<long long>(ld_k), static_cast<long long>(ld_v));
  const int size = elem_size(type);
  if (reinterpret_cast<uintptr_t>(k) % size || reinterpret_cast<uintptr_t>(v) % size)
    return reportf(MOE_ERR_ALIGN, "%s: k or v is not aligned to its elements", name);
  a.c = *cache, a.k = k, a.v = v, a.ld_k = ld_k, a.ld_v = ld_v, a.type = type;
  a.tpu_log2 = 0;
  while ((16 << a.tpu_log2) < cache->head_dim) ++a.tpu_log2;
  const uintptr_t places = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | static_cast<uintptr_t>(ld_k * size) |
                           static_cast<uintptr_t>(ld_v * size);
  a.vec = places % 32 == 0 ? 2 : places % 16 == 0 ? 1 : 0;
  a.heads = divisor(static_cast<uint32_t>(cache->kv_heads));
  // threads are counted in 32 bits: up to 2^24 rows of 7 heads of 256, fewer than 2^17 of 1024
  const int64_t threads_row = static_cast<int64_t>(cache->kv_heads) << a.tpu_log2;
  const int64_t threads = threads_row * seqs->rows;
  if (threads > 0x7FFFFF00)
    return reportf(MOE_ERR_ARG, "%s: %d rows of %d heads of %d are too many for one call", name, seqs->rows, cache->kv_heads,
                   cache->head_dim);
  const unsigned grid = static_cast<unsigned>((threads + kThreads - 1) / kThreads);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (write)
    cache_write_kernel<<<dim3(grid, 2), kThreads, 0, st>>>(a);
  else
    cache_read_kernel<<<grid, kThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e) return reportf(MOE_ERR_CUDA, "%s: %s (%s)", name, cudaGetErrorString(e), cudaGetErrorName(e));
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int moe_cache_write(const moe_kv_cache* cache, const moe_sequences* seqs, const void* k, int64_t ld_k,
                               const void* v, int64_t ld_v, int32_t type, void* stream) {
  return moe::move("moe_cache_write", true, cache, seqs, const_cast<void*>(k), ld_k, const_cast<void*>(v), ld_v, type, stream);
}

extern "C" int moe_cache_read(const moe_kv_cache* cache, const moe_sequences* seqs, void* k, int64_t ld_k, void* v,
                              int64_t ld_v, int32_t type, void* stream) {
  return moe::move("moe_cache_read", false, cache, seqs, k, ld_k, v, ld_v, type, stream);
}
