// cache.cuh -- the paged key/value cache and the sequences of a call
// (include/moe_cache.h) as the kernels see them: where a position's slot lies,
// which sequence a row belongs to, and the host's checks of both.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/moe_cache.h"
#include "elem.cuh"

namespace moe {

constexpr int kMaxSeqs = 65536;
constexpr int kMaxSeqRows = 1 << 24;
constexpr int64_t kMaxPositions = 1 << 30;  // of a sequence

// Division of n < 2^31 by a divisor below 2^31: with s = ceil(log2 d) and
// m = ceil(2^(31 + s) / d) < 2^32, n * m / 2^(31 + s) exceeds n / d by less
// than n / 2^31 / d < 1 / d, so its floor is n / d's (Granlund and Montgomery).
struct Divisor {
  uint32_t m, s, d;
};

inline Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d), 31 + s, d};
}

__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& d) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * d.m) >> d.s);
}

struct Seqs {
  const int32_t *starts, *kv_lens, *table;
  int64_t ld_table;
  int32_t n, rows, cap;  // cap: positions that the page table can hold
  Divisor page;          // slots of a page
  int32_t n_pages;
};

// One sequence: its first row, its rows, and its length.
struct Seq {
  int first, n, len;
};

// `falls`: the sequence ends before it starts, which leaves it without rows.
__device__ __forceinline__ Seq load_seq(const Seqs& q, int s, bool& falls) {
  Seq r;
  r.first = min(max(q.starts[s], 0), q.rows);
  const int end = q.starts[s + 1];
  falls = end < r.first && r.first > 0;  // cut to [0, rows] too
  r.n = min(max(end, r.first), q.rows) - r.first;
  r.len = min(max(q.kv_lens[s], 0), q.cap);
  return r;
}
__device__ __forceinline__ Seq load_seq(const Seqs& q, int s) {
  bool falls;
  return load_seq(q, s, falls);
}

// The page of a position in [0, cap) and the slot in it; -1 for a missing page.
__device__ __forceinline__ int page_of(const Seqs& q, int s, int pos, int& slot) {
  const uint32_t i = divide(static_cast<uint32_t>(pos), q.page);
  slot = pos - static_cast<int>(i * q.page.d);
  const int page = q.table[s * q.ld_table + i];
  return page >= 0 && page < q.n_pages ? page : -1;
}

// Checks shared by the calls; fills `q`.  MOE_OK or an error, reported.
int check_cache(const char* name, const moe_kv_cache* cache, const moe_sequences* seqs, Seqs* q);

}  // namespace moe
