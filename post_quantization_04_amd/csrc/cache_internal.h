// Device-side view of the 8-bit key/value cache, shared by its kernels (gfx950).
#pragma once

#include "kq_internal.h"

namespace kq {

struct SeqArgs {
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* q_start;
  int32_t max_pages;
  int32_t max_q;
  int32_t page_log2;
  int32_t rows;      // rows of the call (< 2^31)
  int64_t pages;
  int32_t* info;
};

inline SeqArgs seq_args(const kq_cache& c, const kq_cache_batch& b, int64_t rows, int32_t* info) {
  SeqArgs s;
  s.table = b.table;
  s.seq_lens = b.seq_lens;
  s.q_start = b.q_start;
  s.max_pages = b.max_pages;
  s.max_q = b.max_q;
  s.page_log2 = __builtin_ctz(c.page);
  s.rows = static_cast<int32_t>(rows);
  s.pages = c.pages;
  s.info = info;
  return s;
}

__device__ __forceinline__ void report(int32_t* info, int bit) {
  if (info) atomicOr(info, bit);
}

// Sequence b with every bound enforced: rows [row0, row0 + n), len tokens in the cache.
struct Seq {
  int row0, n, len;
};

__device__ __forceinline__ Seq sequence(const SeqArgs& a, int b, bool tell) {
  Seq s;
  const int r0 = a.q_start[b], r1 = a.q_start[b + 1], len = a.seq_lens[b];
  const int cap = a.max_pages << a.page_log2;
  s.row0 = min(max(r0, 0), a.rows);
  const int end = min(max(r1, s.row0), a.rows);
  s.n = min(end - s.row0, a.max_q);
  s.len = min(max(len, 0), cap);
  if (tell) {
    if (s.row0 != r0 || end != r1 || end - s.row0 != s.n) report(a.info, KQ_INFO_ROWS);
    if (s.len != len) report(a.info, KQ_INFO_LENGTH);
  }
  return s;
}

// Entry of the table for position p of sequence b, and whether it is a page.
__device__ __forceinline__ int table_entry(const SeqArgs& a, int b, int p) {
  return a.table[int64_t(b) * a.max_pages + (p >> a.page_log2)];
}

__device__ __forceinline__ bool is_page(const SeqArgs& a, int id) { return uint32_t(id) < uint64_t(a.pages); }

// Page of position p of sequence b; -1 (and told) when the table's entry is not a page.
__device__ __forceinline__ int page_of(const SeqArgs& a, int b, int p) {
  const int id = table_entry(a, b, p);
  if (is_page(a, id)) return id;
  report(a.info, KQ_INFO_PAGE);
  return -1;
}

// Two floats to bf16, the first in the low half (to nearest even; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float floatx2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{a, b}), bf16x2));
}

}  // namespace kq
