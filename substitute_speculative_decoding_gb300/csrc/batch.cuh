// Batches of sequences over one paged cache: what the batched kernels share.
#pragma once
#include "common.cuh"

namespace sub {

// A sub_batch and the page table of the cache it runs on, on the device.
struct SeqTable {
  const int32_t* start;   // [n_seqs + 1]
  const int32_t* pos;     // [n_seqs]
  const int32_t* pages;   // [n_seqs][width]
  int n_seqs, n_rows;
  int width;              // page-table entries per sequence
  int page_size, n_pages;
  int64_t capacity;
};

// Pool addressing: element offset of row (page, head, place) in units of one row
// of head_dim values: ((layer * n_pages + page) * n_heads_kv + head) * page_size + place.
__device__ __forceinline__ int64_t pool_row(const SeqTable& t, int layer, int n_heads_kv, int page,
                                            int head, int place) {
  return (((int64_t)layer * t.n_pages + page) * n_heads_kv + head) * t.page_size + place;
}

// (Plain reads, kept by L1: no kernel of this library, which could still be running when
// the next one starts, writes the tables.  Through L2, 8403 rows took half as long again
// to be written and read.)
// First and one past the last row of sequence b, clamped into the row tensors.
__device__ __forceinline__ int seq_first(const SeqTable& t, int b) {
  return min(max(t.start[b], 0), t.n_rows);
}
__device__ __forceinline__ int seq_rows(const SeqTable& t, int b) {
  return max(0, min(max(t.start[b + 1], 0), t.n_rows) - seq_first(t, b));
}

// The sequence of a row (-1: none), by one warp together: the number of
// entries of start[1..n_seqs] at or below the row, found in two rounds of 32
// loads (a bisection would take ten dependent ones).
__device__ __forceinline__ int row_seq(const SeqTable& t, int row, int lane) {
  static_assert(SUB_MAX_SEQS <= 1024, "two rounds of 32");
  const int n = t.n_seqs;
  int groups = 0;
  if (n > 32) {   // entries 32, 64, ..: how many whole groups of 32 lie at or below the row
    const int e = (lane + 1) * 32;
    groups = __popc(__ballot_sync(~0u, e <= n && t.start[min(e, n)] <= row));
  }
  const int f = groups * 32 + lane + 1;
  const int b = groups * 32 + __popc(__ballot_sync(~0u, f <= n && t.start[min(f, n)] <= row));
  return b < n && t.start[0] <= row ? b : -1;
}

// Page of a position of sequence b, or -1.
__device__ __forceinline__ int page_of(const SeqTable& t, int b, int64_t p) {
  if (p < 0 || p >= t.capacity) return -1;
  const int page = t.pages[(int64_t)b * t.width + (uint32_t)p / (uint32_t)t.page_size];
  return page >= 0 && page < t.n_pages ? page : -1;
}

template <class Cache>
inline int32_t make_seq_table(const Cache* kv, int32_t layer, const sub_batch* batch,
                              SeqTable* t) {
  SUB_CHECK_ARG(kv && batch && kv->k && kv->v && kv->page_table && batch->start && batch->pos,
                "null pointer");
  SUB_CHECK_ARG(kv->head_dim == 64 || kv->head_dim == 128, "head_dim must be 64 or 128");
  SUB_CHECK_ARG(kv->n_heads_kv >= 1 && kv->n_heads_kv <= 65535, "n_heads_kv out of range");
  SUB_CHECK_ARG(kv->page_size > 0 && kv->page_size % 16 == 0, "page_size % 16 != 0");
  SUB_CHECK_ARG(kv->n_pages >= 1 && kv->capacity >= 1 && kv->capacity <= (1ll << 31) - 65536,
                "bad cache sizes");
  SUB_CHECK_ARG(layer >= 0 && layer < kv->n_layers, "layer out of range");
  SUB_CHECK_ARG(batch->n_seqs >= 1 && batch->n_seqs <= SUB_MAX_SEQS,
                "n_seqs must be in [1, SUB_MAX_SEQS]");
  SUB_CHECK_ARG(batch->n_rows >= 0 && batch->n_rows <= (1 << 24), "n_rows out of range");
  SUB_CHECK_ARG(batch->max_keys >= 0, "max_keys must be >= 0");
  SUB_CHECK_ARG(aligned16(kv->k) && aligned16(kv->v), "the cache must be 16-byte aligned");
  t->start = batch->start;
  t->pos = batch->pos;
  t->pages = kv->page_table;
  t->n_seqs = batch->n_seqs;
  t->n_rows = batch->n_rows;
  t->width = (int)cdiv(kv->capacity, kv->page_size);
  t->page_size = kv->page_size;
  t->n_pages = kv->n_pages;
  t->capacity = kv->capacity;
  return SUB_OK;
}

inline int32_t check_scales(const sub_kv8_cache* kv) {
  SUB_CHECK_ARG(kv && kv->k_scale && kv->v_scale, "null pointer");
  SUB_CHECK_ARG(aligned16(kv->k_scale) && aligned16(kv->v_scale), "the scales must be 16-byte aligned");
  return SUB_OK;
}

}  // namespace sub
