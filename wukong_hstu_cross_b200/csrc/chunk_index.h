// chunk_index.h — where the rows of a batch of sequences are in the paged cache, and the scale of a quantised
// row: index and bit arithmetic alone, so that the same lines compile for the host, where they are tested.
#pragma once

#include <stdint.h>
#include <string.h>

#ifdef __CUDACC__
#define WHALE_HD __host__ __device__
#else
#define WHALE_HD
#endif

namespace whale {

constexpr int kScaleLo = -100, kScaleHi = 119;

// One batch of sequences and the cache behind them, as the kernels see them. Row i of the n_b rows of
// sequence b (rows [offsets[b], offsets[b+1]) of the packed tensor) is at position lengths[b] - n_b + i.
struct ChunkView {
  const int* offsets;
  const int* lengths;
  const int* table;  // [B, table_stride] page of each page_size positions
  int table_stride, B;
  int page_shift;    // log2(page_size)
  int n_pages, planes, kv_heads;
  long long total;   // rows of the packed tensor
  long long capacity;  // positions a sequence can have: min(max_length, table_stride << page_shift)
};

WHALE_HD inline int chunk_off(const ChunkView& c, int b) {
  const long long o = c.offsets[b];
  return (int)(o < 0 ? 0 : (o > c.total ? c.total : o));
}

// Largest b with offsets[b] <= row (offsets ascend): sequences without rows are passed over.
WHALE_HD inline int chunk_seq(const ChunkView& c, long long row) {
  int lo = 0, hi = c.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.offsets[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Row of the cache's first plane and head, in units of rows: ((page * planes + plane) * heads + head) *
// page_size + slot; -1 if the row is in no page (a position or page outside the cache).
WHALE_HD inline long long page_row(const ChunkView& c, int page, long long pos) {
  if ((unsigned)page >= (unsigned)c.n_pages) return -1;
  return (((long long)page * c.planes * c.kv_heads) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}
WHALE_HD inline long long cache_row(const ChunkView& c, int b, long long pos) {
  if (pos < 0 || pos >= c.capacity) return -1;
  return page_row(c, c.table[(long long)b * c.table_stride + (pos >> c.page_shift)], pos);
}

// Whether slice `slice` of `slices` left an item of several slices to join (at most bm rows, from row0 on of a sequence
// that begins at first_row; `parts` partials, the first in `slot`), with every index that the join forms in
// range: partials below 2 * slices, rows below total, heads below kv_heads * group.
WHALE_HD inline bool cut_valid(const ChunkView& c, int group, int bm, int slices, int slice, int first_row, int row0,
                               int n_rows, int head0, int parts, int slot) {
  return parts > 1 && parts <= slices - slice && (slot >> 1) == slice && n_rows > 0 && n_rows <= bm && first_row >= 0 &&
         row0 >= 0 && (long long)first_row + ((long long)row0 + n_rows - 1) / group < c.total && head0 >= 0 &&
         head0 <= c.kv_heads * group - group;
}

// The scale's exponent of a row whose largest magnitude is amax (finite or infinite, no NaN).
WHALE_HD inline int scale_exponent(float amax) {
  uint32_t u;
  memcpy(&u, &amax, 4);
  // amax = 1.m * 2^E, 448 = 1.75 * 2^8: e = E - 8, one more where 1.m > 1.75
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < kScaleLo ? kScaleLo : (e > kScaleHi ? kScaleHi : e);
  return u == 0u ? 0 : e;
}

}  // namespace whale
