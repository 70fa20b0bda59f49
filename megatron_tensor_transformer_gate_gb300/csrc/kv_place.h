// kv_place.h — which token a row is and which page holds it (see tp_kv_cache
// in tp.h).  Host and device code, so that tables and lengths that are wrong
// are tested without a GPU: whatever they hold, only table entries
// [seq][0, table_cols) with seq < b are read and only pages of the pool are
// returned.
#pragma once

#include <stdint.h>

#include "../../include/tp.h"

#ifdef __CUDACC__
#define TP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TP_HOST_DEVICE inline
#endif

namespace tp {

// The sequence and the position of a row (0 ≤ row < rows); false if it is no
// token.  per_seq: rows of a sequence where start is NULL.
TP_HOST_DEVICE bool kv_token_of(const tp_kv_cache& c, const int32_t* start,
                                int per_seq, int64_t row, int* seq, int* pos) {
  int i;
  int64_t end;
  if (start == nullptr) {
    i = (int)(row / per_seq);
    end = (int64_t)(i + 1) * per_seq;
  } else {
    if (row < start[0] || row >= start[c.b]) return false;
    int hi = c.b;   // start[i] <= row < start[hi], whatever lies between
    i = 0;
    while (hi - i > 1) {
      const int mid = (i + hi) >> 1;
      if (start[mid] <= row)
        i = mid;
      else
        hi = mid;
    }
    end = start[hi];
  }
  const int64_t p = c.lens[i] - (end - row);   // < lens[i]
  *seq = i;
  *pos = (int)p;
  // (what is read twice above may have been changed in between)
  return p >= 0 && row < end;
}

// The page of position pos ≥ 0 of a sequence and the offset in it; −1 where
// the table has no page of the pool for it.
TP_HOST_DEVICE int64_t kv_page_of(const tp_kv_cache& c, int seq, int pos,
                                  int* offset) {
  const int col = pos / c.page;
  *offset = pos - col * c.page;
  if (col >= c.table_cols) return -1;
  const int32_t page = c.table[(int64_t)seq * c.table_stride + col];
  return page >= 0 && page < c.pages ? page : -1;
}

}  // namespace tp
