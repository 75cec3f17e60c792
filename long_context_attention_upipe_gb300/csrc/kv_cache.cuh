// Paged cache of keys and values: rows of head_dim elements (bf16, or e4m3 with one fp32 scale for each row)
// in pages of page_size tokens, found through a table of page numbers for each sequence.
#pragma once

#include "internal.h"

namespace upipe {

// Page and row of a position, or page -1 where there is none.
struct KvPlace {
  int page, row;
};

__device__ __forceinline__ KvPlace kv_place(const KvCache& c, const PageTable& t, int seq, int pos) {
  if ((unsigned)seq >= (unsigned)t.n_seqs || pos < 0) return KvPlace{-1, 0};
  const int i = pos / c.page_size;
  if (i >= t.max_pages) return KvPlace{-1, 0};
  const int page = t.pages[(int64_t)seq * t.stride + i];
  return KvPlace{(unsigned)page < (unsigned)c.n_pages ? page : -1, pos - i * c.page_size};
}

// Offsets, in elements, of a head's row and of its scale.
__device__ __forceinline__ int64_t kv_row(const KvCache& c, const KvPlace& at, int head) {
  return at.page * c.page_stride + head * c.head_stride + at.row * c.token_stride;
}
__device__ __forceinline__ int64_t kv_scale(const KvCache& c, const KvPlace& at, int head) {
  return at.page * c.scale_page_stride + head * c.scale_head_stride + at.row * c.scale_token_stride;
}

}  // namespace upipe
