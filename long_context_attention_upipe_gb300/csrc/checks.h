// Checks of arguments that the entry points share.
#pragma once

#include <initializer_list>

#include "internal.h"

namespace upipe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Status of a launch; a failed one leaves no error behind for the next call's check to find.
inline upipe_status_t finish(cudaError_t e) {
  if (e != cudaSuccess) (void)cudaGetLastError();
  return cuda_status(e);
}

// Two buffers that share some bytes.
inline bool overlaps(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && a_bytes && b_bytes && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

// A buffer of one call.  `rowwise`: every row is read, or written, by the threads that own it alone, so that an
// output may take the very place of an input.
struct Buf {
  const void* p;
  int64_t bytes;
  bool rowwise = false;
};

// Whether every output is apart from every other buffer, but for row-wise ones in one place.
inline bool outputs_apart(std::initializer_list<Buf> outs, std::initializer_list<Buf> ins) {
  for (const Buf* o = outs.begin(); o != outs.end(); ++o) {
    for (const Buf* p = outs.begin(); p != o; ++p)
      if (overlaps(o->p, o->bytes, p->p, p->bytes)) return false;
    for (const Buf& i : ins)
      if (overlaps(o->p, o->bytes, i.p, i.bytes) && !(o->rowwise && i.rowwise && o->p == i.p)) return false;
  }
  return true;
}

// Rows of `elems` elements of a [heads][tokens] tensor with the given strides: whether no two rows
// share an element.
inline bool rows_disjoint(int64_t heads, int64_t tokens, int64_t hs, int64_t ts, int64_t elems) {
  if (heads <= 1 && tokens <= 1) return true;
  if (heads <= 1) return ts >= elems;
  if (tokens <= 1) return hs >= elems;
  const bool head_outer = hs >= ts;
  const int64_t in = head_outer ? ts : hs, n_in = head_outer ? tokens : heads, outer = head_outer ? hs : ts;
  return in >= elems && outer >= in * (n_in - 1) + elems;
}

inline int64_t span_bytes(int64_t heads, int64_t tokens, int64_t hs, int64_t ts, int64_t elems) {
  return 2 * ((heads - 1) * hs + (tokens - 1) * ts + elems);
}

// Rows of one tensor: [heads][tokens] of `elems` elements; strides of single heads or tokens do not count.
struct HeadRows {
  const void* base;
  int64_t heads, tokens, hs, ts, elems;
  int64_t bytes() const { return span_bytes(heads, tokens, hs, ts, elems); }
  bool same(const HeadRows& o) const { return base == o.base && hs == o.hs && ts == o.ts; }
};
inline HeadRows rows_of(const void* base, int64_t heads, int64_t tokens, int64_t hs, int64_t ts, int64_t elems) {
  return HeadRows{base, heads, tokens, heads > 1 ? hs : 0, tokens > 1 ? ts : 0, elems};
}

// Whether two tensors share elements, as far as it can be told from their strides: not if their address ranges
// are apart, nor if they are parts of one token-major (or head-major) tensor, the heads (tokens) of the one in
// the gaps of the other.
inline bool rows_may_meet(const HeadRows& a, const HeadRows& b) {
  if (!overlaps(a.base, a.bytes(), b.base, b.bytes())) return false;
  auto in_gaps = [&](int64_t period_a, int64_t period_b, int64_t inner_a, int64_t inner_b) {
    if (period_a != period_b || period_a <= 0) return false;
    const int64_t d = (reinterpret_cast<intptr_t>(b.base) - reinterpret_cast<intptr_t>(a.base)) / 2;
    const int64_t off = ((d % period_a) + period_a) % period_a;  // b's place in a's period
    return off >= inner_a && off + inner_b <= period_a;
  };
  return !in_gaps(a.ts, b.ts, (a.heads - 1) * a.hs + a.elems, (b.heads - 1) * b.hs + b.elems) &&
         !in_gaps(a.hs, b.hs, (a.tokens - 1) * a.ts + a.elems, (b.tokens - 1) * b.ts + b.elems);
}

}  // namespace upipe
