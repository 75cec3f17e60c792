// What the kernels of the attention over a paged cache share: the line of tiles that the work is cut from, the pieces that a CTA
// leaves for others, and the sum of a row key by key.
#pragma once

#include "internal.h"
#include "kv_cache.cuh"
#include "quant.cuh"
#include "tc_common.cuh"

namespace upipe {

// What a row of a piece (or of a joined run of pieces) leaves beside its D sums.
struct RowSum {
  float m, l;
};

struct DecodeWs {
  int4* meta;     // [row blocks][CTAs] items of the pieces that the CTA leaves: x of one that ends an item, y of one that does
                  // not; z whether the latter begins its item, w the CTA in which it ends
  RowSum* sums;   // [row blocks][CTAs][2][rows]
  float* acc;     // [row blocks][CTAs][2][rows][D]
  int64_t scale_step;  // from a row's scale to the one 16 rows on
  int box_rows;   // rows of a copy: what divides a page and a tile of 128 keys (more than 16 rows)
  int share;      // 0; or the CTAs that each item has, a cluster; or -1: parts of the line that begin and end with items (nothing is left for the
                  // joining kernel)
};

// Rows of a block, blocks of rows, and CTAs for each of them.
struct DecodeShape {
  int rows, blocks, ctas;
};

namespace {

constexpr int kTileKeys = 16;         // rows of a box: what every page is a multiple of
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.0e38f;  // a reference below all scores, whose difference to them is defined
constexpr float kSlack = 8.f;        // a score may exceed the reference by this, in powers of two
constexpr float kSlackV = 5.f, kShiftV = 10.f;  // fp16 weights: the reference of one lies 10 below the score, the largest is 2^15
constexpr int kQueryTop = 15;        // fp16 queries: a row's largest element is in [2^15, 2^16)

__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A box of 16 rows of a page and head.  A row of more than 128 bytes (SEGS 2) has halves, from `half` on as many as the map's box has.
template <int SEGS>
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int row, int half, int head, int page) {
  if (SEGS == 2)
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(half), "r"(head), "r"(page), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(head), "r"(page), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Wait limits of n < 64 ns, which no copy would meet, are for testing: the barrier of place n - 1 of a ring of copies (modulo the ring) takes
// one arrival more than it gets, so waits for it run out (mbar_wait_addr alone may sleep until a copy has come, however short the limit).
constexpr uint64_t kTestNs = 64;
__device__ __forceinline__ int arrivals(int place, int ring, uint64_t wait_ns) {
  return 1 + (wait_ns < kTestNs && place == (int)(wait_ns - 1) % ring);
}
// The longest wait for copies in flight after that: a thousand times what a copy takes, if one of them is never seen to come.
__device__ __forceinline__ uint64_t drain_ns(uint64_t wait_ns) { return wait_ns < kTestNs ? 1000000 : tc::kDrainNs; }

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Four codes as two pairs of fp16.
__device__ __forceinline__ void e4m3x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi) : "r"(four));
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint32_t min_s16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.s16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Keys that the table can hold, and tiles of a sequence of `len` keys.
__host__ __device__ __forceinline__ int table_keys(const PageTable& t, int page_size) {
  const int64_t n = (int64_t)t.max_pages * page_size;
  return n < INT32_MAX ? (int)n : INT32_MAX;
}
template <int KEYS = kTileKeys>
__device__ __forceinline__ int tiles_of(int len, int cap) {
  return (int)(((int64_t)min(max(len, 0), cap) + KEYS - 1) / KEYS);
}

// Length of a sequence's item on the line: its tiles and its end.
template <int END, int KEYS = kTileKeys>
__device__ __forceinline__ int units_of(int len, int cap) {
  const int n = tiles_of<KEYS>(len, cap);
  return n ? n + END : 0;
}

// Sum over a warp of numbers up to 2^27, which may pass 32 bits.
__device__ __forceinline__ int64_t warp_sum(int n) {
  return ((int64_t)__reduce_add_sync(0xffffffffu, (unsigned)n >> 16) << 16) + __reduce_add_sync(0xffffffffu, (unsigned)n & 0xffffu);
}
__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += o;
  }
  return v;
}

// a * b / c of numbers whose product fits 64 bits; most fit 32, where a division takes a fraction of the time.
__device__ __noinline__ int64_t div64(int64_t p, int64_t c) { return p / c; }
__device__ __forceinline__ int64_t mul_div(int64_t a, int b, int c) {
  const int64_t p = a * b;
  return p <= 0xffffffffll ? (int64_t)((uint32_t)p / (uint32_t)c) : div64(p, c);
}

// Parts that a line of `total` tiles is cut into: no CTA gets less than a tile for each warp.
__device__ __forceinline__ int parts_of(int64_t total, int ctas, int warps) {
  return total < (int64_t)ctas * warps ? max((int)(total + warps - 1) / warps, 1) : ctas;
}

// The part that holds tile end - 1 where part i ends before tile total * (i + 1) / parts.
__device__ __forceinline__ int last_part(int64_t end, int64_t total, int parts) {
  const int64_t p = end * parts + total - 1;
  return (int)(p <= 0xffffffffll ? (int64_t)((uint32_t)p / (uint32_t)total) : div64(p, total)) - 1;
}

// A query row of a key head: row R is head R % g of the group and token R / g of the q_len newest.
struct RowAt {
  int64_t head, tok;
};
__device__ __forceinline__ RowAt row_at(const DecodeArgs& a, int g, int b, int hk, int R) {
  const int t = R / g;
  return RowAt{hk * g + (R - t * g), (int64_t)b * a.q_len + t};
}

// Elements e0 .. e0 + E of a cached row, times its scale.
template <int E, bool FP8>
__device__ __forceinline__ void load_row(const void* base, int64_t row, int e0, float scale, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    float2 f;
    if (FP8) {
      f = e4m3x2(*reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(base) + row + e0 + i));
      f.x *= scale;
      f.y *= scale;
    } else {
      f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(reinterpret_cast<const bf16*>(base) + row + e0 + i));
    }
    x[i] = f.x;
    x[i + 1] = f.y;
  }
}

// Reference, l and o of one query row over the keys [k0, k1) that it sees, key by key: a lane gets elements lane * D / 32 .. of o.  (All
// three, since o would not fit the l of scores that were added up in another order, if these are large.)
template <int D, bool FP8>
__device__ __noinline__ RowSum redo(const DecodeArgs& a, int b, int hk, RowAt at, int k0, int k1, float* out) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  RowSum sum{kLowest, 0.f};
  float q[E], acc[E] = {};
  load_row<E, false>(a.q, at.head * a.q_head + at.tok * a.q_tok, lane * E, 1.f, q);
  for (int j = k0; j < k1; ++j) {
    const KvPlace p = kv_place(a.c, a.t, b, j);
    if (p.page < 0) {
      sum.l = __uint_as_float(0x7fffffffu);
      continue;
    }
    const int64_t row = kv_row(a.c, p, hk), sc = FP8 ? kv_scale(a.c, p, hk) : 0;
    float k[E], v[E], s = 0.f;
    load_row<E, FP8>(a.c.k, row, lane * E, FP8 ? a.c.k_scale[sc] : 1.f, k);
    load_row<E, FP8>(a.c.v, row, lane * E, FP8 ? a.c.v_scale[sc] : 1.f, v);
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * k[e];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s = __fmul_rn(s, a.scale * kLog2e);
    if (s > sum.m) {
      const float f = exp2f(sum.m - s);
      sum = RowSum{s, sum.l * f};
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= f;
    }
    const float w = exp2f(s - sum.m);
    sum.l += w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += w * v[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = acc[e];
  return sum;
}

// The largest scale of a sequence's keys [k0, k1).
__device__ __noinline__ float most_key_scale(const DecodeArgs& a, int b, int hk, int k0, int k1) {
  float most = 0.f;
#pragma unroll 4
  for (int64_t j = k0 + (int)(threadIdx.x & 31); j < k1; j += 32) {  // (may pass 32 bits behind the longest sequence's end)
    const KvPlace p = kv_place(a.c, a.t, b, (int)j);
    if (p.page >= 0) most = fmaxf(most, fabsf(a.c.k_scale[kv_scale(a.c, p, hk)]));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
  return most;
}

__device__ __forceinline__ float row_lse(float m, float l) { return m * kLn2 + logf(l); }

// Rows R0 .. R1 of key heads h0 .. h1 of a sequence without tiles: zeros, or NaN where there are keys but no table.  All lanes of a
// warp, D / 8 to a row.
template <int D>
__device__ __forceinline__ void empty_rows(const DecodeArgs& a, int g, int b, int h0, int h1, int R0, int R1, int keys) {
  constexpr int LANES = D / 8;
  const int lane = threadIdx.x & 31, n = R1 - R0;
  for (int i = lane / LANES; i < (h1 - h0) * n; i += 32 / LANES) {
    const int h = i / n, R = R0 + i - h * n;
    const bool lost = max(keys, 0) - a.q_len + 1 + R / g > 0;  // (the lowest lengths less q_len pass 32 bits)
    const RowAt at = row_at(a, g, b, h0 + h, R);
    const uint32_t w = lost ? 0x7fff7fffu : 0u;
    *reinterpret_cast<uint4*>(a.o + at.head * a.o_head + at.tok * a.o_tok + lane % LANES * 8) = make_uint4(w, w, w, w);
    if (a.lse && lane % LANES == 0) a.lse[at.head * a.t.n_seqs * a.q_len + at.tok] = lost ? __uint_as_float(0x7fffffffu) : -INFINITY;
  }
}
// ... of the sequences that have none, a warp of the grid to a sequence (to each of the grid's `warps`th).
template <int D>
__device__ __forceinline__ void empty_sequences(const DecodeArgs& a, int g, int cap, int warp, int warps, int R0, int R1) {
  const int lane = threadIdx.x & 31;
  for (int64_t b0 = warp; b0 < a.t.n_seqs; b0 += (int64_t)32 * warps) {
    const int64_t b = b0 + (int64_t)lane * warps;
    const int len = b < a.t.n_seqs ? a.lens[b] : 1;
    unsigned none = __ballot_sync(0xffffffffu, b < a.t.n_seqs && tiles_of(len, cap) == 0);
    while (none) {
      const int i = __ffs(none) - 1;
      none &= none - 1;
      empty_rows<D>(a, g, (int)(b0 + (int64_t)i * warps), 0, a.c.n_kv_heads, R0, R1, __shfl_sync(0xffffffffu, len, i));
    }
  }
}

// Boxes of box_rows rows of a page and head, rows of SEGS halves of SEG bytes, of which a box has `halves`, side by side in shared memory.
template <int D, bool FP8>
bool tile_map(CUtensorMap* map, const KvCache& c, const void* base, uint32_t box_rows, uint32_t halves) {
  constexpr int ES = FP8 ? 1 : 2, SEG = D * ES > 128 ? 128 : D * ES, SEGS = D * ES / SEG;
  auto stride = [&](int64_t s) { return s ? (uint64_t)s * ES : (uint64_t)16; };  // 0: of a single page or head
  const uint64_t dims[5] = {SEG / ES, (uint64_t)c.page_size, 2, (uint64_t)c.n_kv_heads, (uint64_t)c.n_pages};
  const uint64_t strides[4] = {stride(c.token_stride), 128, stride(c.head_stride), stride(c.page_stride)};
  const uint32_t box[5] = {(uint32_t)(SEG / ES), box_rows, halves, 1, 1};
  return make_tmap_rows(map, base, !FP8, SEGS == 2, dims, strides, box, SEG);
}

}  // namespace

// Blocks of 32 or 64 rows of a bf16 cache (decode_wide.cu): leaves the pieces that the joining kernel takes.
cudaError_t launch_decode_wide(const DecodeArgs& a, const DecodeShape& sh, const DecodeWs& ws, cudaStream_t st);

}  // namespace upipe
