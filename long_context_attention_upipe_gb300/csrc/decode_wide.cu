// The attention of the newest tokens over a paged bf16 cache where more than 16 query rows share a key head: blocks of 32 or 64 rows.
//
// The formulas, the line of tiles that is cut into equal parts and the joining of an item's pieces are those of decode.cu.  There a
// warp holds at most 16 rows (the sums of more do not fit its registers), so 64 rows read the cache four times.  Here a CTA takes
// tiles of 128 keys, and the sums lie in tensor memory:
//   S^T [128 keys, rows] = K Q^T      O^T [D, rows] += V^T P
// so that the long sides are those that the tensor cores want long (rows fill 32 or 64 columns, not 128 lanes), and K and V are read as
// they lie in the cache, V transposed by its descriptor.  A lane of S^T is a key: its thread makes the weights of 16 rows and writes
// them as a piece of the 128-byte row of its key, which is P transposed.  A row's maximum would need all lanes, so it is a reference,
// raised only when a score passes it by 2^16; the threads vote on that once a tile.  Weights are two bf16 numbers (2^-17), two products.
//
// Warps: 0 brings keys and 3 values, in boxes of 16 to 128 rows of a page; 1 issues the products; 2 brings queries; the others make
// weights.  S is double, so the next tile's product runs under this one's weights; P and O are not
// (with rows of 128 elements shared memory is full; with 64 a second P would fit, and has not been tried).
//
// Bound by HBM where few items end: a CTA's share of it brings a tile's 64 KB in 2800 clocks, and a tile's chain with 64 rows (product 600
// clocks, weights 2100, product 980, overlapped but for P) takes 3200.  An item's end costs four tiles' time (kEnd 1: 60.7 instead of
// 48.7 us for 16 sequences up to 16000 keys with 24 rows; 6: 49.8).  A box takes its warp 100 clocks whatever its size: one warp with
// 32 boxes of 16 rows to a tile needed 3300 clocks, hence the two warps and the higher boxes.  Code that runs once for an item is kept in
// loops: unrolled, its instructions took longer to arrive than to run (an item's end 18000 clocks instead of 8000).
// Measured (GB300, bf16, calls back to back; in brackets as blocks of 16 rows, decode.cu):
//   1 sequence of 2000000 keys, 1 head of 128, 24 rows    162 us (190), 64 rows 174 (301), floor 152.9
//   8 sequences up to 30000, 8 heads of 128, 20 rows       77 us (105), 64 rows  83 (141), floor  64.9
//   8 sequences up to 30000, 8 heads of 64, 64 rows        76 us (110), floor 32.5
//
// Not taken for e4m3: with 4 or 8 more warps that convert tiles to fp16 in shared memory it was slower than decode.cu, which converts in
// registers, in batches (20 rows 110 us, 82; 64 rows 147, 153), no faster for 24 rows of one sequence, and 242 instead of 342 us for 64.
#include "decode.cuh"

namespace upipe {

namespace {

constexpr int kKeys = 128;       // of a tile: the lanes of S^T
constexpr int kSide = 4;         // tiles whose words on missing pages are kept
constexpr int kRows = 16;        // rows of a softmax thread
constexpr float kSlackWide = 16.f;  // the reference is raised when a score exceeds it by this many powers of two
constexpr int kEnd = 4;          // tiles' time that an item's end takes

template <int D, int RP>
struct Wide {
  static constexpr int SEGS = D / 64;             // columns of 128 bytes of a 16-bit row
  static constexpr int COL = kKeys * 128;
  static constexpr int OPERAND = SEGS * COL;      // keys or values of a tile, 16-bit
  static constexpr int RING = D == 128 ? 4 : 6;   // keys and values in turn
  static constexpr int P = COL;
  static constexpr int Q = SEGS * RP * 128;
  static constexpr int SOFTMAX = RP / kRows * kKeys;  // threads that make weights
  static constexpr int THREADS = 128 + SOFTMAX;
  static constexpr int AT_P = RING * OPERAND, AT_Q = AT_P + 2 * P;
  static constexpr int AT_SIDE = AT_Q + 2 * Q, SIDE = 32;
  static constexpr int AT_ROWS = AT_SIDE + kSide * SIDE;  // tables of the rows
  static constexpr int TABLES = 14;
  static constexpr int AT_BARS = AT_ROWS + TABLES * RP * 4;
  static constexpr int BARS = 2 * RING + 2 + 2 + 2 + 4 + 2 * kSide + 1;
  static constexpr int AT_WORDS = AT_BARS + BARS * 8;
  static constexpr int BYTES = AT_WORDS + 32 + 1024;
  static constexpr int COLUMNS = RP == 64 ? 256 : 128;    // of tensor memory: two of S, one of O
  static_assert(BYTES <= 227 * 1024 && AT_P >= 2048 * 8, "shared memory");
};

// A place on the line, and what is left of a part.  The lanes hold the lengths of the 32 sequences that b is among.
struct Line {
  int b, hk, tile, raw, len, n, lens;
  int64_t left;
};

__device__ __forceinline__ void line_item(const DecodeArgs& a, int cap, Line& w) {
  w.raw = __shfl_sync(0xffffffffu, w.lens, w.b & 31);
  w.len = min(max(w.raw, 0), cap);
  w.n = max(tiles_of<kKeys>(w.len, cap), 1);
}

// The first tile of the next item, if the part has more.
__device__ __forceinline__ void line_next(const DecodeArgs& a, int cap, Line& w) {
  w.left -= kEnd;
  if (w.left <= 0) return;
  w.tile = 0;
  if (++w.hk < a.c.n_kv_heads) return;
  w.hk = 0;
  const int lane = threadIdx.x & 31;
  unsigned some = __ballot_sync(0xffffffffu, w.lens > 0) & ~((2u << (w.b & 31)) - 1u);
  int b = w.b & ~31;
  while (!some) {
    b += 32;
    if (b >= a.t.n_seqs) {  // only if lengths changed under the call
      w.left = 0;
      return;
    }
    w.lens = b + lane < a.t.n_seqs ? a.lens[b + lane] : 0;
    some = __ballot_sync(0xffffffffu, w.lens > 0);
  }
  w.b = b + __ffs(some) - 1;
  line_item(a, cap, w);
}
__device__ __forceinline__ void line_step(const DecodeArgs& a, int cap, Line& w, int tiles) {
  w.left -= tiles;
  w.tile += tiles;
  if (w.tile >= w.n) line_next(a, cap, w);
}
__device__ __forceinline__ int line_rest(const Line& w) { return (int)min(w.left, (int64_t)(w.n - w.tile)); }  // of the item, in this part

template <int THREADS>
__device__ __forceinline__ bool any_of(bool mine) {  // of the softmax threads, all of which come here
  uint32_t any;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n barrier.cta.red.or.pred p, 1, %2, q;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(any) : "r"((uint32_t)mine), "n"(THREADS) : "memory");
  return any != 0;
}
// The largest number of a warp's that is not NaN: as integers in the same order.
__device__ __forceinline__ float warp_top(float x) {
  const int i = __float_as_int(x == x ? x : -INFINITY), top = __reduce_max_sync(0xffffffffu, i ^ (i >> 31 & 0x7fffffff));
  return __int_as_float(top ^ (top >> 31 & 0x7fffffff));
}
// Four columns of tensor memory, complete on return; and back.
__device__ __forceinline__ void tmem_ld4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\ntcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t at, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int D, int RP>
__global__ void __launch_bounds__(Wide<D, RP>::THREADS, 1)
    k_decode_wide(const __grid_constant__ DecodeArgs a, const DecodeWs ws, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, uint64_t wait_ns) {
  using L = Wide<D, RP>;
  constexpr int RH = kRows, SEGS = L::SEGS, RING = L::RING;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int X = gridDim.x, rb = blockIdx.y;
  const int hkv = a.c.n_kv_heads, g = a.hq / hkv, rows = g * a.q_len, n_seqs = a.t.n_seqs, cap = table_keys(a.t, a.c.page_size);
  const int ps = a.c.page_size;

  // ---- barriers
  const uint32_t full = base + L::AT_BARS, empty = full + 8 * RING, s_full = empty + 8 * RING, s_empty = s_full + 16;
  const uint32_t p_full = s_empty + 16, p_empty = p_full + 8;
  const uint32_t q_full = p_empty + 8, q_empty = q_full + 16, side_full = q_empty + 16, side_empty = side_full + 8 * kSide;
  const uint32_t done = side_empty + 8 * kSide;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::AT_WORDS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::AT_WORDS + 4);
  uint32_t* again = reinterpret_cast<uint32_t*>(smem + L::AT_WORDS + 8);  // [sixteen of the rows]
  if (threadIdx.x == 0) {
    auto init = [](uint32_t bar, int n, uint32_t count) {
      for (int i = 0; i < n; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar + 8 * i), "r"(count) : "memory");
    };
    for (int i = 0; i < RING; ++i) init(full + 8 * i, 1, arrivals(i, RING, wait_ns));
    init(empty, RING, 1);
    init(s_full, 2, 1);
    init(s_empty, 2, L::SOFTMAX / 32);
    init(p_full, 1, L::SOFTMAX / 32);
    init(p_empty, 1, 1);
    init(q_full, 2, 32);
    init(q_empty, 2, 1 + L::SOFTMAX / 32);
    init(side_full, kSide, 32);
    init(side_empty, kSide, L::SOFTMAX / 32);
    init(done, 1, 1);
    tc::fence_mbar_init();
    *abort_flag = 0;
    again[0] = again[1] = again[2] = again[3] = 0;
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, L::COLUMNS);
    tc::tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_trigger();  // the joining kernel reads nothing of this one before it has ended

  // ---- the CTA's part of the line
  int64_t* sums = reinterpret_cast<int64_t*>(smem);
  const int chunks = (n_seqs + 31) / 32;
  for (int ch = warp; ch < chunks; ch += L::THREADS / 32) {
    const int b = ch * 32 + lane;
    const int64_t n = warp_sum(b < n_seqs ? units_of<kEnd, kKeys>(a.lens[b], cap) : 0);
    if (lane == 0) sums[ch] = n;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  int64_t total = 0;
  for (int ch = lane; ch < chunks; ch += 32) total += sums[ch];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  total *= hkv;
  const int parts = parts_of(total, X, 1);
  Line at{};
  int64_t part_end = 0;
  if (blockIdx.x < parts && total > 0) {
    const int64_t first = mul_div(total, blockIdx.x, parts);
    part_end = mul_div(total, blockIdx.x + 1, parts);
    at.left = part_end - first;
    const int64_t seq_first = mul_div(first, 1, hkv);  // the tile's place if there were one head
    int64_t before = 0;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
      const int64_t v = c0 + lane < chunks ? sums[c0 + lane] : 0, in = warp_scan(v, lane);
      const unsigned hit = __ballot_sync(0xffffffffu, before + in > seq_first);
      if (hit) {
        at.b = (c0 + __ffs(hit) - 1) * 32;
        before += __shfl_sync(0xffffffffu, in - v, __ffs(hit) - 1);
        break;
      }
      before += __shfl_sync(0xffffffffu, in, 31);
    }
    at.lens = at.b + lane < n_seqs ? a.lens[at.b + lane] : 0;
    const int64_t upto = warp_scan(units_of<kEnd, kKeys>(at.lens, cap), lane);
    const int i = max(__ffs(__ballot_sync(0xffffffffu, before + upto > seq_first)) - 1, 0);
    const int n = max(units_of<kEnd, kKeys>(__shfl_sync(0xffffffffu, at.lens, i), cap), 1);
    before += __shfl_sync(0xffffffffu, upto, i) - n;
    at.b = min(at.b + i, n_seqs - 1);
    const int64_t rest = max(first - before * hkv, (int64_t)0);
    at.hk = (int)min(mul_div(rest, 1, n), (int64_t)(hkv - 1));  // within bounds even if lengths change under the call
    at.tile = (int)min(rest - (int64_t)at.hk * n, (int64_t)(n - 1));
    line_item(a, cap, at);
    if (at.tile >= at.n) {  // within an item's end
      at.left -= n - at.tile - kEnd;
      line_next(a, cap, at);
    }
  }
  fence_async();  // copies fill the place of the sums
  __syncthreads();

  auto wait = [&](uint32_t bar, uint32_t parity) {
    return (bool)__all_sync(0xffffffffu, tc::mbar_wait_addr(bar, parity, abort_flag, wait_ns));
  };
  const uint32_t units = base, ptile = base + L::AT_P, qtile = base + L::AT_Q, side = base + L::AT_SIDE;
  // of each row: the reference, its change's factor, maxima and sums of four warps, the whole sum, o's factor, the first key that it does
  // not see less the sequence's length, offsets in o and in q from those of the item's first row (q: -1 where there is none)
  float* t_m = reinterpret_cast<float*>(smem + L::AT_ROWS);
  float *t_f = t_m + RP, *t_top = t_f + RP, *t_sum = t_top + 4 * RP, *t_by = t_sum + RP;
  int* t_see = reinterpret_cast<int*>(t_by + RP);
  int64_t *t_off = reinterpret_cast<int64_t*>(t_see + RP), *t_qat = t_off + RP;

  // Tiles of keys (warp 0) and values (warp 3), in turn in the ring: boxes of a page's rows, a lane to each.
  const int box_rows = ws.box_rows, boxes_col = kKeys / box_rows, my_box = lane % boxes_col, my_col = lane / boxes_col;
  const bool mine = lane < boxes_col * SEGS;
  auto entry = [&](const Line& w, int key) {
    if (w.left <= 0) return -1;  // the tile may be the one after the longest sequence's last
    key += w.tile * kKeys;
    return key < w.len && key / ps < a.t.max_pages ? a.t.pages[(int64_t)w.b * a.t.stride + key / ps] : -1;
  };
  auto bring = [&](const CUtensorMap* map, uint32_t u, int page, int hk, int row) {
    const uint32_t slot = u % RING;
    if (!wait(empty + slot * 8, (u / RING & 1) ^ 1)) return false;
    const bool have = mine && (unsigned)page < (unsigned)a.c.n_pages;
    const int boxes = __popc(__ballot_sync(0xffffffffu, have));
    if (lane == 0) {
      if (boxes) expect_tx(full + slot * 8, boxes * box_rows * 128);
      else tc::mbar_arrive_addr(full + slot * 8);
    }
    __syncwarp();
    if (have) tma_tile<SEGS>(units + slot * L::OPERAND + my_col * L::COL + my_box * box_rows * 128, map, full + slot * 8, row, my_col, hk, page);
    __syncwarp();
    return true;
  };
  static_assert(RING % 2 == 0, "keys and values have slots of their own");
  // waits for what is on its way of this warp's units (every other one) before `end`
  auto settle = [&](uint32_t end) {
    const uint64_t t0 = tc::globaltimer();
    for (uint32_t u = end > RING ? end - RING : end & 1; u < end; u += 2)
      while (!tc::mbar_try_wait_addr(full + u % RING * 8, u / RING & 1))
        if (tc::globaltimer() - t0 > drain_ns(wait_ns)) return;
  };
  if (warp == 0) {
    Line w = at;
    int next = entry(w, my_box * box_rows);
    uint32_t u = 0;
    while (w.left > 0) {
      const int page = next, hk = w.hk, row = (w.tile * kKeys + my_box * box_rows) % ps;
      line_step(a, cap, w, 1);
      next = entry(w, my_box * box_rows);
      if (!bring(&map_k, u, page, hk, row)) break;
      u += 2;
    }
    settle(u);
  } else if (warp == 1) {
    // ---- products
    constexpr uint32_t id_s = tc::idesc_bf16(128, RP, false, false), id_o = tc::idesc_bf16(128, RP, true, true);
    const uint64_t k_desc = tc::sdesc_sw128(units, 16, 1024), q_desc = tc::sdesc_sw128(qtile, 16, 1024);
    // with D 64 the lanes of O^T above 63 have some of the same rows again, which nobody reads
    const uint64_t v_desc = tc::sdesc_sw128(units, SEGS == 2 ? L::COL : 1024, 1024), p_desc = tc::sdesc_sw128(ptile, L::COL, 1024);
    Line wt = at, wp = at;  // the tile whose scores are next, and whose weights
    uint32_t ts = 0, tp = 0, item = 0;
    bool ok = true, fresh_s = true, fresh_o = true;
    auto product_s = [&]() {
      const uint32_t u = 2 * ts, slot = u % RING, buf = item & 1;
      if (fresh_s) ok = ok && wait(q_full + buf * 8, item >> 1 & 1);
      ok = ok && wait(full + slot * 8, u / RING & 1) && wait(s_empty + (ts & 1) * 8, (ts >> 1 & 1) ^ 1);
      tc::fence_after_sync();
      const bool last = line_rest(wt) == 1;
      if (ok && tc::elect_one()) {
        const uint64_t ad = tc::sdesc_add(k_desc, slot * L::OPERAND), bd = tc::sdesc_add(q_desc, buf * L::Q);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(tmem + (ts & 1) * RP, tc::sdesc_add(ad, k / 4 * L::COL + k % 4 * 32), tc::sdesc_add(bd, k / 4 * (RP * 128) + k % 4 * 32), id_s, k > 0);
        tc::mma_commit(reinterpret_cast<uint64_t*>(smem + (empty + slot * 8 - base)));
        tc::mma_commit(reinterpret_cast<uint64_t*>(smem + (s_full + (ts & 1) * 8 - base)));
        if (last) tc::mma_commit(reinterpret_cast<uint64_t*>(smem + (q_empty + buf * 8 - base)));
      }
      __syncwarp();
      fresh_s = last;
      item += last;
      ++ts;
      line_step(a, cap, wt, 1);
    };
    while (wp.left > 0) {
      while (wt.left > 0 && ts <= tp + 1) product_s();
      const uint32_t u = 2 * tp + 1, slot = u % RING;
      ok = ok && wait(full + slot * 8, u / RING & 1) && wait(p_full, tp & 1);
      tc::fence_after_sync();
      if (ok && tc::elect_one()) {
        const uint64_t ad = tc::sdesc_add(v_desc, slot * L::OPERAND);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            tc::mma_ss(tmem + 2 * RP, tc::sdesc_add(ad, k * 2048), tc::sdesc_add(p_desc, part * L::P + k * 2048), id_o, part || k || !fresh_o);
        tc::mma_commit(reinterpret_cast<uint64_t*>(smem + (empty + slot * 8 - base)));
        tc::mma_commit(reinterpret_cast<uint64_t*>(smem + (p_empty - base)));
      }
      __syncwarp();
      fresh_o = line_rest(wp) == 1;
      ++tp;
      line_step(a, cap, wp, 1);
    }
    if (tc::elect_one()) tc::mma_commit(reinterpret_cast<uint64_t*>(smem + (done - base)));
    __syncwarp();
    tc::drain_ring(done, 1, 1);
  } else if (warp == 2) {
    // ---- queries of an item
    constexpr int CH = D / 8, PER = 32 / CH;  // 16-byte pieces of a row, rows at a time
    for (int r = lane; r < RP; r += 32) {
      const int R = rb * RP + r;
      t_qat[r] = R < rows ? R % g * a.q_head + R / g * a.q_tok : -1;
    }
    __syncwarp();
    Line w = at;
    bool ok = true;
    for (uint32_t item = 0; w.left > 0 && ok; ++item) {
      const uint32_t buf = item & 1;
      const bf16* from = a.q + (int64_t)w.hk * g * a.q_head + (int64_t)w.b * a.q_len * a.q_tok + lane % CH * 8;
      ok = wait(q_empty + buf * 8, (item >> 1 & 1) ^ 1);
      if (!ok) break;
      auto to = [&](int r) { return qtile + buf * L::Q + lane % CH / 8 * (RP * 128) + r * 128 + ((lane ^ r) & 7) * 16; };
#pragma unroll 8
      for (int r = lane / CH; r < RP; r += PER) {
        const int64_t off = t_qat[r];
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to(r)), "l"(from + max(off, (int64_t)0)), "r"(off < 0 ? 0 : 16) : "memory");
      }
      cp_commit();
      cp_wait<0>();
      fence_async();
      tc::mbar_arrive_addr(q_full + buf * 8);
      line_step(a, cap, w, line_rest(w));
    }
  } else if (warp == 3) {
    // ---- values, and a word for each 16 keys: NaN where their page is missing
    Line w = at;
    const int chunk = lane & 7;
    int next = entry(w, chunk * kTileKeys), next_v = entry(w, my_box * box_rows);
    uint32_t t = 0;
    for (; w.left > 0; ++t) {
      const uint32_t slot = t % kSide, to = side + slot * L::SIDE;
      const int page = next, hk = w.hk;
      const int page_v = next_v, row_v = (w.tile * kKeys + my_box * box_rows) % ps;
      line_step(a, cap, w, 1);
      next = entry(w, chunk * kTileKeys);
      next_v = entry(w, my_box * box_rows);
      if (!wait(side_empty + slot * 8, (t / kSide & 1) ^ 1)) break;
      if (lane < 8)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + lane * 4), "r"((unsigned)page < (unsigned)a.c.n_pages ? 0u : 0x7fffffffu) : "memory");
      tc::mbar_arrive_addr(side_full + slot * 8);
      if (!bring(&map_v, 2 * t + 1, page_v, hk, row_v)) break;
    }
    settle(2 * t + 1);
  } else {
    // ---- weights.  A thread has key 32 * quarter + lane of a tile and rows col .. of the block; later element 32 * quarter + lane of o
    const int quarter = warp & 3, side_of = (warp - 4) >> 2, col = side_of * RH, key = quarter * 32 + lane, st = threadIdx.x - 128;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16, o_tm = tmem + lanes + 2 * RP + col;
    const float cs = a.scale * kLog2e;
    int4 meta = make_int4(-1, -1, 0, 0);
    const int64_t place = (int64_t)rb * X + blockIdx.x;
    if (st < RP) {
      const int R = min(rb * RP + st, rows - 1);
      t_see[st] = R / g - a.q_len + 1;
      t_off[st] = R % g * a.o_head + R / g * a.o_tok;
    }
    Line w = at;
    bool ok = true;
    uint32_t t = 0;
    float l[RH];
    for (uint32_t item = 0; w.left > 0; ++item) {
      const int begin = w.tile, tiles = line_rest(w), b = w.b, hk = w.hk, len = w.len;
      if (st < RP) t_m[st] = kLowest;
#pragma unroll
      for (int j = 0; j < RH; ++j) l[j] = 0.f;
      tc::named_bar_sync(2, L::SOFTMAX);
      const int all_seen = len - a.q_len + 1;  // keys before this are seen by every row
      for (int i = 0; i < tiles; ++i, ++t) {
        const int k0 = (begin + i) * kKeys;
        const uint32_t from = side + t % kSide * L::SIDE, s_at = tmem + lanes + (t & 1) * RP + col;
        float nan;
        ok = ok && wait(side_full + t % kSide * 8, t / kSide & 1);
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(nan) : "r"(from + key / kTileKeys * 4) : "memory");
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_addr(side_empty + t % kSide * 8);
        ok = ok && wait(s_full + (t & 1) * 8, t >> 1 & 1);
        tc::fence_after_sync();
        if (!ok) nan = __uint_as_float(0x7fffffffu);
        // (k0 + kKeys may pass 32 bits in the last tile of the longest sequence)
        const bool some_hidden = k0 > all_seen - kKeys || __any_sync(0xffffffffu, nan != 0.f);
        const int unseen = k0 + key - len;  // less than a row's `see`: seen
        // scores in units of log2, less the references; until none exceeds them by too much
        float d[RH];
        for (bool raised = false;; raised = true) {
          uint32_t x[RH];
          tc::tmem_ld16(s_at, x);
          tc::tmem_ld16_ready(x);
          float most = -INFINITY;
#pragma unroll
          for (int j = 0; j < RH; j += 4) {
            const float4 m = *reinterpret_cast<const float4*>(t_m + col + j);
            d[j] = __fsub_rn(__fmul_rn(__uint_as_float(x[j]), cs), m.x);  // two roundings, as in decode.cu
            d[j + 1] = __fsub_rn(__fmul_rn(__uint_as_float(x[j + 1]), cs), m.y);
            d[j + 2] = __fsub_rn(__fmul_rn(__uint_as_float(x[j + 2]), cs), m.z);
            d[j + 3] = __fsub_rn(__fmul_rn(__uint_as_float(x[j + 3]), cs), m.w);
            most = fmax3(fmax3(most, d[j], d[j + 1]), d[j + 2], d[j + 3]);
          }
          if (some_hidden) {
            most = -INFINITY;
#pragma unroll
            for (int j = 0; j < RH; ++j) {
              d[j] = unseen < t_see[col + j] ? d[j] + nan : -INFINITY;
              most = fmaxf(most, d[j]);
            }
          }
          if (!any_of<L::SOFTMAX>(most > kSlackWide) || raised) break;
#pragma unroll 1
          for (int j = 0; j < RH; j += 4) {
            tmem_ld4(s_at + j, *reinterpret_cast<uint32_t(*)[4]>(x));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float top = warp_top(unseen < t_see[col + j + k] ? __fmul_rn(__uint_as_float(x[k]), cs) : -INFINITY);
              if (lane == 0) t_top[quarter * RP + col + j + k] = top;
            }
          }
          tc::named_bar_sync(2, L::SOFTMAX);
          if (st < RP) {
            const float m = t_m[st];
            const float top = fmaxf(m, fmaxf(fmaxf(t_top[st], t_top[RP + st]), fmaxf(t_top[2 * RP + st], t_top[3 * RP + st])));
            t_m[st] = top;
            t_f[st] = fast_exp2(m - top);
          }
          tc::named_bar_sync(2, L::SOFTMAX);
#pragma unroll
          for (int j = 0; j < RH; ++j) l[j] *= t_f[col + j];
          if (i > 0) {
            ok = ok && wait(p_empty, (t & 1) ^ 1);
            tc::fence_after_sync();
#pragma unroll 1
            for (int j = 0; j < RH; j += 4) {
              tmem_ld4(o_tm + j, *reinterpret_cast<uint32_t(*)[4]>(x));
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * t_f[col + j + k]);
              tmem_st4(o_tm + j, *reinterpret_cast<uint32_t(*)[4]>(x));
            }
            tc::tmem_st_wait();
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_addr(s_empty + (t & 1) * 8);
        ok = ok && wait(p_empty, (t & 1) ^ 1);  // the weights of the tile before have been used
        if (side_of == 0 && k0 > len - kKeys) {  // rows behind the sequence's end may hold anything: the values' become zeros
          const uint32_t u = 2 * t + 1, slot = u % RING;
          ok = ok && wait(full + slot * 8, u / RING & 1);
          if (ok && k0 + key >= len)
#pragma unroll
            for (int c = 0; c < 8 * SEGS; ++c) sts128(units + slot * L::OPERAND + c / 8 * L::COL + key * 128 + c % 8 * 16, 0, 0, 0, 0);
        }
        const uint32_t to = ptile + key * 128;
#pragma unroll
        for (int j = 0; j < RH; j += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const float p0 = fast_exp2(d[j + k]), p1 = fast_exp2(d[j + k + 1]);
            l[j + k] += p0;
            l[j + k + 1] += p1;
            hi[k / 2] = pack_bf16(p0, p1);
            lo[k / 2] = pack_bf16(p0 - __uint_as_float(hi[k / 2] << 16), p1 - __uint_as_float(hi[k / 2] & 0xffff0000u));
          }
          const uint32_t piece = (((col + j) / 8 ^ key) & 7) * 16;
          sts128(to + piece, hi[0], hi[1], hi[2], hi[3]);
          sts128(to + L::P + piece, lo[0], lo[1], lo[2], lo[3]);
        }
        fence_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_addr(p_full);
      }

      // ---- the piece ends
      const bool begins = begin == 0, ends = begin + tiles == w.n, whole = begins && ends;
      if (!ends) {
        meta.y = b * hkv + hk;
        meta.z = begins;
        meta.w = last_part(part_end + (w.n - begin - tiles), total, parts);  // the CTA whose part holds the item's last tile
      } else if (!whole) {
        meta.x = b * hkv + hk;
      }
      // sums of the rows over the lanes: of row lane / 2
#pragma unroll
      for (int n = RH / 2, off = 16; n > 0; n >>= 1, off >>= 1)
#pragma unroll
        for (int j = 0; j < n; ++j) {
          const bool up = lane & off;
          const float keep = up ? l[j + n] : l[j], give = up ? l[j] : l[j + n];
          l[j] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
      t_top[quarter * RP + col + (lane >> 1)] = l[0];
      ok = ok && wait(p_empty, (t & 1) ^ 1);
      tc::fence_after_sync();
      tc::named_bar_sync(2, L::SOFTMAX);
      const int64_t left_at = (place * 2 + (ends ? 0 : 1)) * RP;
      if (st < RP) {
        const int R = rb * RP + st;
        float sum = t_top[st] + t_top[RP + st] + t_top[2 * RP + st] + t_top[3 * RP + st];
        if (w.raw > cap || !ok || *abort_flag) sum = __uint_as_float(0x7fffffffu);
        const float m = t_m[st];
        t_sum[st] = sum;
        t_by[st] = whole ? 1.f / sum : 1.f;
        if (R < rows) {
          if (whole) {
            if (a.lse) {
              const RowAt row = row_at(a, g, b, hk, R);
              a.lse[row.head * n_seqs * a.q_len + row.tok] = len + t_see[st] <= 0 ? -INFINITY : row_lse(m, sum);
            }
          } else {
            ws.sums[left_at + st] = RowSum{m, sum};
          }
        }
      }
      tc::named_bar_sync(2, L::SOFTMAX);
      bf16* const o_at = a.o + (int64_t)hk * g * a.o_head + (int64_t)b * a.q_len * a.o_tok + key;
      uint32_t bad = 0;
      if (quarter * 32 < D) {
#pragma unroll 1
        for (int j = 0; j < RH; j += 4) {
          uint32_t o[4];
          tmem_ld4(o_tm + j, o);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = col + j + k;
            if (rb * RP + r >= rows) break;
            const float v = __uint_as_float(o[k]);
            if (!(fabsf(v) < INFINITY) && fabsf(t_sum[r]) < INFINITY) bad |= 1u << (j + k);
            if (whole) o_at[t_off[r]] = __float2bfloat16(len + t_see[r] <= 0 ? 0.f : v * t_by[r]);
            else ws.acc[(left_at + r) * D + key] = v * t_by[r];
          }
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (lane == 0 && bad) atomicOr(&again[side_of], bad);
      }
      tc::fence_before_sync();
      tc::named_bar_sync(2, L::SOFTMAX);
      const uint32_t redone = again[side_of];
      if (redone) {  // rows whose sums have to be made once more
        constexpr int E = D / 32;
#pragma unroll 1
        for (int j = quarter; j < RH; j += 4) {
          if (!(redone >> j & 1)) continue;
          const int r = col + j, R = rb * RP + r, end = (int)min((int64_t)(begin + tiles) * kKeys, (int64_t)(len + t_see[r]));
          const RowAt row = row_at(a, g, b, hk, R);
          float out[E];
          const RowSum sum = redo<D, false>(a, b, hk, row, begin * kKeys, end, out);
          __syncwarp();
          if (w.raw > cap) continue;  // NaN
          if (!whole) {
#pragma unroll
            for (int e = 0; e < E; ++e) ws.acc[(left_at + r) * D + lane * E + e] = out[e];
            if (lane == 0) ws.sums[left_at + r] = sum;
          } else if (end > 0) {
            bf16* o = a.o + row.head * a.o_head + row.tok * a.o_tok + lane * E;
            const float inv = 1.f / sum.l;
#pragma unroll
            for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16(out[e] * inv, out[e + 1] * inv);
            if (a.lse && lane == 0) a.lse[row.head * n_seqs * a.q_len + row.tok] = row_lse(sum.m, sum.l);
          }
        }
      }
      tc::named_bar_sync(2, L::SOFTMAX);
      if (st < RP / kRows) again[st] = 0;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_addr(q_empty + (item & 1) * 8);
      line_step(a, cap, w, tiles);
    }
    if (st == 0) ws.meta[place] = meta;
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::COLUMNS);
  }
}

template <int D, int RP>
cudaError_t run_wide(const DecodeArgs& a, const DecodeShape& sh, DecodeWs ws, cudaStream_t st) {
  using L = Wide<D, RP>;
  auto kfn = k_decode_wide<D, RP>;
  CUtensorMap mk, mv;
  ws.box_rows = kTileKeys;
  while (ws.box_rows < kKeys && a.c.page_size % (2 * ws.box_rows) == 0) ws.box_rows *= 2;
  if (!tile_map<D, false>(&mk, a.c, a.c.k, ws.box_rows, 1) || !tile_map<D, false>(&mv, a.c, a.c.v, ws.box_rows, 1)) return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (e != cudaSuccess) return e;
  return launch_pdl(kfn, dim3(sh.ctas, sh.blocks), dim3(L::THREADS), L::BYTES, st, a, ws, mk, mv, wait_limit_ns());
}

}  // namespace

cudaError_t launch_decode_wide(const DecodeArgs& a, const DecodeShape& sh, const DecodeWs& ws, cudaStream_t st) {
  if (a.c.head_dim == 64) return run_wide<64, 64>(a, sh, ws, st);
  return sh.rows == 64 ? run_wide<128, 64>(a, sh, ws, st) : run_wide<128, 32>(a, sh, ws, st);
}

}  // namespace upipe
