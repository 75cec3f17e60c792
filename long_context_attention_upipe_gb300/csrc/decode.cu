// Attention of the newest tokens of many sequences over their cached keys and values.
//
// For query t of the T newest tokens of a sequence of len keys, over the keys j < len - T + 1 + t:
//   s_j = scale q . k_j,   lse = log sum_j exp s_j,   o = sum_j exp(s_j - lse) v_j
// and o = 0, lse = -infinity where no key is seen.
//
// The cache is read once, and that bounds the kernel: with g query heads to a key head it takes 2 g T operations for each byte of
// bf16 (4 g T of e4m3), where the tensor cores have hundreds to spare; a tcgen05 tile of 128 rows would be empty but for g T of
// them.  So the split follows the bytes.  All tiles of 16 keys of all (sequence, key head) items form one line, in order, with a
// few tiles' time added at each item's end for what an end costs (without: 94 instead of 88.6 us for 64 sequences up to 16384
// keys).  The CTAs, one to an SM, take equal parts of the line, and a CTA's warps equal parts of that, whatever the lengths.
// A warp runs its tiles through a queue of its own in shared memory: one TMA box each for 16 keys and 16 values of a page, so any
// page, head and token strides cost no instructions, and warps wait for nobody but their copies.  (Memory does care: rows that lie token
// by token, 8 heads of 256 bytes, take 60 instead of 58 us for 48 sequences up to 8192 keys in bf16; of 128 bytes, with their scales
// token by token too, 127 instead of 88 for 64 up to 16384 in e4m3, 118 with scales head by head.)
//
// Per tile, keys are the 16 rows of m16n8k16 and up to 8 (NT = 2: 16) query rows its columns:
//   S^T = K Q^T,   P = exp2(S - m),   O^T += V^T P^T
// K's fragments come by ldmatrix, V's by its transposing form, P^T by an 8 x 8 transposition in registers.
//   bf16  weights enter as the sum of two bf16 numbers (2^-17); a single one would double the error of o.
//   e4m3  codes are converted to fp16 (exact).  A 16-byte piece of codes gives a lane four neighbouring elements, so the steps of
//         S^T take the head dimension in that order and the rows of O^T are pairs of elements.  q goes to fp16 under a power of two
//         for each row (exact, but for elements below 2^-32 of the largest: redo, if they can move a score), K's scale to the score, and
//         V's scale to the weight's exponent, s_j - m + log2 sv_j, under a maximum of its own; weights are fp16 (2^-11) up to 2^15, which
//         leaves 2^-35 of the largest.
// The maximum is a reference that is raised, and the sums rescaled, only when a score exceeds it by a margin: one vote for each
// tile, no shuffles.  m, l and O are fp32.
//
// A warp's part may begin or end within an item.  The CTA joins such pieces in shared memory, in order, and what an item leaves
// in several CTAs a second kernel joins, in order: no atomics, equal calls give equal bits.
// Few short sequences have a cluster of CTAs to each item instead, which join their sums through each other's shared memory, and somewhat
// more get parts that begin and end with items: one launch.  Rows of empty sequences are written by all warps of the last launch, a
// sequence to each (200 sequences of 8 heads, one in eight empty: 14 us; with 32 sequences to a warp 58).
// (More than 16 rows of a long bf16 cache: decode_wide.cu.)
//
// A value that is infinite or NaN spoils the products of query rows that do not see it (zero times infinity), and of those that do
// where a weight's second part is zero.  Then o is not finite although l is, and the piece is made again key by key (redo), as
// is that of a query row that fp16 does not hold.  (Which takes 40 times as long: 3.6 ms for 64 sequences up to 16384 keys, each query
// with an element that towers 2^40 over the others; to make sure that dead channels need none of it takes 108 us instead of 90.)
//
// Measured (GB300, calls back to back; floor: the cached bytes at the copy rate of 6698 GB/s):
//   1 sequence of 1048576 keys, 4 / 1 heads, bf16       86 - 88 us, floor 80.2
//   1 of 5242880, 8 / 1, e4m3                           206 - 222 us, 206.6 (as fast as the box's memory)
//   64 up to 16384, 32 / 8, e4m3                             88 us, 76.0
//   48 up to 8192, 40 / 8, bf16                              58 us, 48.3
//   16 up to 32768, 4 tokens each, 32 / 8, e4m3         64 - 65 us, 47.3
//   256 up to 500, 4 / 2 heads of 64, bf16                 10.4 us, 2.2
//   1 of 4097, 32 / 8, bf16                           9.2 - 9.6 us, 2.5
// (With tables as wide as the longest sequence is long: kernels are chosen by the table's room, and 1000 keys of 8 heads take 8.7 instead
// of 7.2 us, 256 sequences up to 500 11.2 instead of 10.4, in a table for 131072.)
// One long sequence streams at the copy rate.  What a call adds: 5 us until the first tile lands (lengths, table entries and
// queries are read one after another), 2 to 4 us for the ends of the last items, 2 to 3 us for the second launch.  With 16 rows
// of an e4m3 cache the tiles' own chain of instructions shows as well: 254 registers leave room for 8 warps.
#include <type_traits>

#include "decode.cuh"

namespace upipe {

namespace {

template <int D, bool FP8, int NT, int W>
struct Lay {
  static constexpr int ROWB = D * (FP8 ? 1 : 2);        // bytes of a cached row
  static constexpr int SEG = ROWB > 128 ? 128 : ROWB;   // ... of which a box is so many wide: what a swizzle spans
  static constexpr int SEGS = ROWB / SEG;
  static constexpr int KBYTES = kTileKeys * ROWB;
  static constexpr int STAGE = 2 * KBYTES;              // keys and values of a tile
  static constexpr int SCALES = FP8 ? 128 : 0;          // their scales
  static constexpr int ROWS = 8 * NT;
  static constexpr int SLOT = ROWS * D * 4;             // sums of a piece's o
  static constexpr int WARPS = W;
  static constexpr int END = FP8 ? 4 : 2;               // tiles' time that an item's end (and the next one's begin) takes
  static constexpr int FIT = ((226 * 1024 - 16) / WARPS - 44 - SLOT - 2 * ROWS * (int)sizeof(RowSum)) / (STAGE + SCALES + 8);
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int QUEUE = STAGES * STAGE;
  static constexpr int AT_SCALES = WARPS * QUEUE, AT_SLOTS = AT_SCALES + WARPS * STAGES * SCALES;
  static constexpr int AT_SUMS = AT_SLOTS + WARPS * SLOT, AT_BARS = AT_SUMS + WARPS * 2 * ROWS * (int)sizeof(RowSum);
  static constexpr int AT_INFO = AT_BARS + WARPS * STAGES * 8;
  static constexpr int BYTES = AT_INFO + WARPS * 44 + 16 + 1024;  // the queues start on 1024 bytes
  static constexpr int MT = D / 16;                     // tiles of O^T
  static constexpr int KS = D / 16;                     // steps of S^T
  static_assert(STAGES >= 2 && QUEUE >= 2 * SLOT && WARPS * QUEUE >= 2048 * 8 && BYTES <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ float lds32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void lds_floats(float* v, uint32_t at) {
  if (N == 4)
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[N - 2]), "=f"(v[N - 1]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(at) : "memory");
}
// From the shared memory of another CTA of the cluster.
template <int N>
__device__ __forceinline__ void ld_cluster(float* v, uint32_t at) {
  if (N == 4)
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[N - 2]), "=f"(v[N - 1]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(at) : "memory");
}
// Four 8 x 8 matrices of 16-bit elements, a lane's address naming a row of one.
template <int AT>
__device__ __forceinline__ void ldm4(uint32_t (&w)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at), "n"(AT) : "memory");
}
template <int AT>
__device__ __forceinline__ void ldm4_trans(uint32_t (&w)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at), "n"(AT) : "memory");
}
// f(0), f(1) .. f(N - 1), the argument known at compile time.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(const F& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    each<N, I + 1>(f);
  }
}

template <bool FP8>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (FP8)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Waits, a second at most, for the `n` copies from `stage` on that are on their way although a wait for one ran out.
__device__ __forceinline__ void drain(uint32_t bars, int stages, int stage, uint32_t parity, int n, uint64_t ns) {
  if (n == 0) return;
  const uint64_t t0 = tc::globaltimer();
  for (; n > 0; --n) {
    while (!tc::mbar_try_wait_addr(bars + stage * 8, parity))
      if (tc::globaltimer() - t0 > ns) return;
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
  }
}

constexpr int kJoinThreads = 256;

// LINE: parts of the line, the last of whose items may go on in the next CTA; else items have CTAs of their own (ws.share).
template <int D, bool FP8, int NT, int W, bool LINE>
__global__ void __launch_bounds__(32 * W, 1)
    k_decode(const __grid_constant__ DecodeArgs a, const DecodeWs ws, const __grid_constant__ CUtensorMap map_k,
             const __grid_constant__ CUtensorMap map_v, uint64_t wait_ns) {
  using L = Lay<D, FP8, NT, W>;
  constexpr int kWarps = W;
  const int share = LINE ? 0 : max(ws.share, 0);        // CTAs of an item
  const bool whole_items = !LINE && ws.share < 0;       // ... or parts of the line that begin and end with items
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int X = gridDim.x, rb = blockIdx.y;
  const int hkv = a.c.n_kv_heads, g = a.hq / hkv, rows = g * a.q_len, cap = table_keys(a.t, a.c.page_size);
  const int n_seqs = a.t.n_seqs;
  // pieces of this warp: the one that ends the item that it began within, and the one left at its end, over the empty queue
  float* head_slot = reinterpret_cast<float*>(smem + L::AT_SLOTS + warp * L::SLOT);
  float* tail_slot = reinterpret_cast<float*>(smem + warp * L::QUEUE);
  RowSum* piece_sums = reinterpret_cast<RowSum*>(smem + L::AT_SUMS);  // [2 warp: head, 2 warp + 1: tail][row]
  int4* info = reinterpret_cast<int4*>(smem + L::AT_INFO);  // [warp]: item of the head piece, of the tail, tail begins, its last CTA
  int2* info_len = reinterpret_cast<int2*>(info + kWarps);  // ... keys of their sequences
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::AT_INFO + kWarps * 40);
  volatile uint32_t* far_rows = reinterpret_cast<volatile uint32_t*>(smem + L::AT_INFO + kWarps * 40 + 16) + warp;  // of the item: see `convert`
  const uint32_t bars = smem_u32(smem + L::AT_BARS) + warp * L::STAGES * 8;
  if (lane < L::STAGES)
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bars + lane * 8), "r"(arrivals(lane, L::STAGES, wait_ns)) : "memory");
  if (threadIdx.x == 0) *abort_flag = 0;
  tc::fence_mbar_init();
  __syncthreads();  // the flag may hold anything before, and another lane than that which prepared a barrier may use it
  grid_dep_wait();
  grid_dep_trigger();  // the joining kernel may start when CTAs leave; it reads nothing of this one before it has ended

  // ---- the warp's part of the line of tiles
  const int own = share ? blockIdx.x / share : 0, rank = share ? blockIdx.x - own * share : 0;  // item, and which of its CTAs
  int b0 = own / hkv;
  int lens = (b0 & ~31) + lane < n_seqs ? a.lens[(b0 & ~31) + lane] : 0;  // of the 32 sequences that b0 is among
  const int lens2 = lane + 32 < n_seqs ? a.lens[lane + 32] : 0;
  int64_t upto = 0, before = 0, total = 0, first32 = 0;  // tiles up to and with a lane's sequence, before the 32, of all
  const int chunks = share ? 0 : (n_seqs + 31) / 32;
  int64_t* sums = reinterpret_cast<int64_t*>(smem);
  if (chunks > 2) {  // a sum for each 32 sequences
    for (int ch = warp; ch < chunks; ch += kWarps) {
      const int b = ch * 32 + lane;
      const int64_t n = warp_sum(b < n_seqs ? units_of<L::END>(a.lens[b], cap) : 0);
      if (lane == 0) sums[ch] = n;
    }
    __syncthreads();
    for (int ch = lane; ch < chunks; ch += 32) total += sums[ch];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  } else {
    upto = warp_scan(units_of<L::END>(lens, cap), lane);
    first32 = __shfl_sync(0xffffffffu, upto, 31);
    total = first32 + warp_sum(units_of<L::END>(lens2, cap));
  }
  total *= hkv;
  const int parts = parts_of(total, X, kWarps);
  // the next sequence with keys, or none; `seq_lens`: the lanes' lengths of b's 32 sequences
  auto next_seq = [&](int& b, int& seq_lens) {
    unsigned some = __ballot_sync(0xffffffffu, seq_lens > 0) & ~((2u << (b & 31)) - 1u);
    b &= ~31;
    while (!some) {
      b += 32;
      if (b >= n_seqs) return false;
      seq_lens = b + lane < n_seqs ? a.lens[b + lane] : 0;
      some = __ballot_sync(0xffffffffu, seq_lens > 0);
    }
    b += __ffs(some) - 1;
    return true;
  };
  int64_t first = 0, left = 0;
  // the tile after the part, and all tiles (LINE): read again when the part ends
  volatile int64_t* part_end = reinterpret_cast<volatile int64_t*>(smem + L::AT_INFO + kWarps * 24) + 2 * warp;
  int hk0 = 0, tile0 = 0;
  if (share) {
    hk0 = own - b0 * hkv;
    const int keys = __shfl_sync(0xffffffffu, lens, b0 & 31), n = tiles_of(keys, cap), of = max(share, 1) * kWarps, me = rank * kWarps + warp;
    tile0 = n * me / of;
    left = n * (me + 1) / of - tile0;
    if (n == 0 && rank == 0 && warp == 0) empty_rows<D>(a, g, b0, hk0, hk0 + 1, rb * L::ROWS, min((rb + 1) * L::ROWS, rows), keys);
  } else if (blockIdx.x < parts) {
    int64_t t0 = mul_div(total, blockIdx.x, parts), t1 = mul_div(total, blockIdx.x + 1, parts);
    // the item that a place on the line lies in, and the tile; the item's length
    auto find = [&](int64_t place) {
      const int64_t seq_first = mul_div(place, 1, hkv);  // the tile's place if there were one head
      if (chunks > 2) {
        for (int base = 0; base < chunks; base += 32) {
          const int64_t v = base + lane < chunks ? sums[base + lane] : 0, in = warp_scan(v, lane);
          const unsigned hit = __ballot_sync(0xffffffffu, before + in > seq_first);
          if (hit) {
            b0 = (base + __ffs(hit) - 1) * 32;
            before += __shfl_sync(0xffffffffu, in - v, __ffs(hit) - 1);
            break;
          }
          before += __shfl_sync(0xffffffffu, in, 31);
        }
        lens = b0 + lane < n_seqs ? a.lens[b0 + lane] : 0;
        upto = warp_scan(units_of<L::END>(lens, cap), lane);
      } else if (seq_first >= first32) {
        b0 = 32;
        before = first32;
        lens = lens2;
        upto = warp_scan(units_of<L::END>(lens, cap), lane);
      }
      const int at = max(__ffs(__ballot_sync(0xffffffffu, before + upto > seq_first)) - 1, 0);
      const int n = max(units_of<L::END>(__shfl_sync(0xffffffffu, lens, at), cap), 1);
      before += __shfl_sync(0xffffffffu, upto, at) - n;
      b0 = min(b0 + at, n_seqs - 1);
      const int64_t rest = max(place - before * hkv, (int64_t)0);
      hk0 = (int)min(mul_div(rest, 1, n), (int64_t)(hkv - 1));  // within bounds even if lengths change under the call
      tile0 = (int)min(rest - (int64_t)hk0 * n, (int64_t)(n - 1));
      return n;
    };
    if (whole_items) {  // on to the next begin of an item: warp 0 of the part's begin, the others of its end
      const int lens0 = lens;
      const int64_t upto0 = upto, place = warp == 0 ? t0 : t1;
      const int n = find(place);
      int64_t* bounds = reinterpret_cast<int64_t*>(smem + L::AT_INFO);
      if (lane == 0 && warp < 2) bounds[warp] = place >= total ? total : tile0 ? place - tile0 + n : place;
      __syncthreads();
      t0 = bounds[0];
      t1 = bounds[1];
      __syncthreads();
      lens = lens0;
      upto = upto0;
      before = 0;
      b0 = 0;
    }
    first = t0 + (int64_t)((uint64_t)((t1 - t0) * warp) / kWarps);
    left = t0 + (int64_t)((uint64_t)((t1 - t0) * (warp + 1)) / kWarps) - first;
    if (LINE && lane == 0) {
      part_end[0] = first + left;
      part_end[1] = total;
    }
    if (left > 0) {
      const int n = find(first);
      if (tile0 >= n - L::END) {  // within an item's end
        left -= n - tile0;
        tile0 = 0;
        if (++hk0 == hkv) {
          hk0 = 0;
          if (!next_seq(b0, lens)) left = 0;
        }
      }
    }
  }
  if (chunks > 2) {
    fence_async();  // the queues, which the copies fill, take the place of the sums
    __syncthreads();
  }

  int4 left_over = make_int4(-1, -1, 0, 0);
  int2 left_len = make_int2(0, 0);
  if (left > 0) {
    const uint32_t queue = smem_u32(smem) + warp * L::QUEUE, scale_queue = smem_u32(smem + L::AT_SCALES) + warp * L::STAGES * L::SCALES + lane * 4;
    const float* scales = FP8 ? (c < 2 ? a.c.k_scale : a.c.v_scale) : nullptr;
    const int s_key = r + 8 * (c & 1);  // the key whose scale this lane brings in: of K for c < 2, else of V

    // ---- queries of an item, fetched as they lie and then made fragments
    float rs[NT][2];
    uint32_t q[NT][L::KS][2];
    auto fetch = [&](int b, int hk) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int R = rb * L::ROWS + nt * 8 + r;
        const RowAt at = row_at(a, g, b, hk, min(R, rows - 1));
        const bf16* src = a.q + at.head * a.q_head + at.tok * a.q_tok;
#pragma unroll
        for (int s = 0; s < L::KS; ++s) {  // a step's 16 elements; with e4m3 in fours to a lane, as the codes of a 16-byte piece
          if (FP8) {
            const uint2 w = R < rows ? *reinterpret_cast<const uint2*>(src + 16 * s + 4 * c) : make_uint2(0, 0);
            q[nt][s][0] = w.x;
            q[nt][s][1] = w.y;
          } else {
            q[nt][s][0] = R < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * s + 2 * c) : 0u;
            q[nt][s][1] = R < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * s + 8 + 2 * c) : 0u;
          }
        }
      }
    };
    // fp16 under a power of two for each row, the largest element in [2^15, 2^16): bf16's 8 bits fit exactly down to 2^-17.  Rows with
    // elements below that are remembered, and their sums made key by key in the end if it can matter.
    auto convert = [&]() {
      uint32_t far = 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t big = 0, small = 0x7fff7fffu;  // of pairs: the smallest magnitude but zero, as the signed number magnitude - 0x8001
#pragma unroll
        for (int s = 0; s < L::KS; ++s) {
          big = amax2(big, amax2(q[nt][s][0], q[nt][s][1]));
          small = min_s16x2(small, min_s16x2((q[nt][s][0] | 0x80008000u) - 0x00010001u, (q[nt][s][1] | 0x80008000u) - 0x00010001u));
        }
        big = pair_bits(big);
        small = min_s16x2(small, small >> 16 | small << 16);
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        small = min_s16x2(small, __shfl_xor_sync(0xffffffffu, small, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        small = min_s16x2(small, __shfl_xor_sync(0xffffffffu, small, 2));
        const int ex = min(max((int)(big >> 23) - 127, -111), 127);
        const float down = pow2(kQueryTop - ex), up = pow2(ex) * (a.scale * kLog2e);  // 2^-15 goes to the key's scale
        const int least = max((int)((small + 1) >> 7 & 0xff), 1) - 127;  // exponent (all zeros: the lowest)
        const unsigned lost = __ballot_sync(0xffffffffu, c == 0 && big < 0x7f800000u && small != 0x7fff7fffu && least + kQueryTop - ex < -17);
        for (unsigned rest = lost; rest; rest &= rest - 1) far |= 1u << (nt * 8 + (__ffs(rest) - 1) / 4);
#pragma unroll
        for (int s = 0; s < L::KS; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            q[nt][s][i] = pack_half(__uint_as_float(q[nt][s][i] << 16) * down, __uint_as_float(q[nt][s][i] & 0xffff0000u) * down);
        rs[nt][0] = __shfl_sync(0xffffffffu, up, 8 * c);
        rs[nt][1] = __shfl_sync(0xffffffffu, up, 8 * c + 4);
      }
      if (lane == 0) *far_rows = far;
    };

    // ---- the end of the line that loads.  Lengths of 32 sequences and 32 entries of the table lie in the lanes; the
    // entries that follow are on their way while those are used.
    const int ps = a.c.page_size;
    int pb = b0, phk = hk0, pt = tile0, plen = min(max(__shfl_sync(0xffffffffu, lens, b0 & 31), 0), cap), pn = tiles_of(plen, cap);
    int ppi = pt * kTileKeys / ps, prow = pt * kTileKeys - ppi * ps;
    int held = (int)(((unsigned)plen + (ps - 1)) / ps);  // pages of the sequence
    int plens = lens;
    int load_left = (int)min(left, (int64_t)(pn - pt));  // tiles of this item that are still to be loaded
    int64_t to_load = left - load_left;                  // and what follows it
    auto entries = [&](int b, int first_page) {
      const int i = first_page + lane;
      return i < a.t.max_pages ? a.t.pages[(int64_t)b * a.t.stride + i] : -1;
    };
    // entries that follow those of pages ppi / 32 * 32 ..: of the same sequence, again its first ones, or the next sequence's
    auto following = [&]() {
      const int batch = ppi & ~31;
      if (batch + 32 < held) return entries(pb, batch + 32);
      if (held > 32 && phk + 1 < hkv) return entries(pb, 0);
      int b = pb, l = plens;
      return next_seq(b, l) ? entries(b, 0) : -1;
    };
    int ids = entries(pb, ppi & ~31), ids_after = following();
    fetch(b0, hk0);  // behind the copies it would take microseconds
    int page = __shfl_sync(0xffffffffu, ids, ppi & 31);
    const float* scale = scales;  // this lane's of the next tile
    auto scale_row = [&]() {
      if (FP8)
        scale = scales + ((unsigned)page < (unsigned)a.c.n_pages ? page * a.c.scale_page_stride + phk * a.c.scale_head_stride +
                                                                       (prow + s_key) * a.c.scale_token_stride : 0);
    };
    scale_row();
    uint32_t missing = 0;  // stages of tiles whose page does not exist
    int in_flight = 0;     // copies that have not been waited for
    bool ok = true;        // no wait ran out; else
    int lost_at = 0;       // 2 * the stage of the first that did, + its parity
    auto load = [&](int stage) {
      const uint32_t bar = bars + stage * 8;
      missing &= ~(1u << stage);
      ++in_flight;
      if ((unsigned)page < (unsigned)a.c.n_pages) {
        if (tc::elect_one()) {
          const uint32_t at = queue + stage * L::STAGE;
          expect_tx(bar, L::STAGE);
          tma_tile<L::SEGS>(at, &map_k, bar, prow, 0, phk, page);
          tma_tile<L::SEGS>(at + L::KBYTES, &map_v, bar, prow, 0, phk, page);
        }
        if (FP8) cp4(scale_queue + stage * L::SCALES, scale);  // those behind the sequence's end are not used
      } else {
        if (lane == 0) tc::mbar_arrive_addr(bar);
        missing |= 1u << stage;
      }
      // on to the next tile
      prow += kTileKeys;
      if (FP8) scale += ws.scale_step;
      if (--load_left > 0 && prow < ps) return;
      bool fresh = false;
      if (load_left > 0) {  // the next page
        prow = 0;
        fresh = (++ppi & 31) == 0;
      } else {  // the next item
        if (to_load > 0) to_load -= L::END;
        if (to_load <= 0) return;
        ppi = prow = 0;
        fresh = held > 32;
        if (++phk == hkv) {
          phk = 0;
          fresh = true;
          if (!next_seq(pb, plens)) pb = n_seqs - 1;  // only if the lengths changed meanwhile
          plen = min(max(__shfl_sync(0xffffffffu, plens, pb & 31), 0), cap);
          pn = tiles_of(plen, cap);
          held = (int)(((unsigned)plen + (ps - 1)) / ps);
        }
        load_left = (int)min(to_load, (int64_t)max(pn, 1));
        to_load -= load_left;
      }
      if (fresh) {
        ids = ids_after;
        ids_after = following();
      }
      page = __shfl_sync(0xffffffffu, ids, ppi & 31);
      scale_row();
    };
#pragma unroll 1
    for (int s = 0; s < L::STAGES - 1; ++s) {
      if (load_left > 0) load(s);
      if (FP8) cp_commit();
    }

    // ---- the end that computes
    // rows of the 8 x 8 matrices that this lane names: keys lane % 8 (+ 8 by bit 3 for K and e4m3's V, bit 4 for bf16's V), 16-byte
    // pieces of them by the other bit, under the copies' swizzle
    auto matrix_row = [&](bool key_bit3) {
      const int key = (lane & 7) + ((key_bit3 ? lane : lane >> 1) & 8), piece = (key_bit3 ? lane >> 4 : lane >> 3) & 1;
      return key * L::SEG + ((piece ^ (L::SEG == 128 ? key & 7 : (key >> 1) & 3)) << 4);
    };
    constexpr int STEPS = L::SEG / 32;  // pairs of 16-byte pieces of a box's row
    uint32_t k_row[STEPS], v_row[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      k_row[i] = matrix_row(true) ^ (32 * i);
      v_row[i] = matrix_row(FP8) ^ (32 * i);
    }
    int cb = b0, chk = hk0, ct = tile0, raw = __shfl_sync(0xffffffffu, lens, b0 & 31), len = min(max(raw, 0), cap), cn = tiles_of(len, cap);
    int stage = 0;
    uint32_t parity = 0;
    float m[NT][2], l[NT][2], mv[NT][2], acc[NT][L::MT][4];  // mv: the reference of the weights with values' scales in them, less m
    int see[NT][2];  // a row sees keys before len + see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) see[nt][e] = min((rb * L::ROWS + nt * 8 + 2 * c + e) / g, a.q_len - 1) - a.q_len + 1;
    while (left > 0) {
      if (FP8) convert();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = kLowest;
          mv[nt][e] = l[nt][e] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < L::MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[nt][mt][i] = 0.f;
      }
      const int begin = ct;
      const int all_seen = max(len - a.q_len + 1, 0) / kTileKeys;    // tiles before this are seen by every row
      const int partial = len % kTileKeys ? cn - 1 : -1;             // a tile that the sequence ends in
      int tiles = (int)min(left, (int64_t)max(cn - ct, 1));
      left -= tiles;
      // ---- its tiles
      do {
        __syncwarp();  // all lanes have read the stage that is loaded next
        if (load_left > 0 && ok) load(stage == 0 ? L::STAGES - 1 : stage - 1);
        if (FP8) {
          cp_commit();
          cp_wait<L::STAGES - 1>();
        }
        const uint32_t at = queue + stage * L::STAGE;
        if (ok) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait_addr(bars + stage * 8, parity, abort_flag, wait_ns));
          if (ok) --in_flight;
          else lost_at = 2 * stage + parity;
        }
        const bool lost = !ok || (missing >> stage & 1);  // a wait ran out, or the page does not exist
        if (ct == partial) {  // rows behind the sequence's end may hold anything: the values' become zeros
          for (int i = len % kTileKeys * (L::SEG / 16) + lane; i < kTileKeys * (L::SEG / 16); i += 32)
#pragma unroll
            for (int sg = 0; sg < L::SEGS; ++sg)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + L::KBYTES + sg * (kTileKeys * L::SEG) + i * 16), "r"(0) : "memory");
          fence_async();  // a later copy may fill them
          __syncwarp();
        }
        float x[NT][4];
        {
          float s2[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[nt][i] = s2[nt][i] = 0.f;
          uint32_t from[STEPS];
#pragma unroll
          for (int i = 0; i < STEPS; ++i) from[i] = at + k_row[i];
          each<L::ROWB / 32>([&](auto jc) {  // two 16-byte pieces: keys 0-7, 8-15 of the first, of the second
            constexpr int j = decltype(jc)::value;
            uint32_t w[4];
            ldm4<j / STEPS * (kTileKeys * L::SEG)>(w, from[j % STEPS]);
            if constexpr (FP8) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t a0, a1, a2, a3;
                e4m3x4(w[2 * i], a0, a2);
                e4m3x4(w[2 * i + 1], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma<FP8>(i ? s2[nt] : x[nt], a0, a1, a2, a3, q[nt][2 * j + i][0], q[nt][2 * j + i][1]);
              }
            } else {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<FP8>(j & 1 ? s2[nt] : x[nt], w[0], w[1], w[2], w[3], q[nt][j][0], q[nt][j][1]);
            }
          });
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[nt][i] += s2[nt][i];
        }
        // ---- weights.  x: products of keys r (0, 1) and r + 8 (2, 3) with rows 2 c and 2 c + 1, times the key's scale; a score in units
        // of log2 is x * rs.  d, dv: scores relative to the references, dv with the value's scale in it (e4m3).
        float d[NT][4], dv[NT][4], lv[2];
        if (FP8) {
          // (exact for scales from 2^-111 on, and kv_write makes none below 2^-109; to take 2^-15 from the products instead costs 1 to 2%
          // with 16 rows)
          const float sc = lds32(scale_queue + stage * L::SCALES), lg = fast_log2(sc), sk = sc * pow2(-kQueryTop);
          const float ks[2] = {__shfl_sync(0xffffffffu, sk, lane & 28), __shfl_sync(0xffffffffu, sk, (lane & 28) + 1)};
          lv[0] = __shfl_sync(0xffffffffu, lg, (lane & 28) + 2);
          lv[1] = __shfl_sync(0xffffffffu, lg, (lane & 28) + 3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[nt][i] *= ks[i >> 1];
        }
        const bool some_hidden = ct >= all_seen || lost;
        auto relative = [&]() {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // (two roundings: equal keys have equal scores, and the largest of a row is 0 however large it is)
              d[nt][i] = __fsub_rn(__fmul_rn(x[nt][i], FP8 ? rs[nt][i & 1] : a.scale * kLog2e), m[nt][i & 1]);
              if (FP8) dv[nt][i] = d[nt][i] + (lv[i >> 1] - mv[nt][i & 1]);
            }
          if (some_hidden) {
            const float nan = lost ? __uint_as_float(0x7fffffffu) : 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const bool in = ct * kTileKeys + r + 8 * (i >> 1) < len + see[nt][i & 1];
                d[nt][i] = in ? d[nt][i] + nan : -INFINITY;
                if (FP8) dv[nt][i] = in ? dv[nt][i] + nan : -INFINITY;
              }
          }
        };
        relative();
        float most = d[0][0], most_v = dv[0][0];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          most = fmax3(most, d[nt][0], fmax3(d[nt][1], d[nt][2], d[nt][3]));
          if (FP8) most_v = fmax3(most_v, dv[nt][0], fmax3(dv[nt][1], dv[nt][2], dv[nt][3]));
        }
        if (__any_sync(0xffffffffu, most > kSlack || (FP8 && most_v > kSlackV + kShiftV))) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float by = FP8 ? rs[nt][e] : a.scale * kLog2e;
              float top = m[nt][e], score[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                score[i] = d[nt][e + 2 * i] == -INFINITY ? -INFINITY : __fmul_rn(x[nt][e + 2 * i], by);
                top = fmaxf(top, score[i]);
              }
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
              const float step = m[nt][e] - top;
              m[nt][e] = top;
              float f = fast_exp2(step);
              l[nt][e] *= f;
              if (FP8) {
                float top_v = mv[nt][e] + kShiftV + step;  // less the new m, so that a large score takes no bits of it
#pragma unroll
                for (int i = 0; i < 2; ++i) top_v = fmaxf(top_v, score[i] - top + lv[i]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, off));
                f = fast_exp2(step + mv[nt][e] - (top_v - kShiftV));
                mv[nt][e] = top_v - kShiftV;
              }
#pragma unroll
              for (int mt = 0; mt < L::MT; ++mt) {
                acc[nt][mt][e] *= f;
                acc[nt][mt][e + 2] *= f;
              }
            }
          relative();
        }
        uint32_t hi[NT][2], lo[NT][2];  // P^T: rows r, keys 2 c, 2 c + 1 (0) and + 8 (1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = fast_exp2(d[nt][2 * i]), p1 = fast_exp2(d[nt][2 * i + 1]);
            l[nt][0] += p0;
            l[nt][1] += p1;
            if (FP8) {
              hi[nt][i] = transpose8(pack_half(fast_exp2(dv[nt][2 * i]), fast_exp2(dv[nt][2 * i + 1])));
            } else {
              const uint32_t h = pack_bf16(p0, p1);
              hi[nt][i] = transpose8(h);
              lo[nt][i] = transpose8(pack_bf16(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u)));
            }
          }
        // ---- O^T += V^T P^T
        uint32_t from[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) from[i] = at + v_row[i];
        if constexpr (FP8) {
          each<L::MT / 2>([&](auto jc) {  // pieces 2 j, 2 j + 1: pairs of elements by pairs of keys
            constexpr int j = decltype(jc)::value;
            uint32_t w[4];
            ldm4_trans<L::KBYTES>(w, from[j]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t a0, a1, a2, a3;
              e4m3x4(__byte_perm(w[2 * i], 0, 0x3120), a0, a1);
              e4m3x4(__byte_perm(w[2 * i + 1], 0, 0x3120), a2, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<FP8>(acc[nt][2 * j + i], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
            }
          });
        } else {
          each<L::MT>([&](auto mc) {
            constexpr int mt = decltype(mc)::value;
            uint32_t w[4];
            ldm4_trans<L::KBYTES + mt / STEPS * (kTileKeys * L::SEG)>(w, from[mt % STEPS]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma<FP8>(acc[nt][mt], w[0], w[1], w[2], w[3], hi[nt][0], hi[nt][1]);
              mma<FP8>(acc[nt][mt], w[0], w[1], w[2], w[3], lo[nt][0], lo[nt][1]);
            }
          });
        }
        if (++stage == L::STAGES) {
          stage = 0;
          parity ^= 1;
        }
        ++ct;
      } while (--tiles > 0);

      // ---- the piece ends: whole items are done, others wait in shared memory
      const bool begins = begin == 0, ends = ct == cn, whole = begins && ends;
      float* slot = ends ? head_slot : tail_slot;
      const int item = cb * hkv + chk;
      if (!ends) {
        drain(bars, L::STAGES, lost_at >> 1, lost_at & 1, in_flight, drain_ns(wait_ns));
        in_flight = 0;
        if (FP8) cp_wait<0>();
        left_over.y = item;
        left_len.y = len;
        left_over.z = begins;
        __syncwarp();
        if constexpr (LINE) {  // the CTA whose part holds the item's last tile
          const int64_t next = part_end[0], all = part_end[1];
          left_over.w = last_part(max(next + cn - ct, next), all, parts_of(all, X, kWarps));
        }
      } else if (!whole) {
        left_over.x = item;
        left_len.x = len;
      }
      __syncwarp();
      uint32_t again = 0;  // rows (8 nt + row) whose sums have to be made once more
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float by[2];  // what o's sums are multiplied with
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[nt][e], zero = 0.f;
#pragma unroll
          for (int mt = 0; mt < L::MT; ++mt) zero = acc[nt][mt][e] * 0.f + (acc[nt][mt][e + 2] * 0.f + zero);  // or NaN
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          const int row = nt * 8 + 2 * c + e, R = rb * L::ROWS + row;
          unsigned bad = __ballot_sync(0xffffffffu, zero != 0.f && fabsf(sum) < INFINITY && R < rows);
          bad |= bad >> 16;
          bad |= bad >> 8;
          bad |= bad >> 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) again |= (bad >> i & 1) << (nt * 8 + 2 * i + e);
          if (raw > cap) sum = __uint_as_float(0x7fffffffu);
          by[e] = FP8 ? fast_exp2(mv[nt][e]) : 1.f;
          if (whole) {
            by[e] /= sum;
            if (a.lse && r == 0 && R < rows) {
              const RowAt at = row_at(a, g, cb, chk, R);
              a.lse[at.head * n_seqs * a.q_len + at.tok] = len + see[nt][e] <= 0 ? -INFINITY : row_lse(m[nt][e], sum);
            }
          } else {
            float* dst = slot + row * D + (FP8 ? 2 * r : r);
#pragma unroll
            for (int mt = 0; mt < L::MT; ++mt) {
              if (FP8) {
                *reinterpret_cast<float2*>(dst + 16 * mt) = make_float2(acc[nt][mt][e] * by[e], acc[nt][mt][e + 2] * by[e]);
              } else {
                dst[16 * mt] = acc[nt][mt][e];
                dst[16 * mt + 8] = acc[nt][mt][e + 2];
              }
            }
            if (r == 0) piece_sums[(2 * warp + !ends) * L::ROWS + row] = RowSum{m[nt][e], sum};
          }
        }
        if (whole) {  // a lane gets neighbouring elements of one row: of row r by a transposition, of rows 2 c, 2 c + 1 with e4m3
#pragma unroll
          for (int e = 0; e < (FP8 ? 2 : 1); ++e) {
            const int R = rb * L::ROWS + nt * 8 + (FP8 ? 2 * c + e : r), Rin = min(R, rows - 1);
            const RowAt at = row_at(a, g, cb, chk, Rin);
            const bool none = len - a.q_len + 1 + Rin / g <= 0;
            bf16* o = a.o + at.head * a.o_head + at.tok * a.o_tok + (FP8 ? 2 * r : 2 * c);
#pragma unroll
            for (int mt = 0; mt < L::MT; ++mt) {
              if (FP8) {
                const uint32_t w = pack_bf16(acc[nt][mt][e] * by[e], acc[nt][mt][e + 2] * by[e]);
                if (R < rows) *reinterpret_cast<uint32_t*>(o + 16 * mt) = none ? 0u : w;
              } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t w = transpose8(pack_bf16(acc[nt][mt][2 * i] * by[0], acc[nt][mt][2 * i + 1] * by[1]));
                  if (R < rows) *reinterpret_cast<uint32_t*>(o + 16 * mt + 8 * i) = none ? 0u : w;
                }
              }
            }
          }
        }
      }
      __syncwarp();
      uint32_t far = FP8 ? *far_rows : 0;
      if (far) {
        // What fp16 leaves of such a row's small elements is within 2^-25, so a score in units of log2 within D 2^-25 448 times its two scales.
        // Below 2^-20 no weight shows it: channels that are dead, not one that towers over the others, and nothing has to be made anew.
        const float most = most_key_scale(a, cb, chk, begin * kTileKeys, (int)min((int64_t)ct * kTileKeys, (int64_t)len)) * pow2(-kQueryTop);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            unsigned fine = __ballot_sync(0xffffffffu, r == 0 && fabsf(rs[nt][e]) * most * (D * 448.f * pow2(-25)) < pow2(-20));
            for (; fine; fine &= fine - 1) far &= ~(1u << (nt * 8 + 2 * (__ffs(fine) - 1) + e));
          }
        again |= far;
      }
      if (again) {
        constexpr int E = D / 32;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            if (!(again >> (nt * 8 + i) & 1)) continue;
            const int row = nt * 8 + i, R = rb * L::ROWS + row;
            const RowAt at = row_at(a, g, cb, chk, R);
            const int end = (int)min((int64_t)ct * kTileKeys, (int64_t)(len - a.q_len + 1 + R / g));
            float out[E];
            const RowSum sum = redo<D, FP8>(a, cb, chk, at, begin * kTileKeys, end, out);
            __syncwarp();
            if (raw > cap) continue;  // NaN
            if (!whole) {
#pragma unroll
              for (int e = 0; e < E; ++e) slot[row * D + lane * E + e] = out[e];
              if (lane == 0) piece_sums[(2 * warp + !ends) * L::ROWS + row] = sum;
            } else if (end > 0) {
              bf16* o = a.o + at.head * a.o_head + at.tok * a.o_tok + lane * E;
              const float inv = 1.f / sum.l;
#pragma unroll
              for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16(out[e] * inv, out[e + 1] * inv);
              if (a.lse && lane == 0) a.lse[at.head * n_seqs * a.q_len + at.tok] = row_lse(sum.m, sum.l);
            }
          }
      }
      // ---- on to the next item
      if (ends) left -= L::END;
      if (left > 0 && ends) {
        ct = 0;
        if (++chk == hkv) {
          chk = 0;
          if (!next_seq(cb, lens)) cb = n_seqs - 1;
          raw = __shfl_sync(0xffffffffu, lens, cb & 31);
          len = min(max(raw, 0), cap);
          cn = tiles_of(len, cap);
        }
        fetch(cb, chk);
      }
    }
    drain(bars, L::STAGES, lost_at >> 1, lost_at & 1, in_flight, drain_ns(wait_ns));
    if (FP8) cp_wait<0>();
  }

  // ---- the CTA's pieces, in order: lane i of every warp has piece i (2 warp: head, 2 warp + 1: tail).  Runs of one item are
  // joined.
  if (lane == 0) {
    info[warp] = left_over;
    info_len[warp] = left_len;
  }
  __syncthreads();
  int4 meta = make_int4(-1, -1, 0, 0);
  const int64_t place = (int64_t)rb * X + blockIdx.x;
  static_assert(2 * kWarps <= 32, "a piece to a lane");
  const int4 mine = lane < 2 * kWarps ? info[lane >> 1] : make_int4(-1, -1, 0, 0);
  const int2 my_len = lane < 2 * kWarps ? info_len[lane >> 1] : make_int2(0, 0);
  const int my_item = lane & 1 ? mine.y : mine.x;
  const unsigned valid = __ballot_sync(0xffffffffu, my_item >= 0), below = valid & ((1u << lane) - 1u);
  const int prev = __shfl_sync(0xffffffffu, my_item, below ? 31 - __clz(below) : 0);
  unsigned starts = __ballot_sync(0xffffffffu, my_item >= 0 && (!below || prev != my_item));
  constexpr int RB = NT;  // rows at a time
  // with several CTAs to an item: what this one leaves, beside the pieces
  float* cta_o = reinterpret_cast<float*>(smem + L::SLOT);
  RowSum* cta_sums = reinterpret_cast<RowSum*>(smem + L::QUEUE + L::SLOT);
  const int groups = (min(L::ROWS, rows - rb * L::ROWS) + RB - 1) / RB;  // units of work of a run: the warps take them in turns
#pragma unroll 1
  for (int i = 0; starts; ++i) {
    const int s = __ffs(starts) - 1;
    starts &= starts - 1;
    const unsigned run = valid & ~((1u << s) - 1u) & (starts ? (1u << (__ffs(starts) - 1)) - 1u : 0xffffffffu);
    const int last = 31 - __clz(run), item = __shfl_sync(0xffffffffu, my_item, s);
    const bool begins = (s & 1) && __shfl_sync(0xffffffffu, mine.z, s), ends = !(last & 1);
    if (!ends) {
      meta.y = item;
      meta.z = begins;
      meta.w = __shfl_sync(0xffffffffu, mine.w, last);
    } else if (!begins) {
      meta.x = item;
    }
    constexpr int E = D / 32;  // elements of a lane
    const int b = item / hkv, hk = item - b * hkv, len = __shfl_sync(0xffffffffu, lane & 1 ? my_len.y : my_len.x, s);
#pragma unroll 1
    for (int row0 = (warp + kWarps - i * groups % kWarps) % kWarps * RB; row0 < groups * RB; row0 += kWarps * RB) {
      RowSum sum[RB];
      float o[RB][E];
#pragma unroll
      for (int k = 0; k < RB; ++k) {
        sum[k] = RowSum{kLowest, 0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) o[k][e] = 0.f;
      }
#pragma unroll 1
      for (unsigned rest = run; rest;) {  // two pieces at a time
        RowSum ps[2][RB];
        float v[2][RB][E];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool in = rest;
          const int p = in ? __ffs(rest) - 1 : s;
          rest &= rest - 1;
          const uint32_t at = smem_u32(smem) + (p & 1 ? (p >> 1) * L::QUEUE : L::AT_SLOTS + (p >> 1) * L::SLOT);
#pragma unroll
          for (int k = 0; k < RB; ++k) {
            ps[j][k] = piece_sums[p * L::ROWS + row0 + k];
            lds_floats<E>(v[j][k], at + ((row0 + k) * D + lane * E) * 4);
            if (!in) {
              ps[j][k] = RowSum{kLowest, 0.f};
#pragma unroll
              for (int e = 0; e < E; ++e) v[j][k][e] = 0.f;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < RB; ++k) {
          const float top = fmaxf(fmaxf(ps[0][k].m, ps[1][k].m), sum[k].m);
          const float f = fast_exp2(sum[k].m - top), f0 = fast_exp2(ps[0][k].m - top), f1 = fast_exp2(ps[1][k].m - top);
          sum[k] = RowSum{top, sum[k].l * f + ps[0][k].l * f0 + ps[1][k].l * f1};
#pragma unroll
          for (int e = 0; e < E; ++e) o[k][e] = o[k][e] * f + v[0][k][e] * f0 + v[1][k][e] * f1;
        }
      }
#pragma unroll
      for (int k = 0; k < RB; ++k) {
        const int row = row0 + k, R = rb * L::ROWS + row;
        if (R >= rows) break;
        if (begins && ends) {
          const bool none = len - a.q_len + 1 + R / g <= 0;
          const RowAt at = row_at(a, g, b, hk, R);
          const float inv = 1.f / sum[k].l;
          uint32_t w[E / 2];
#pragma unroll
          for (int e = 0; e < E; e += 2) w[e / 2] = none ? 0u : pack_bf16(o[k][e] * inv, o[k][e + 1] * inv);
          uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + at.head * a.o_head + at.tok * a.o_tok + lane * E);
          if (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[E / 2 - 1]);
          else *dst = w[0];
          if (a.lse && lane == 0) a.lse[at.head * n_seqs * a.q_len + at.tok] = none ? -INFINITY : row_lse(sum[k].m, sum[k].l);
        } else if (share) {
          float* dst = cta_o + row * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; ++e) dst[e] = o[k][e];
          if (lane == 0) cta_sums[row] = sum[k];
        } else {
          const int64_t at = (place * 2 + (ends ? 0 : 1)) * L::ROWS + row;
          float* dst = ws.acc + at * D + lane * E;
          if (E == 4) *reinterpret_cast<float4*>(dst) = make_float4(o[k][0], o[k][1], o[k][E - 2], o[k][E - 1]);
          else *reinterpret_cast<float2*>(dst) = make_float2(o[k][0], o[k][1]);
          if (lane == 0) ws.sums[at] = sum[k];
        }
      }
    }
  }
  if (whole_items) {  // no other kernel writes the rows of empty sequences
    empty_sequences<D>(a, g, cap, blockIdx.x * kWarps + warp, X * kWarps, rb * L::ROWS, min((rb + 1) * L::ROWS, rows));
  } else if (!share) {
    if (threadIdx.x == 0) ws.meta[place] = meta;
  } else if (share > 1) {  // the item's CTAs are a cluster: each joins some of the rows, in order
    constexpr int E = D / 32;
    if (valid == 0 || (meta.x < 0 && meta.y < 0))  // nothing left: no tiles, or all of them and the rows are written
      for (int row = threadIdx.x; row < L::ROWS; row += 32 * kWarps) cta_sums[row] = RowSum{kLowest, -1.f};
    tc::cluster_sync();
#pragma unroll 1
    for (int row = warp * share + rank; row < min(L::ROWS, rows - rb * L::ROWS); row += kWarps * share) {
      RowSum sum{kLowest, 0.f};
      float o[E] = {};
      bool some = false;
#pragma unroll 1
      for (int i = 0; i < share; i += 2) {  // two at a time
        RowSum part[2];
        float v[2][E];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          ld_cluster<2>(reinterpret_cast<float*>(&part[j]), tc::mapa_cluster(smem_u32(cta_sums + row), i + j));
          ld_cluster<E>(v[j], tc::mapa_cluster(smem_u32(cta_o + row * D + lane * E), i + j));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (part[j].l == -1.f) continue;
          some = true;
          const float top = fmaxf(sum.m, part[j].m), f = fast_exp2(sum.m - top), f1 = fast_exp2(part[j].m - top);
          sum = RowSum{top, sum.l * f + part[j].l * f1};
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = o[e] * f + v[j][e] * f1;
        }
      }
      if (some) {
        const int R = rb * L::ROWS + row, keys = min(__shfl_sync(0xffffffffu, lens, b0 & 31), cap);
        const bool none = keys - a.q_len + 1 + R / g <= 0;
        const RowAt at = row_at(a, g, b0, own - b0 * hkv, R);
        const float inv = 1.f / sum.l;
        bf16* dst = a.o + at.head * a.o_head + at.tok * a.o_tok + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = none ? 0u : pack_bf16(o[e] * inv, o[e + 1] * inv);
        if (a.lse && lane == 0) a.lse[at.head * n_seqs * a.q_len + at.tok] = none ? -INFINITY : row_lse(sum.m, sum.l);
      }
    }
    tc::cluster_sync();  // the others have read this one's sums
  }
}

// Joins what an item left in several CTAs, in order; one block for each CTA in which an item begins that goes on, and each row.
// Sequences without keys get their zeros here.
//
// ROWS 8: a warp to a row, for the short chains of many items (the rest of a block's rows would only be launched to leave);
// ROWS 1: all warps share a row's pieces, for the long chains of few.
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) k_decode_join(const __grid_constant__ DecodeArgs a, const DecodeWs ws, int block_rows) {
  constexpr int LN = D / 4, GR = kJoinThreads / LN / ROWS, AHEAD = ROWS == 1 ? 5 : 4;  // lanes and groups of a row, pieces in flight
  __shared__ float4 part[ROWS == 1 ? GR : 1][LN];
  __shared__ RowSum part_sums[GR];
  const int tid = threadIdx.x, warp = tid >> 5, x = blockIdx.x, X = gridDim.x;
  const int hkv = a.c.n_kv_heads, g = a.hq / hkv, rows = g * a.q_len, n_seqs = a.t.n_seqs, cap = table_keys(a.t, a.c.page_size);
  // lengths were there before the kernel that this one follows began
  empty_sequences<D>(a, g, cap, x * (kJoinThreads / 32) + warp, X * (kJoinThreads / 32), blockIdx.y * ROWS, min((int)(blockIdx.y + 1) * ROWS, rows));
  const int R = blockIdx.y * ROWS + (ROWS == 1 ? 0 : tid / (kJoinThreads / ROWS));
  const int rb = R / block_rows, row = R - rb * block_rows;
  grid_dep_wait();
  const int64_t place = (int64_t)rb * X + x;
  const int4 me = ws.meta[place];
  if (me.y < 0 || !me.z || R >= rows) return;
  // pieces 0 .. n - 2 are what CTAs from x on left unfinished, the last is what the item's last CTA began with
  const int n = min(me.w, X - 1) - x + 1, grp = tid % (kJoinThreads / ROWS) / LN, d = tid % LN;
  const int b = me.y / hkv, hk = me.y - b * hkv, len = a.lens[b];
  RowSum run{kLowest, 0.f};
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = grp; i0 < n; i0 += GR * AHEAD) {
    RowSum s[AHEAD];
    float4 v[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = i0 + j * GR;
      const int64_t at = ((place + i) * 2 + (i < n - 1)) * block_rows + row;
      s[j] = RowSum{kLowest, 0.f};
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        s[j] = ws.sums[at];
        v[j] = *reinterpret_cast<const float4*>(ws.acc + at * D + d * 4);
      }
    }
    float top = run.m;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) top = fmaxf(top, s[j].m);
    float f = fast_exp2(run.m - top);
    run = RowSum{top, run.l * f};
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      f = fast_exp2(s[j].m - top);
      run.l += s[j].l * f;
      o = make_float4(o.x + v[j].x * f, o.y + v[j].y * f, o.z + v[j].z * f, o.w + v[j].w * f);
    }
  }
  if (ROWS == 1) {
    part[grp][d] = o;
    if (d == 0) part_sums[grp] = run;
    __syncthreads();
    if (grp) return;
    const int used = min(n, GR);
    float top = kLowest;
#pragma unroll
    for (int i = 0; i < GR; ++i) top = fmaxf(top, i < used ? part_sums[i].m : kLowest);
    run = RowSum{top, 0.f};
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      if (i >= used) break;
      const float f = fast_exp2(part_sums[i].m - top);
      const float4 v = part[i][d];
      run.l += part_sums[i].l * f;
      o = make_float4(o.x + v.x * f, o.y + v.y * f, o.z + v.z * f, o.w + v.w * f);
    }
  } else if (GR == 2) {  // two halves of a warp share a row
    const float m = __shfl_xor_sync(0xffffffffu, run.m, 16), l = __shfl_xor_sync(0xffffffffu, run.l, 16);
    const float top = fmaxf(run.m, m), f = fast_exp2(run.m - top), h = fast_exp2(m - top);
    auto both = [&](float v) { return v * f + __shfl_xor_sync(0xffffffffu, v, 16) * h; };
    run = RowSum{top, run.l * f + l * h};
    o = make_float4(both(o.x), both(o.y), both(o.z), both(o.w));
    if (grp) return;
  }
  const int seen = min(len, cap) - a.q_len + 1 + R / g;
  const RowAt at = row_at(a, g, b, hk, R);
  const float inv = 1.f / run.l;
  const uint2 w = seen <= 0 ? make_uint2(0, 0) : make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  *reinterpret_cast<uint2*>(a.o + at.head * a.o_head + at.tok * a.o_tok + d * 4) = w;
  if (a.lse && d == 0) a.lse[at.head * n_seqs * a.q_len + at.tok] = seen <= 0 ? -INFINITY : row_lse(run.m, run.l);
}

// Blocks of 16 rows where there are more than 8: 63.8 us for 16 sequences up to 32768 keys with 16 rows, 85.6 as two blocks of 8 that
// read the cache twice; 8 rows in a block of 16 take 224 us instead of 214 for 5242880 keys e4m3, and 87.5 instead of 85.9 for 1048576
// keys bf16.
DecodeShape narrow_shape(const DecodeArgs& a) {
  const int all = a.hq / a.c.n_kv_heads * a.q_len;
  const int rows = all <= 8 ? 8 : 16, blocks = (int)ceil_div(all, rows);
  return DecodeShape{rows, blocks, std::max(1, std::min(sm_count(), 1024) / blocks)};
}

// More rows of a bf16 cache may go to decode_wide.cu.  Rows of 64 elements, half the bytes of a tile, from 33 on: one sequence of 128000
// keys, 8 key heads, 69.2 us as blocks of 16 and 77.4 as one of 32 with 32 rows, 96.0 and 89.7 with 40.
bool may_be_wide(const DecodeArgs& a) { return !a.c.e4m3 && a.hq / a.c.n_kv_heads * a.q_len > (a.c.head_dim == 128 ? 16 : 32); }
DecodeShape wide_shape(const DecodeArgs& a) {
  const int all = a.hq / a.c.n_kv_heads * a.q_len;
  const int rows = all <= 32 ? 32 : 64, blocks = (int)ceil_div(all, rows);
  return DecodeShape{rows, blocks, std::max(1, std::min(sm_count(), 1024) / blocks)};
}

template <int D>
cudaError_t join(const DecodeArgs& a, const DecodeShape& sh, const DecodeWs& ws, cudaStream_t st) {
  const int rows = a.hq / a.c.n_kv_heads * a.q_len;
  // A joining block for 8 rows where items are of 8 CTAs at most, if they are alike (16 sequences of 8 heads, 16 rows: 63.8 us, 66.5 with
  // a block to a row), a block to a row where they are longer (one item of 152 CTAs: 214 us, 235 with a warp to a row).
  const bool many = (int64_t)a.t.n_seqs * a.c.n_kv_heads * 8 >= sh.ctas;
  const cudaError_t e = launch_pdl(many ? k_decode_join<D, 8> : k_decode_join<D, 1>, dim3(sh.ctas, many ? (int)ceil_div(rows, 8) : rows),
                                   dim3(kJoinThreads), 0, st, a, ws, sh.rows);
  note_launch();
  return e;
}

template <int D, bool FP8, int NT, int W>
cudaError_t run(const DecodeArgs& a, const DecodeShape& sh, DecodeWs ws, cudaStream_t st) {
  using L = Lay<D, FP8, NT, W>;
  CUtensorMap mk, mv;
  if (!tile_map<D, FP8>(&mk, a.c, a.c.k, kTileKeys, 2) || !tile_map<D, FP8>(&mv, a.c, a.c.v, kTileKeys, 2)) return cudaErrorInvalidValue;
  cudaError_t e;
  if constexpr (W == 8) {  // 16 warps are for far more keys
    // Few short sequences: a CTA or a cluster of CTAs to each item, and one launch, where the line of tiles takes two.  One CTA up to 512 keys
    // of the longest sequence that the table has room for (320 keys 6.6 us on the device, 7.1 as a cluster of 2), then as many as get 256
    // keys each, if the items are few enough.  us on the device and a call, bf16, 8 key heads, on the line, with one CTA and in clusters: 1000
    // keys 7.9 and 11.3, 9.2 and 9.8, 7.6 and 8.2; 2000 keys 8.7 and 10.2 on the line, 8.2 and 9.1 in clusters of 8 (e4m3 9.2 and 10.2, 8.7
    // and 9.5; 16 rows 13.0 and 13.5, 10.9 and 11.7); with 512 keys to a CTA, 4000 of one head, the line is as fast (9.6 and 10.3, 9.6
    // and 10.5).  Clusters of 8 find room for 12 items at once (8.8 us; 9.2 in clusters of 4), not for 16 (12.7 instead of 8.6 us): as
    // this GPU's 152 SMs are grouped.
    const int64_t items = (int64_t)a.t.n_seqs * a.c.n_kv_heads;
    const int keys = table_keys(a.t, a.c.page_size);
    int share = 1;
    while (share < 8 && keys > (share == 1 ? 512 : 256 * share) && items * sh.blocks * 2 * share <= (share == 4 ? 96 : 128)) share *= 2;
    ws.share = items <= sh.ctas && keys <= share * (FP8 || share > 1 ? 512 : 1024) ? share : 0;
    // Up to four times as many short items as CTAs: parts of the line that begin and end with items, and one launch.  bf16, keys of the longest
    // sequence: 64 sequences of 4 key heads up to 300 keys 8.6 us a call (10.3 with a second launch), 256 of 2 heads of 64 up to 500
    // 11.0 (12.0); but 64 of 8 heads up to 1000, e4m3, 15.0 (14.2), 200 of 8 heads up to 500 20.4 (19.3).
    if (!ws.share && items <= 4 * (int64_t)sh.ctas && keys <= 512) ws.share = -1;
    if (ws.share) {
      auto kfn = k_decode<D, FP8, NT, W, false>;
      e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
      if (e != cudaSuccess) return e;
      e = launch_pdl_cluster(kfn, dim3(ws.share > 0 ? (unsigned)items * ws.share : sh.ctas, sh.blocks), dim3(32 * W), L::BYTES, st,
                             std::max(ws.share, 1), a, ws, mk, mv, wait_limit_ns());
      note_launch();
      return e;
    }
  }
  auto kfn = k_decode<D, FP8, NT, W, true>;
  e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kfn, dim3(sh.ctas, sh.blocks), dim3(32 * W), L::BYTES, st, a, ws, mk, mv, wait_limit_ns());
  note_launch();
  if (e != cudaSuccess) return e;
  return join<D>(a, sh, ws, st);
}

template <int D, bool FP8>
cudaError_t run_rows(const DecodeArgs& a, const DecodeShape& sh, const DecodeWs& ws, cudaStream_t st) {
  if (sh.rows == 16) return run<D, FP8, 2, 8>(a, sh, ws, st);
  if constexpr (FP8) {
    // Converting codes takes instructions, which 16 warps overlap better; fewer warps leave fewer pieces to join where there is
    // little to read.  One sequence of 8 key heads: 4096 keys 9.3 us with 8 warps, 11.6 with 16; 262144 keys 92.7 and 93.3;
    // 524288 keys 176.7 and 172.7; 5242880 keys of one head 221 and 217.
    constexpr int kFewTiles = 1200;  // to a CTA, if all sequences were as long as the table allows
    const int64_t tiles = (int64_t)a.t.n_seqs * a.c.n_kv_heads * ceil_div(table_keys(a.t, a.c.page_size), kTileKeys);
    if (tiles > (int64_t)sh.ctas * kFewTiles) return run<D, FP8, 1, 16>(a, sh, ws, st);
  }
  return run<D, FP8, 1, 8>(a, sh, ws, st);
}

}  // namespace

size_t decode_workspace(const DecodeArgs& a) {
  auto bytes = [&](const DecodeShape& sh) {
    return (size_t)sh.ctas * sh.blocks * (sizeof(int4) + 2 * sh.rows * (sizeof(RowSum) + sizeof(float) * a.c.head_dim));
  };
  return may_be_wide(a) ? std::max(bytes(narrow_shape(a)), bytes(wide_shape(a))) : bytes(narrow_shape(a));
}

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st) {
  if (a.t.n_seqs <= 0) return cudaSuccess;
  // Tiles of 128 keys cost more to begin and to end, and pay where a CTA has enough of them, if all sequences were as long as the table
  // allows.  bf16, 8 key heads of 128, us as blocks of 16 rows and as one of 32 or 64: one sequence of 16000 keys (7 tiles to a CTA) 22.4
  // and 23.2 with 24 rows, 31.4 and 32.9 with 64; 64000 keys (26 tiles) 66.6 and 52.9, 86.7 and 63.1; 16 sequences up to 1000 keys
  // (7) 16.9 and 21.2, up to 4000 (27) 30.2 and 26.8, up to 16000 64.2 and 48.7, with 64 rows 88.4 and 55.3.  (64 up to 1000, 27
  // tiles but 8 to an item, lose: 36 and 45 with 64 rows of 64 elements.)
  constexpr int kManyTiles = 24;
  const int64_t tiles = (int64_t)a.t.n_seqs * a.c.n_kv_heads * ceil_div(table_keys(a.t, a.c.page_size), 128);
  const bool wide = may_be_wide(a) && tiles >= (int64_t)wide_shape(a).ctas * kManyTiles;
  const DecodeShape sh = wide ? wide_shape(a) : narrow_shape(a);
  const size_t places = (size_t)sh.ctas * sh.blocks;
  uint8_t* p = reinterpret_cast<uint8_t*>(a.ws);
  DecodeWs ws{};
  ws.acc = reinterpret_cast<float*>(p);
  p += places * 2 * sh.rows * sizeof(float) * a.c.head_dim;
  ws.sums = reinterpret_cast<RowSum*>(p);
  p += places * 2 * sh.rows * sizeof(RowSum);
  ws.meta = reinterpret_cast<int4*>(p);
  ws.scale_step = kTileKeys * a.c.scale_token_stride;
  if (wide) {
    const cudaError_t e = launch_decode_wide(a, sh, ws, st);
    note_launch();
    if (e != cudaSuccess) return e;
    return a.c.head_dim == 128 ? join<128>(a, sh, ws, st) : join<64>(a, sh, ws, st);
  }
  if (a.c.head_dim == 128) return a.c.e4m3 ? run_rows<128, true>(a, sh, ws, st) : run_rows<128, false>(a, sh, ws, st);
  return a.c.e4m3 ? run_rows<64, true>(a, sh, ws, st) : run_rows<64, false>(a, sh, ws, st);
}

}  // namespace upipe
