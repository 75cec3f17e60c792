// Attention of the newest tokens of many sequences over their cached keys and values.
//
// For query t of the T newest tokens of a sequence of len keys, over the keys j < len - T + 1 + t:
//   s_j = scale q . k_j,   lse = log sum_j exp s_j,   o = sum_j exp(s_j - lse) v_j
// and o = 0, lse = -infinity where no key is seen.
//
// The cache is read once, and that bounds the kernel: 4 T g flops for every cached byte pair (g query heads share a
// key head) are far below the tensor cores' rate.  So the split follows the bytes.  All tiles of 16 keys of all
// (sequence, key head) items form one line, in order; the CTAs take equal parts of it, and a CTA's eight warps equal
// parts of that.  A warp runs its tiles through a queue of its own in shared memory: every lane copies exactly the
// 16-byte pieces that it will read (cp.async), in the order that the matrix instructions want them, so there is no
// barrier, no bank conflict and no swizzle, and any page, head and token strides cost nothing.
//
// Per tile, with keys as the 16 rows of the matrix instruction (m16n8k16) and up to 8 (NT = 2: 16) query rows as its
// columns:   S^T = K Q^T,   P = exp2(S - m),   O^T += V^T P^T.   The order of the head dimension in the first product
// and of O's rows in the second is free; it is chosen so that a lane's 16 bytes are whole fragments.  Pairs of keys
// of V are brought together by byte permutations, P^T by one 8 x 8 transposition in registers.
//   bf16  weights enter as the sum of two bf16 numbers (2^-17), as one they would double the error of o.
//   e4m3  codes are converted to fp16 (exact), q is scaled by a power of two for each row, and V's scale joins the
//         weight's exponent, s_j + log2 sv_j, under a maximum of its own; weights are fp16 (2^-11), up to 2^15, which
//         leaves 2^-35 of the largest.
// The maximum is a reference that is raised, and the sums rescaled, only when a score exceeds it by a margin: one vote
// for each tile, no shuffles.  m, l and O are fp32.
//
// A warp's part may begin or end within an item.  The CTA joins such pieces in shared memory in order, and what an item
// leaves in several CTAs a second kernel joins in order: no atomics, equal calls give equal bits.
//
// A value that is infinite or NaN spoils the products of query rows that do not see it (zero times infinity), and of
// those that do where a weight's second part is zero.  Then o is not finite although l is, and the piece's o is summed
// again key by key (redo).
#include "internal.h"
#include "kv_cache.cuh"
#include "quant.cuh"

namespace upipe {

namespace {

constexpr int kWarps = 8;
constexpr int kTileKeys = 16;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.0e38f;  // a reference below all scores, whose difference to them is defined
constexpr float kSlack = 8.f;        // a score may exceed the reference by this, in powers of two
constexpr float kSlackV = 5.f, kShiftV = 10.f;  // fp16 weights: the reference stands for 2^10, the largest is below 2^15

// What a row of a piece (or of a joined run of pieces) leaves beside its D sums.
struct RowSum {
  float m, l;
};

template <int D, bool FP8, int NT>
struct Lay {
  static constexpr int ROWB = D * (FP8 ? 1 : 2);        // bytes of a cached row
  static constexpr int KCH = ROWB / 64;                 // 16-byte pieces of a key that a lane holds (4 lanes to a key)
  static constexpr int VB = ROWB / 8;                   // bytes of a value that a lane holds (8 lanes to a value)
  static constexpr int VCH = VB > 16 ? VB / 16 : 1;     // ... in pieces of 16 (or one of 8)
  static constexpr int VW = VB > 16 ? 16 : VB;
  static constexpr int KBYTES = 16 * ROWB;
  static constexpr int STAGE = 2 * KBYTES + (FP8 ? 128 : 0);  // keys, values, scales of a tile
  static constexpr int ROWS = 8 * NT;
  static constexpr int SLOT = ROWS * (D * 4 + (int)sizeof(RowSum));  // a piece
  static constexpr int PER_WARP = 28800;                // of 227 KB
  static constexpr int FIT = (PER_WARP - SLOT) / STAGE;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int QUEUE = STAGES * STAGE;
  static constexpr int WARP = QUEUE + SLOT;
  static constexpr int BYTES = kWarps * WARP + 256;
  static constexpr int MT = D / 16;                     // tiles of O^T
  static constexpr int KS = D / 16;                     // steps of S^T
  static_assert(STAGES >= 2 && QUEUE >= SLOT && QUEUE * kWarps >= 2048 * 8, "shared memory");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float lds32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
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

__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)two));
  return d;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
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
__device__ __forceinline__ int tiles_of(int len, int cap) { return (int)(((int64_t)min(max(len, 0), cap) + kTileKeys - 1) / kTileKeys); }

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

// The sums of one query row over the keys [k0, k1) that it sees, key by key, relative to the reference m: a lane gets
// elements lane * D / 32 .. of o.
template <int D, bool FP8>
__device__ __noinline__ void redo(const DecodeArgs& a, int b, int hk, RowAt at, int k0, int k1, float m, float* out) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float q[E], acc[E] = {};
  load_row<E, false>(a.q, at.head * a.q_head + at.tok * a.q_tok, lane * E, 1.f, q);
  for (int j = k0; j < k1; ++j) {
    const KvPlace p = kv_place(a.c, a.t, b, j);
    if (p.page < 0) continue;  // its l is NaN
    const int64_t row = kv_row(a.c, p, hk), sc = FP8 ? kv_scale(a.c, p, hk) : 0;
    float k[E], v[E], s = 0.f;
    load_row<E, FP8>(a.c.k, row, lane * E, FP8 ? a.c.k_scale[sc] : 1.f, k);
    load_row<E, FP8>(a.c.v, row, lane * E, FP8 ? a.c.v_scale[sc] : 1.f, v);
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * k[e];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float w = exp2f(s * (a.scale * kLog2e) - m);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += w * v[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = acc[e];
}

__device__ __forceinline__ float row_lse(float m, float l) { return m * kLn2 + logf(l); }

struct DecodeWs {
  int4* meta;     // [row blocks][CTAs] items of the pieces that the CTA leaves: one that ends an item, one that does not, whether
                  // the latter begins its item
  RowSum* sums;   // [row blocks][CTAs][2][rows]
  float* acc;     // [row blocks][CTAs][2][rows][D]
};

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(32 * kWarps, 1) k_decode(const __grid_constant__ DecodeArgs a, const DecodeWs ws) {
  using L = Lay<D, FP8, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int X = gridDim.x, rb = blockIdx.y;
  const int hkv = a.c.n_kv_heads, g = a.hq / hkv, rows = g * a.q_len, cap = table_keys(a.t, a.c.page_size);
  const int n_seqs = a.t.n_seqs;
  uint8_t* mine = smem + warp * L::WARP;
  float* head_acc = reinterpret_cast<float*>(mine + L::QUEUE);  // the piece that ends the item the warp began within
  float* tail_acc = reinterpret_cast<float*>(mine);             // the piece that is left at the end, over the empty queue
  int2* info = reinterpret_cast<int2*>(smem + kWarps * L::WARP);  // [warp]: item of the head piece, 2 * item + begins of the tail
  grid_dep_wait();
  grid_dep_trigger();  // the joining kernel may start when CTAs leave; it reads nothing of this one before it has ended

  // ---- the warp's part of the line of tiles
  int64_t* sums = reinterpret_cast<int64_t*>(smem);
  const int chunks = (n_seqs + 31) / 32;
  for (int ch = warp; ch < chunks; ch += kWarps) {
    const int b = ch * 32 + lane;
    const int64_t s = warp_sum(b < n_seqs ? tiles_of(a.lens[b], cap) : 0);
    if (lane == 0) sums[ch] = s;
  }
  __syncthreads();
  int64_t total = 0;
  for (int ch = lane; ch < chunks; ch += 32) total += sums[ch];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  total *= hkv;
  // no CTA gets less than a tile for each warp
  const int64_t parts = min((int64_t)X, max((total + kWarps - 1) / kWarps, (int64_t)1));
  int64_t first = 0, left = 0;
  if (blockIdx.x < parts) {
    const int64_t t0 = total * blockIdx.x / parts, t1 = total * (blockIdx.x + 1) / parts;
    first = t0 + (t1 - t0) * warp / kWarps;
    left = t0 + (t1 - t0) * (warp + 1) / kWarps - first;
  }
  int b0 = 0, hk0 = 0, tile0 = 0;
  if (left > 0) {
    int64_t before = 0;
    int ch = 0;
    for (int base = 0; base < chunks; base += 32) {
      const int64_t v = base + lane < chunks ? sums[base + lane] : 0, in = warp_scan(v, lane);
      const unsigned hit = __ballot_sync(0xffffffffu, (before + in) * hkv > first);
      if (hit) {
        ch = base + __ffs(hit) - 1;
        before += __shfl_sync(0xffffffffu, in - v, __ffs(hit) - 1);
        break;
      }
      before += __shfl_sync(0xffffffffu, in, 31);
    }
    const int b = ch * 32 + lane;
    const int64_t v = b < n_seqs ? tiles_of(a.lens[b], cap) : 0, in = warp_scan(v, lane);
    const int at = max(__ffs(__ballot_sync(0xffffffffu, (before + in) * hkv > first)) - 1, 0);
    before += __shfl_sync(0xffffffffu, in - v, at);
    b0 = ch * 32 + at;
    const int64_t n = max(__shfl_sync(0xffffffffu, v, at), (int64_t)1), rest = first - before * hkv;
    hk0 = (int)min(max(rest / n, (int64_t)0), (int64_t)(hkv - 1));  // within bounds even if lengths change under the call
    tile0 = (int)min(max(rest - hk0 * n, (int64_t)0), n - 1);
  }
  __syncthreads();  // the queues take the place of the sums

  int2 left_over = make_int2(-1, -1);
  if (left > 0) {
    // ---- places of this lane's pieces of a tile, relative to the tile's first row
    const int64_t es = FP8 ? 1 : 2, ts = a.c.token_stride * es;
    const int64_t k_off = r * ts + c * 16, v_off = 2 * c * ts + r * L::VW;
    const uint32_t queue = smem_u32(mine);
    const float* scales = FP8 ? (c < 2 ? a.c.k_scale : a.c.v_scale) : nullptr;
    const int s_key = r + 8 * (c & 1);  // the key whose scale this lane brings in: of K for c < 2, else of V

    // ---- the end of the line that loads
    int pb = b0, phk = hk0, pt = tile0, plen = min(max(a.lens[b0], 0), cap), pn = tiles_of(plen, cap);
    int ppi = pt * kTileKeys / a.c.page_size, prow = pt * kTileKeys - ppi * a.c.page_size;
    int64_t to_load = left;
    int page = a.t.pages[(int64_t)pb * a.t.stride + ppi];
    uint32_t missing = 0;  // stages whose page does not exist
    auto load = [&](int stage) {
      const uint32_t at = queue + stage * L::STAGE;
      const int keys = plen - pt * kTileKeys;  // from 16 on: a whole tile
      const bool ok = (unsigned)page < (unsigned)a.c.n_pages;
      missing = ok ? missing & ~(1u << stage) : missing | (1u << stage);
      const int64_t row = ok ? page * a.c.page_stride + phk * a.c.head_stride + prow * a.c.token_stride : 0;
      const uint8_t* k = reinterpret_cast<const uint8_t*>(a.c.k) + row * es + (ok ? k_off : 0);
      const uint8_t* v = reinterpret_cast<const uint8_t*>(a.c.v) + row * es + (ok ? v_off : 0);
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // keys r and r + 8
        const bool in = ok && r + 8 * i < keys;
        const uint8_t* p = in ? k + i * 8 * ts : reinterpret_cast<const uint8_t*>(a.c.k);
#pragma unroll
        for (int j = 0; j < L::KCH; ++j) cp16(at + (i * L::KCH + j) * 512 + lane * 16, p + j * 64, in ? 16 : 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // values 2 c, 2 c + 1, 2 c + 8, 2 c + 9
        const int key = (i & 1) + 8 * (i >> 1);
        const bool in = ok && 2 * c + key < keys;
        const uint8_t* p = in ? v + key * ts : reinterpret_cast<const uint8_t*>(a.c.v);
#pragma unroll
        for (int j = 0; j < L::VCH; ++j) {
          const uint32_t dst = at + L::KBYTES + ((i * L::VCH + j) * 32 + lane) * L::VW;
          if (L::VW == 16) cp16(dst, p + j * 128, in ? 16 : 0);
          else cp_small<8>(dst, p, in ? 8 : 0);
        }
      }
      if (FP8) {
        const bool in = ok && s_key < keys;
        const float* p = scales + (in ? page * a.c.scale_page_stride + phk * a.c.scale_head_stride +
                                            (prow + s_key) * a.c.scale_token_stride : 0);
        cp_small<4>(at + 2 * L::KBYTES + lane * 4, p, in ? 4 : 0);
      }
      // on to the next tile; its page number is on the way when it is needed
      if (--to_load > 0) {
        prow += kTileKeys;
        if (prow == a.c.page_size) {
          prow = 0;
          ++ppi;
        }
        if (++pt == pn) {
          pt = ppi = prow = 0;
          if (++phk == hkv) {
            phk = 0;
            do {
              ++pb;
              plen = pb < n_seqs ? min(max(a.lens[pb], 0), cap) : 1;
            } while (plen == 0);
            if (pb >= n_seqs) pb = n_seqs - 1;  // only if the lengths changed meanwhile
            pn = tiles_of(plen, cap);
          }
        }
        page = ppi < a.t.max_pages ? a.t.pages[(int64_t)pb * a.t.stride + ppi] : -1;
      }
    };
#pragma unroll
    for (int s = 0; s < L::STAGES - 1; ++s) {
      if (to_load > 0) load(s);
      cp_commit();
    }

    // ---- the end that computes
    int cb = b0, chk = hk0, ct = tile0, raw = a.lens[b0], len = min(max(raw, 0), cap), cn = tiles_of(len, cap);
    int stage = 0;
    float m[NT][2], l[NT][2], mv[NT][2], acc[NT][L::MT][4], rs[NT][2];
    uint32_t q[NT][L::KS][2];
    int see[NT][2];  // a row sees keys before len + see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) see[nt][e] = min((rb * L::ROWS + nt * 8 + 2 * c + e) / g, a.q_len - 1) - a.q_len + 1;
    while (left > 0) {
      // ---- an item begins: its queries
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int R = rb * L::ROWS + nt * 8 + r;
        const RowAt at = row_at(a, g, cb, chk, min(R, rows - 1));
        const bf16* src = a.q + at.head * a.q_head + at.tok * a.q_tok;
        if (!FP8) {
#pragma unroll
          for (int j = 0; j < L::KS / 2; ++j) {
            const uint4 w = R < rows ? *reinterpret_cast<const uint4*>(src + 32 * j + 8 * c) : make_uint4(0, 0, 0, 0);
            q[nt][2 * j][0] = w.x;
            q[nt][2 * j][1] = w.y;
            q[nt][2 * j + 1][0] = w.z;
            q[nt][2 * j + 1][1] = w.w;
          }
          rs[nt][0] = rs[nt][1] = a.scale * kLog2e;
        } else {
          // fp16 under a power of two for each row: bf16's 8 bits fit, elements below 2^-14 of the largest lose what fp32 sums
          // would lose
          uint4 w[L::KS / 2];
          uint32_t big = 0;
#pragma unroll
          for (int j = 0; j < L::KS / 2; ++j) {  // elements 64 (j / 2) + 16 c + 8 (j % 2) ..
            w[j] = R < rows ? *reinterpret_cast<const uint4*>(src + 64 * (j >> 1) + 16 * c + 8 * (j & 1)) : make_uint4(0, 0, 0, 0);
            big = amax2(big, amax2(w[j]));
          }
          big = pair_bits(big);
          big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
          const int ex = min(max((int)(big >> 23) - 127, -126), 126);
          const float down = pow2(-ex), up = pow2(ex) * (a.scale * kLog2e);
#pragma unroll
          for (int j = 0; j < L::KS / 2; ++j) {
            const V8 f = unpack8(w[j]);
            q[nt][2 * j][0] = pack_half(f.v[0] * down, f.v[1] * down);
            q[nt][2 * j][1] = pack_half(f.v[2] * down, f.v[3] * down);
            q[nt][2 * j + 1][0] = pack_half(f.v[4] * down, f.v[5] * down);
            q[nt][2 * j + 1][1] = pack_half(f.v[6] * down, f.v[7] * down);
          }
          rs[nt][0] = __shfl_sync(0xffffffffu, up, 8 * c);
          rs[nt][1] = __shfl_sync(0xffffffffu, up, 8 * c + 4);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = mv[nt][e] = kLowest;
          l[nt][e] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < L::MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[nt][mt][i] = 0.f;
      }
      const int begin = ct;

      // ---- its tiles
      do {
        const int ahead = stage + L::STAGES - 1;
        if (to_load > 0) load(ahead >= L::STAGES ? ahead - L::STAGES : ahead);
        cp_commit();
        cp_wait<L::STAGES - 1>();
        const uint32_t at = queue + stage * L::STAGE;
        float x[NT][4];
        {
          float s2[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[nt][i] = s2[nt][i] = 0.f;
#pragma unroll
          for (int j = 0; j < L::KCH; ++j) {
            const uint4 k0 = lds128(at + j * 512 + lane * 16), k1 = lds128(at + (L::KCH + j) * 512 + lane * 16);
            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (FP8) {
#pragma unroll
                for (int w = 0; w < 4; ++w)
                  mma<FP8>(w & 1 ? s2[nt] : x[nt], e4m3_to_half2(w0[w]), e4m3_to_half2(w1[w]), e4m3_to_half2(w0[w] >> 16),
                           e4m3_to_half2(w1[w] >> 16), q[nt][4 * j + w][0], q[nt][4 * j + w][1]);
              } else {
                mma<FP8>(x[nt], w0[0], w1[0], w0[1], w1[1], q[nt][2 * j][0], q[nt][2 * j][1]);
                mma<FP8>(s2[nt], w0[2], w1[2], w0[3], w1[3], q[nt][2 * j + 1][0], q[nt][2 * j + 1][1]);
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[nt][i] += s2[nt][i];
        }
        // ---- scores in units of log2: x of keys r (0, 1) and r + 8 (2, 3), rows 2 c and 2 c + 1; y weighs values (e4m3)
        float y[NT][4];
        float lv[2];
        if (FP8) {
          const float sc = lds32(at + 2 * L::KBYTES + lane * 4), lg = fast_log2(sc);
          const float ks[2] = {__shfl_sync(0xffffffffu, sc, lane & 28), __shfl_sync(0xffffffffu, sc, (lane & 28) + 1)};
          lv[0] = __shfl_sync(0xffffffffu, lg, (lane & 28) + 2);
          lv[1] = __shfl_sync(0xffffffffu, lg, (lane & 28) + 3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[nt][i] *= ks[i >> 1];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[nt][i] *= rs[nt][i & 1];
            if (FP8) y[nt][i] = x[nt][i] + lv[i >> 1];
          }
        const int k0 = ct * kTileKeys;
        if (k0 > len - a.q_len + 1 - kTileKeys || (missing >> stage & 1)) {
          const float lost = missing >> stage & 1 ? __uint_as_float(0x7fffffffu) : 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool in = k0 + r + 8 * (i >> 1) < len + see[nt][i & 1];
              x[nt][i] = in ? x[nt][i] + lost : -INFINITY;
              if (FP8) y[nt][i] = in ? y[nt][i] + lost : -INFINITY;
            }
        }
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            raise |= x[nt][i] > m[nt][i & 1] + kSlack;
            if (FP8) raise |= y[nt][i] > mv[nt][i & 1] + kSlackV;
          }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(x[nt][e], x[nt][e + 2]), topv = FP8 ? fmaxf(y[nt][e], y[nt][e + 2]) : 0.f;
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                if (FP8) topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, off));
              }
              top = fmaxf(top, m[nt][e]);
              float f = fast_exp2(m[nt][e] - top);
              m[nt][e] = top;
              l[nt][e] *= f;
              if (FP8) {
                topv = fmaxf(topv, mv[nt][e]);
                f = fast_exp2(mv[nt][e] - topv);
                mv[nt][e] = topv;
              }
#pragma unroll
              for (int mt = 0; mt < L::MT; ++mt) {
                acc[nt][mt][e] *= f;
                acc[nt][mt][e + 2] *= f;
              }
            }
        }
        uint32_t hi[NT][2], lo[NT][2];  // P^T: rows r, keys 2 c, 2 c + 1 (0) and + 8 (1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = fast_exp2(x[nt][2 * i] - m[nt][0]), p1 = fast_exp2(x[nt][2 * i + 1] - m[nt][1]);
            l[nt][0] += p0;
            l[nt][1] += p1;
            if (FP8) {
              hi[nt][i] = transpose8(pack_half(fast_exp2(y[nt][2 * i] - mv[nt][0] + kShiftV), fast_exp2(y[nt][2 * i + 1] - mv[nt][1] + kShiftV)));
            } else {
              const uint32_t h = pack_bf16(p0, p1);
              hi[nt][i] = transpose8(h);
              lo[nt][i] = transpose8(pack_bf16(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u)));
            }
          }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int j = 0; j < L::VCH; ++j) {
          uint32_t w[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t src = at + L::KBYTES + ((i * L::VCH + j) * 32 + lane) * L::VW;
            if (L::VW == 16) {
              const uint4 t = lds128(src);
              w[i][0] = t.x;
              w[i][1] = t.y;
              w[i][2] = t.z;
              w[i][3] = t.w;
            } else {
              const uint2 t = lds64(src);
              w[i][0] = t.x;
              w[i][1] = t.y;
            }
          }
#pragma unroll
          for (int u = 0; u < L::VW / 4; ++u) {
            if (FP8) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t x0 = __byte_perm(w[0][u], w[1][u], half ? 0x7362 : 0x5140);
                const uint32_t x8 = __byte_perm(w[2][u], w[3][u], half ? 0x7362 : 0x5140);
                const uint32_t a0 = e4m3_to_half2(x0), a1 = e4m3_to_half2(x0 >> 16), a2 = e4m3_to_half2(x8), a3 = e4m3_to_half2(x8 >> 16);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma<FP8>(acc[nt][2 * u + half], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
              }
            } else {
              const uint32_t a0 = __byte_perm(w[0][u], w[1][u], 0x5410), a1 = __byte_perm(w[0][u], w[1][u], 0x7632);
              const uint32_t a2 = __byte_perm(w[2][u], w[3][u], 0x5410), a3 = __byte_perm(w[2][u], w[3][u], 0x7632);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma<FP8>(acc[nt][4 * j + u], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
                mma<FP8>(acc[nt][4 * j + u], a0, a1, a2, a3, lo[nt][0], lo[nt][1]);
              }
            }
          }
        }
        if (++stage == L::STAGES) stage = 0;
        --left;
        ++ct;
      } while (left > 0 && ct < cn);

      // ---- the piece ends: whole items are done, others wait in shared memory
      const bool begins = begin == 0, ends = ct == cn, whole = begins && ends;
      float* slot = ends ? head_acc : tail_acc;
      RowSum* slot_sums = reinterpret_cast<RowSum*>(slot + L::ROWS * D);
      if (!ends) cp_wait<0>();  // the queue is empty
      const int item = cb * hkv + chk;
      if (!whole) (ends ? left_over.x : left_over.y) = ends ? item : 2 * item + begins;
      __syncwarp();
      uint32_t again = 0;  // rows (8 nt + row) whose o has to be summed once more
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[nt][e];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          const float back = FP8 ? fast_exp2(mv[nt][e] - m[nt][e] - kShiftV) : 1.f;
          const int row = nt * 8 + 2 * c + e, R = rb * L::ROWS + row;
          bool fine = true;
#pragma unroll
          for (int mt = 0; mt < L::MT; ++mt) {
            acc[nt][mt][e] *= back;
            acc[nt][mt][e + 2] *= back;
            fine = fine && fabsf(acc[nt][mt][e]) < INFINITY && fabsf(acc[nt][mt][e + 2]) < INFINITY;
          }
          const unsigned bad = __ballot_sync(0xffffffffu, !fine && fabsf(sum) < INFINITY && R < rows);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (bad & (0x11111111u << i)) again |= 1u << (nt * 8 + 2 * i + e);
          if (raw > cap) sum = __uint_as_float(0x7fffffffu);
          const float inv = 1.f / sum;
          if (whole) {
            if (R < rows) {
              const bool none = len + see[nt][e] <= 0;
              const RowAt at = row_at(a, g, cb, chk, R);
              bf16* o = a.o + at.head * a.o_head + at.tok * a.o_tok;
#pragma unroll
              for (int j = 0; j < L::MT / 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  w[i] = none ? 0u : pack_bf16(acc[nt][4 * j + i][e] * inv, acc[nt][4 * j + i][e + 2] * inv);
                *reinterpret_cast<uint4*>(o + (FP8 ? D / 8 * r + 8 * j : 64 * j + 8 * r)) = make_uint4(w[0], w[1], w[2], w[3]);
              }
              if (a.lse && r == 0) a.lse[at.head * n_seqs * a.q_len + at.tok] = none ? -INFINITY : row_lse(m[nt][e], sum);
            }
          } else {
#pragma unroll
            for (int j = 0; j < L::MT / 4; ++j) {
              float4* dst = reinterpret_cast<float4*>(slot + row * D + (FP8 ? D / 8 * r + 8 * j : 64 * j + 8 * r));
              dst[0] = make_float4(acc[nt][4 * j][e], acc[nt][4 * j][e + 2], acc[nt][4 * j + 1][e], acc[nt][4 * j + 1][e + 2]);
              dst[1] = make_float4(acc[nt][4 * j + 2][e], acc[nt][4 * j + 2][e + 2], acc[nt][4 * j + 3][e], acc[nt][4 * j + 3][e + 2]);
            }
            if (r == 0) slot_sums[row] = RowSum{m[nt][e], sum};
          }
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
            const float ref = __shfl_sync(0xffffffffu, i & 1 ? m[nt][1] : m[nt][0], i >> 1);
            float part = i & 1 ? l[nt][1] : l[nt][0];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
            const float inv = 1.f / __shfl_sync(0xffffffffu, part, i >> 1);
            float out[E];
            redo<D, FP8>(a, cb, chk, at, begin * kTileKeys, end, ref, out);
            __syncwarp();
            if (whole) {
              bf16* o = a.o + at.head * a.o_head + at.tok * a.o_tok + lane * E;
#pragma unroll
              for (int e = 0; e < E; e += 2)
                if (raw <= cap && end > 0) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16(out[e] * inv, out[e + 1] * inv);
            } else {
#pragma unroll
              for (int e = 0; e < E; ++e) slot[row * D + lane * E + e] = out[e];
            }
          }
      }
      // ---- on to the next item
      if (left > 0 && ends) {
        ct = 0;
        if (++chk == hkv) {
          chk = 0;
          do {
            ++cb;
            raw = cb < n_seqs ? a.lens[cb] : 1;
            len = min(max(raw, 0), cap);
          } while (len == 0);
          if (cb >= n_seqs) cb = n_seqs - 1;
          cn = tiles_of(len, cap);
        }
      }
    }
    cp_wait<0>();
  }

  // ---- the CTA's pieces, in order: runs of one item are joined
  if (lane == 0) info[warp] = left_over;
  __syncthreads();
  int4 meta = make_int4(-1, -1, 0, 0);
  int p = 0;  // pieces: 2 warp (head), 2 warp + 1 (tail)
  const int64_t place = (int64_t)rb * X + blockIdx.x;
  while (p < 2 * kWarps) {
    auto item_of = [&](int i) { return i & 1 ? (info[i >> 1].y < 0 ? -1 : info[i >> 1].y >> 1) : info[i >> 1].x; };
    const int item = item_of(p);
    if (item < 0) {
      ++p;
      continue;
    }
    const bool begins = (p & 1) && (info[p >> 1].y & 1);
    int end = p + 1, last = p;
    for (; end < 2 * kWarps; ++end) {
      const int it = item_of(end);
      if (it >= 0 && it != item) break;
      if (it == item) last = end;
      if (it == item && !(end & 1)) {
        ++end;
        break;
      }
    }
    const bool ends = !(last & 1);
    const int b = item / hkv, hk = item - b * hkv;
    for (int row = warp; row < L::ROWS && rb * L::ROWS + row < rows; row += kWarps) {
      const int R = rb * L::ROWS + row;
      constexpr int E = D / 32;
      float top = kLowest;
      auto sums_of = [&](int i) {
        return reinterpret_cast<const RowSum*>(smem + (i >> 1) * L::WARP + (i & 1 ? 0 : L::QUEUE) + L::ROWS * D * 4)[row];
      };
      for (int i = p; i <= last; ++i)
        if (item_of(i) == item) top = fmaxf(top, sums_of(i).m);
      float sum = 0.f, o[E] = {};
      for (int i = p; i <= last; ++i) {
        if (item_of(i) != item) continue;
        const RowSum s = sums_of(i);
        const float f = fast_exp2(s.m - top);
        sum += s.l * f;
        const float* src = reinterpret_cast<const float*>(smem + (i >> 1) * L::WARP + (i & 1 ? 0 : L::QUEUE)) + row * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += src[e] * f;
      }
      if (begins && ends) {
        const int seen = min(a.lens[b], cap) - a.q_len + 1 + R / g;
        const RowAt at = row_at(a, g, b, hk, R);
        bf16* dst = a.o + at.head * a.o_head + at.tok * a.o_tok + lane * E;
        const float inv = 1.f / sum;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = seen <= 0 ? 0u : pack_bf16(o[e] * inv, o[e + 1] * inv);
        if (a.lse && lane == 0) a.lse[at.head * n_seqs * a.q_len + at.tok] = seen <= 0 ? -INFINITY : row_lse(top, sum);
      } else {
        const int64_t at = (place * 2 + (ends ? 0 : 1)) * L::ROWS + row;
        float* dst = ws.acc + at * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) dst[e] = o[e];
        if (lane == 0) ws.sums[at] = RowSum{top, sum};
      }
    }
    if (!(begins && ends)) {
      if (ends) meta.x = item;
      else {
        meta.y = item;
        meta.z = begins;
      }
    }
    p = end;
  }
  if (threadIdx.x == 0) ws.meta[place] = meta;
}

// Joins what an item left in several CTAs, in order; one block for each CTA in which an item begins that goes on, and each row.
// Sequences without keys get their zeros here.
template <int D>
__global__ void __launch_bounds__(128) k_decode_join(const __grid_constant__ DecodeArgs a, const DecodeWs ws, int block_rows) {
  constexpr int E = 4, LN = D / E, GR = 128 / LN;
  __shared__ float weight[1024];
  __shared__ float4 part[GR][LN];
  __shared__ float red[4];
  __shared__ int stop;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, x = blockIdx.x, X = gridDim.x;
  const int hkv = a.c.n_kv_heads, g = a.hq / hkv, R = blockIdx.y, rb = R / block_rows, row = R - rb * block_rows, n_seqs = a.t.n_seqs;
  const int cap = table_keys(a.t, a.c.page_size);
  // lengths were there before the kernel that this one follows began
  for (int base = (x * 4 + warp) * 32; base < n_seqs; base += X * 128) {
    const int b = base + lane, len = b < n_seqs ? a.lens[b] : 1;
    unsigned none = __ballot_sync(0xffffffffu, b < n_seqs && tiles_of(len, cap) == 0);
    while (none) {
      const int i = __ffs(none) - 1;
      none &= none - 1;
      const bool lost = __shfl_sync(0xffffffffu, len, i) - a.q_len + 1 + R / g > 0;  // keys, but no table
      for (int hk = 0; hk < hkv; ++hk) {
        const RowAt at = row_at(a, g, base + i, hk, R);
        bf16* o = a.o + at.head * a.o_head + at.tok * a.o_tok;
        if (lane < D / 8) *reinterpret_cast<uint4*>(o + lane * 8) = lost ? make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu) : make_uint4(0, 0, 0, 0);
        if (a.lse && lane == 0) a.lse[at.head * n_seqs * a.q_len + at.tok] = lost ? __uint_as_float(0x7fffffffu) : -INFINITY;
      }
    }
  }
  grid_dep_wait();
  const int4* meta = ws.meta + (int64_t)rb * X;
  const int4 me = meta[x];
  if (me.y < 0 || !me.z) return;
  const int item = me.y;
  if (tid == 0) stop = -1;
  __syncthreads();
  for (int j = x + 1 + tid; j < X; j += 128)
    if (meta[j].x == item) stop = j;  // one CTA ends it
  __syncthreads();
  const int n = stop - x + 1;
  if (stop < 0 || n > 1024) return;
  auto slot = [&](int i) { return ((((int64_t)rb * X + x + i) * 2 + (i == n - 1 ? 0 : 1)) * block_rows + row); };
  float top = kLowest;
  for (int i = tid; i < n; i += 128) top = fmaxf(top, ws.sums[slot(i)].m);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (lane == 0) red[warp] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  float sum = 0.f;
  for (int i = tid; i < n; i += 128) {
    const RowSum s = ws.sums[slot(i)];
    const float f = fast_exp2(s.m - top);
    weight[i] = f;
    sum += s.l * f;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  sum = red[0] + red[1] + red[2] + red[3];
  const int grp = tid / LN, d = tid - grp * LN;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = grp; i < n; i += GR) {
    const float4 v = *reinterpret_cast<const float4*>(ws.acc + slot(i) * D + d * E);
    const float f = weight[i];
    o.x += v.x * f;
    o.y += v.y * f;
    o.z += v.z * f;
    o.w += v.w * f;
  }
  part[grp][d] = o;
  __syncthreads();
  if (grp) return;
#pragma unroll
  for (int i = 1; i < GR; ++i) {
    const float4 v = part[i][d];
    o.x += v.x;
    o.y += v.y;
    o.z += v.z;
    o.w += v.w;
  }
  const int b = item / hkv, hk = item - b * hkv;
  const int seen = min(a.lens[b], cap) - a.q_len + 1 + R / g;
  const RowAt at = row_at(a, g, b, hk, R);
  const float inv = 1.f / sum;
  const uint2 w = seen <= 0 ? make_uint2(0, 0) : make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  *reinterpret_cast<uint2*>(a.o + at.head * a.o_head + at.tok * a.o_tok + d * E) = w;
  if (a.lse && d == 0) a.lse[at.head * n_seqs * a.q_len + at.tok] = seen <= 0 ? -INFINITY : row_lse(top, sum);
}

// Rows of a block, blocks of rows, and CTAs for each of them.
struct DecodeShape {
  int rows, blocks, ctas;
};
DecodeShape decode_shape(const DecodeArgs& a) {
  const int all = a.hq / a.c.n_kv_heads * a.q_len;
  const int rows = all <= 8 ? 8 : 16, blocks = (int)ceil_div(all, rows);
  return DecodeShape{rows, blocks, std::max(1, std::min(sm_count(), 1024) / blocks)};
}

template <int D, bool FP8, int NT>
cudaError_t run(const DecodeArgs& a, const DecodeShape& sh, const DecodeWs& ws, cudaStream_t st) {
  using L = Lay<D, FP8, NT>;
  auto kfn = k_decode<D, FP8, NT>;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kfn, dim3(sh.ctas, sh.blocks), dim3(32 * kWarps), L::BYTES, st, a, ws);
  note_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_decode_join<D>, dim3(sh.ctas, a.hq / a.c.n_kv_heads * a.q_len), dim3(128), 0, st, a, ws, sh.rows);
  note_launch();
  return e;
}

template <int D, bool FP8>
cudaError_t run_rows(const DecodeArgs& a, const DecodeShape& sh, const DecodeWs& ws, cudaStream_t st) {
  return sh.rows == 8 ? run<D, FP8, 1>(a, sh, ws, st) : run<D, FP8, 2>(a, sh, ws, st);
}

}  // namespace

size_t decode_workspace(const DecodeArgs& a) {
  const DecodeShape sh = decode_shape(a);
  const size_t places = (size_t)sh.ctas * sh.blocks;
  return places * (sizeof(int4) + 2 * sh.rows * (sizeof(RowSum) + sizeof(float) * a.c.head_dim));
}

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st) {
  if (a.t.n_seqs <= 0) return cudaSuccess;
  const DecodeShape sh = decode_shape(a);
  const size_t places = (size_t)sh.ctas * sh.blocks;
  uint8_t* p = reinterpret_cast<uint8_t*>(a.ws);
  DecodeWs ws;
  ws.acc = reinterpret_cast<float*>(p);
  p += places * 2 * sh.rows * sizeof(float) * a.c.head_dim;
  ws.sums = reinterpret_cast<RowSum*>(p);
  p += places * 2 * sh.rows * sizeof(RowSum);
  ws.meta = reinterpret_cast<int4*>(p);
  if (a.c.head_dim == 128) return a.c.e4m3 ? run_rows<128, true>(a, sh, ws, st) : run_rows<128, false>(a, sh, ws, st);
  return a.c.e4m3 ? run_rows<64, true>(a, sh, ws, st) : run_rows<64, false>(a, sh, ws, st);
}

}  // namespace upipe
