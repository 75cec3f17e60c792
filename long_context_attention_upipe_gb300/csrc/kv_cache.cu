// Writing new tokens' keys and values into the pages of a cache, and reading cached rows back.
//
//   write  bf16: the row;  e4m3: s = max|x| fp32(1 / 448) (1 below 2^-100), q = e4m3(fp32(x / s)) for each row
//   read   bf16: the row;  e4m3: bf16(q s)
//
// A row belongs to head_dim / 8 neighbouring lanes, 16 bytes of bf16 each, so its maximum is three or four
// shuffles.  The lanes of a token look its place up once and walk over heads, keys first, then values.
#include "internal.h"
#include "kv_cache.cuh"
#include "quant.cuh"

namespace upipe {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // rows of a token in flight

struct KvParams {
  KvCache c;
  PageTable t;
  KvHeads k, v;  // the bf16 side
  const int32_t *seq, *pos;
  int64_t tokens;
  int rows_per_block;  // of the 2 n_kv_heads rows of a token
};

template <bool FP8>
__global__ void __launch_bounds__(kThreads) k_kv_write(const __grid_constant__ KvParams p) {
  const int lanes = p.c.head_dim >> 3;
  const int u = threadIdx.x & (lanes - 1);
  const int64_t i = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  grid_dep_wait();
  KvPlace at{-1, 0};
  if (i < p.tokens) at = kv_place(p.c, p.t, p.seq[i], p.pos[i]);
  const bool ok = at.page >= 0;  // lanes of a token that is not written stay for the shuffles
  const int nh = p.c.n_kv_heads;
  const int r0 = blockIdx.y * p.rows_per_block, r1 = min(2 * nh, r0 + p.rows_per_block);
  for (int rb = r0; rb < r1; rb += kAhead) {
    uint4 x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = rb + j, h = r < nh ? r : r - nh;
      const KvHeads& s = r < nh ? p.k : p.v;
      x[j] = ok && r < r1 ? *reinterpret_cast<const uint4*>(s.p + h * s.head_stride + i * s.token_stride + u * 8)
                          : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = rb + j, h = r < nh ? r : r - nh;
      if (r >= r1) break;  // the same for every thread
      const int64_t row = kv_row(p.c, at, h);
      void* dst = r < nh ? p.c.k : p.c.v;
      if (!FP8) {
        if (ok) *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(dst) + row + u * 8) = x[j];
      } else {
        uint32_t m = pair_bits(amax2(x[j]));
        for (int off = lanes >> 1; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float s = block_scale(m);
        const Divisor by = divisor(s);
        const V8 f = unpack8(x[j]);
        const uint2 q = by.doubt ? quant8_divided(f, s) : quant8(f, by);
        if (ok) {
          *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(dst) + row + u * 8) = q;
          if (u == 0) (r < nh ? p.c.k_scale : p.c.v_scale)[kv_scale(p.c, at, h)] = s;
        }
      }
    }
  }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads) k_kv_read(const __grid_constant__ KvParams p) {
  const int lanes = p.c.head_dim >> 3;
  const int u = threadIdx.x & (lanes - 1);
  const int64_t i = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  grid_dep_wait();
  if (i >= p.tokens) return;
  const int seq = p.seq[i];
  if (seq < 0) return;  // padding: its rows stay as they were
  const KvPlace at = kv_place(p.c, p.t, seq, p.pos[i]);
  const bool ok = at.page >= 0;  // a row that the cache does not hold is NaN
  const int nh = p.c.n_kv_heads;
  const int r0 = blockIdx.y * p.rows_per_block, r1 = min(2 * nh, r0 + p.rows_per_block);
  for (int rb = r0; rb < r1; rb += kAhead) {
    uint4 x[kAhead];
    float s[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = rb + j, h = r < nh ? r : r - nh;
      x[j] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
      if (ok && r < r1) {
        const void* src = r < nh ? p.c.k : p.c.v;
        const int64_t row = kv_row(p.c, at, h) + u * 8;
        if (FP8) {
          const uint2 q = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(src) + row);
          x[j].x = q.x;
          x[j].y = q.y;
          s[j] = (r < nh ? p.c.k_scale : p.c.v_scale)[kv_scale(p.c, at, h)];
        } else {
          x[j] = *reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(src) + row);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = rb + j, h = r < nh ? r : r - nh;
      if (r >= r1) break;
      const KvHeads& d = r < nh ? p.k : p.v;
      if (FP8 && ok) {
        V8 f = e4m3x8(make_uint2(x[j].x, x[j].y));
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e] *= s[j];
        x[j] = pack8(f);
      }
      *reinterpret_cast<uint4*>(d.p + h * d.head_stride + i * d.token_stride + u * 8) = x[j];
    }
  }
}

template <typename K>
cudaError_t run(K kfn, const KvArgs& a, cudaStream_t st) {
  if (a.tokens <= 0) return cudaSuccess;
  KvParams p{a.c, a.t, a.k, a.v, a.seq, a.pos, a.tokens, 0};
  const int64_t bx = ceil_div(a.tokens, kThreads / (a.c.head_dim >> 3));
  // few tokens: their rows are spread over blocks too, until there are about 8 blocks per SM
  const int rows = 2 * a.c.n_kv_heads;
  const int64_t want = std::min<int64_t>(ceil_div((int64_t)sm_count() * 8, bx), rows);
  p.rows_per_block = (int)ceil_div(rows, want);
  const dim3 grid((unsigned)bx, (unsigned)ceil_div(rows, p.rows_per_block));
  const cudaError_t e = launch_pdl(kfn, grid, dim3(kThreads), 0, st, p);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_kv_write(const KvArgs& a, cudaStream_t st) {
  return run(a.c.e4m3 ? k_kv_write<true> : k_kv_write<false>, a, st);
}

cudaError_t launch_kv_read(const KvArgs& a, cudaStream_t st) {
  return run(a.c.e4m3 ? k_kv_read<true> : k_kv_read<false>, a, st);
}

}  // namespace upipe
