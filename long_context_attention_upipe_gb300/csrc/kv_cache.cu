// Writing new tokens' keys and values into the pages of a cache, and reading cached rows back.
//
//   write  bf16: the row;  e4m3: s = max|x| fp32(1 / 448) (1 below 2^-100), q = e4m3(fp32(x / s)) for each row
//   read   bf16: the row;  e4m3: bf16(q s)
//
// A row belongs to a group of neighbouring lanes: head_dim / 8 with 16 bytes of bf16 each, or, with e4m3, head_dim / 16 with
// two such pieces half a row apart, since what a row costs beside its elements (the place, the maximum's shuffles, the scale
// and its reciprocal) then falls to half as many.  A block takes a chunk of tokens: its threads look up a token's place
// each, then a group takes one head of keys or values for a run of up to 16 tokens, several rows in flight.  Runs are as
// long as the number of tokens allows: a decode step's few tokens spread over blocks, a prompt's rows share their lookups.
// Bound by HBM for prompts (and, quantising, by the instructions beside it); a few tokens are bound by the launch.
#include "internal.h"
#include "kv_cache.cuh"
#include "quant.cuh"

namespace upipe {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxRun = 16;                             // tokens of a group
constexpr int kMaxChunk = kMaxRun * (kThreads / 4) / 2;  // of a block: two rows of one head, four lanes each

struct KvParams {
  KvCache c;
  PageTable t;
  KvHeads k, v;  // the bf16 side
  const int32_t *seq, *pos;
  int64_t tokens;
  int run, runs, rows;  // tokens of a run, runs and rows (heads of keys, then of values) of a block
};

// Where a token's rows of head 0 lie; row < 0: nowhere (-1), or padding that is left alone (-2).
struct Place {
  int64_t row, scale;
};

// Five blocks to an SM for the quantiser (112K tokens x 8 heads: 83.8 us, 6.0 TB/s; with four 93.2, with six 85.8); the others are
// given registers as the compiler likes (read of 1M tokens x 1 head from e4m3: 124 us, 6.6 TB/s; 140 at 64 registers).  Writing
// 32768 tokens x 8 heads in bf16 takes 42 us, 6.4 TB/s.
template <bool WRITE, bool FP8>
__global__ void __launch_bounds__(kThreads, WRITE && FP8 ? 5 : 1) k_kv_copy(const __grid_constant__ KvParams p) {
  constexpr int PIECES = FP8 ? 2 : 1, AHEAD = 4;
  __shared__ Place places[kMaxChunk];
  const int chunk = p.run * p.runs;
  const int64_t first = (int64_t)blockIdx.x * chunk;
  const int n = (int)min((int64_t)chunk, p.tokens - first);
  grid_dep_wait();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int seq = p.seq[first + i];
    const KvPlace at = kv_place(p.c, p.t, seq, p.pos[first + i]);
    Place q{seq < 0 ? -2 : -1, 0};
    if (at.page >= 0) q = Place{kv_row(p.c, at, 0), FP8 ? kv_scale(p.c, at, 0) : 0};
    places[i] = q;
  }
  __syncthreads();
  const int lanes = p.c.head_dim / (8 * PIECES), half = p.c.head_dim >> 1, u = threadIdx.x & (lanes - 1), grp = threadIdx.x / lanes;
  const int nh = p.c.n_kv_heads, local = grp / p.runs, r = blockIdx.y * p.rows + local;
  if (local >= p.rows || r >= 2 * nh) return;
  const int start = (grp - local * p.runs) * p.run, len = min(p.run, n - start);
  const int h = r < nh ? r : r - nh;
  const KvHeads& s = r < nh ? p.k : p.v;
  bf16* plain = s.p + h * s.head_stride + (first + start) * s.token_stride + u * 8;
  const int64_t head = h * p.c.head_stride + u * 8;
  uint8_t* codes = reinterpret_cast<uint8_t*>(r < nh ? p.c.k : p.c.v) + head;
  bf16* cached = reinterpret_cast<bf16*>(r < nh ? p.c.k : p.c.v) + head;
  float* scales = (r < nh ? p.c.k_scale : p.c.v_scale) + h * p.c.scale_head_stride;
  const unsigned group = ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
#pragma unroll 1
  for (int i = 0; i < len; i += AHEAD, plain += AHEAD * s.token_stride) {
    Place at[AHEAD];
    uint4 x[AHEAD][PIECES];
    float sc[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      at[j] = i + j < len ? places[start + i + j] : Place{-2, 0};
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        // a row that is not written counts as zeros; one that the cache does not hold reads as NaN
        x[j][k] = WRITE ? make_uint4(0, 0, 0, 0) : make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        if (at[j].row < 0) continue;
        if (WRITE) {
          x[j][k] = *reinterpret_cast<const uint4*>(plain + j * s.token_stride + k * half);
        } else if (FP8) {
          const uint2 q = *reinterpret_cast<const uint2*>(codes + at[j].row + k * half);
          x[j][k].x = q.x;
          x[j][k].y = q.y;
        } else {
          x[j][k] = *reinterpret_cast<const uint4*>(cached + at[j].row);
        }
      }
      if (FP8 && !WRITE && at[j].row >= 0) sc[j] = scales[at[j].scale];
    }
    if (WRITE && FP8) {
      uint32_t m[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) m[j] = pair_bits(amax2(amax2(x[j][0]), amax2(x[j][PIECES - 1])));
      for (int off = lanes >> 1; off > 0; off >>= 1)
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) m[j] = max(m[j], __shfl_xor_sync(group, m[j], off));
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) sc[j] = block_scale(m[j]);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (at[j].row < (WRITE ? 0 : -1)) continue;
      // Where both the row and its largest magnitude are bf16, no quotient lies so near to a border of the codes that its last bits
      // matter (checked for every pair of significands, tests/test_kv_ops_abi.py), so the scales that quant.cuh divides by, one
      // in ten for such rows, need no division here: only those from 2^60 on, infinity and NaN.
      const Divisor by = divisor(WRITE && FP8 ? sc[j] : 1.f);
      const bool divide = !(sc[j] < 1.152921504606846976e18f);
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        if (WRITE && FP8) {
          const V8 f = unpack8(x[j][k]);
          *reinterpret_cast<uint2*>(codes + at[j].row + k * half) = divide ? quant8_divided(f, sc[j]) : quant8(f, by);
        } else if (WRITE) {
          *reinterpret_cast<uint4*>(cached + at[j].row) = x[j][k];
        } else {
          if (FP8 && at[j].row >= 0) {
            V8 f = e4m3x8(make_uint2(x[j][k].x, x[j][k].y));
#pragma unroll
            for (int e = 0; e < 8; ++e) f.v[e] *= sc[j];
            x[j][k] = pack8(f);
          }
          *reinterpret_cast<uint4*>(plain + j * s.token_stride + k * half) = x[j][k];
        }
      }
    }
    if (WRITE && FP8) {  // a scale to a lane
      float mine = sc[0];
      Place to = at[0];
#pragma unroll
      for (int j = 1; j < AHEAD; ++j)
        if (u == j) {
          mine = sc[j];
          to = at[j];
        }
      if (u < AHEAD && to.row >= 0) scales[to.scale] = mine;
    }
  }
}

template <typename K>
cudaError_t run(K kfn, const KvArgs& a, cudaStream_t st) {
  if (a.tokens <= 0) return cudaSuccess;
  const int groups = kThreads * (a.c.e4m3 ? 16 : 8) / a.c.head_dim, rows = 2 * a.c.n_kv_heads;
  KvParams p{a.c, a.t, a.k, a.v, a.seq, a.pos, a.tokens, kMaxRun, 1, std::min(rows, groups)};
  p.runs = groups / p.rows;
  const int64_t by = ceil_div(rows, p.rows);
  // shorter runs until there are about 4 blocks per SM
  while (p.run > 1 && ceil_div(a.tokens, p.run * p.runs) * by < (int64_t)sm_count() * 4) p.run >>= 1;
  if (p.run == 1) p.runs = (int)std::min<int64_t>(p.runs, a.tokens);
  const cudaError_t e = launch_pdl(kfn, dim3((unsigned)ceil_div(a.tokens, p.run * p.runs), (unsigned)by), dim3(kThreads), 0, st, p);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_kv_write(const KvArgs& a, cudaStream_t st) {
  return run(a.c.e4m3 ? k_kv_copy<true, true> : k_kv_copy<true, false>, a, st);
}

cudaError_t launch_kv_read(const KvArgs& a, cudaStream_t st) {
  return run(a.c.e4m3 ? k_kv_copy<false, true> : k_kv_copy<false, false>, a, st);
}

}  // namespace upipe
