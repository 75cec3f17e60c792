// Writing new tokens' keys and values into the pages of a cache, and reading cached rows back.
//
//   write  bf16: the row;  e4m3: s = max|x| fp32(1 / 448) (1 below 2^-100), q = e4m3(fp32(x / s)) for each row
//   read   bf16: the row;  e4m3: bf16(q s)
//
// A row belongs to a group of head_dim / 8 neighbouring lanes, 16 bytes of bf16 each, so its maximum is three or four
// shuffles.  A block takes a chunk of tokens: its threads look up a token's place each, then a group takes one head of keys
// or values for a run of up to 16 tokens, several rows in flight, and writes the run's scales together.  Runs are as long as
// the number of tokens allows: a decode step's few tokens spread over blocks, a prompt's rows share their lookups.  Bound by
// HBM for prompts; a few tokens are bound by the launch.
#include "internal.h"
#include "kv_cache.cuh"
#include "quant.cuh"

namespace upipe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRun = 16, kMaxChunk = kMaxRun * kThreads / 8 / 2;  // tokens of a group, of a block (two rows of one head at least)

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

// The rows of a run, AHEAD at a time: load(j, token, place) and store(j, token, place) see the same places.
template <int AHEAD, typename Load, typename Store>
__device__ __forceinline__ void walk(const Place* places, int64_t first, int n, const Load& load, const Store& store) {
  for (int i = 0; i < n; i += AHEAD) {
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (i + j < n) load(j, first + i + j, places[i + j]);
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (i + j < n) store(j, i + j, first + i + j, places[i + j]);
  }
}

template <bool WRITE, bool FP8>
__global__ void __launch_bounds__(kThreads) k_kv_copy(const __grid_constant__ KvParams p) {
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
  const int lanes = p.c.head_dim >> 3, u = threadIdx.x & (lanes - 1), grp = threadIdx.x / lanes;
  const int nh = p.c.n_kv_heads, local = grp / p.runs, r = blockIdx.y * p.rows + local;
  if (local >= p.rows || r >= 2 * nh) return;
  const int start = (grp - local * p.runs) * p.run, len = min(p.run, n - start);
  if (len <= 0) return;
  const int h = r < nh ? r : r - nh;
  const KvHeads& s = r < nh ? p.k : p.v;
  bf16* plain = s.p + h * s.head_stride + u * 8;
  const int64_t ts = s.token_stride, head = h * p.c.head_stride + u * 8, scale_head = h * p.c.scale_head_stride;
  uint8_t* codes = reinterpret_cast<uint8_t*>(r < nh ? p.c.k : p.c.v);
  bf16* cached = reinterpret_cast<bf16*>(codes);
  float* scales = r < nh ? p.c.k_scale : p.c.v_scale;
  const unsigned group = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
  if (WRITE) {
    constexpr int AHEAD = 4;
    uint4 x[AHEAD];
    float my_scale = 1.f;  // of the run's token u
    walk<AHEAD>(
        places + start, first + start, len,
        [&](int j, int64_t tok, const Place& at) {
          x[j] = at.row >= 0 ? *reinterpret_cast<const uint4*>(plain + tok * ts) : make_uint4(0, 0, 0, 0);
        },
        [&](int j, int i, int64_t, const Place& at) {
          if (!FP8) {
            if (at.row >= 0) *reinterpret_cast<uint4*>(cached + at.row + head) = x[j];
            return;
          }
          uint32_t m = pair_bits(amax2(x[j]));
          for (int off = lanes >> 1; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(group, m, off));
          const float sc = block_scale(m);
          const Divisor by = divisor(sc);
          const V8 f = unpack8(x[j]);
          const uint2 q = by.doubt ? quant8_divided(f, sc) : quant8(f, by);
          if (at.row >= 0) *reinterpret_cast<uint2*>(codes + at.row + head) = q;
          if ((i & (lanes - 1)) == u) my_scale = sc;
          if ((i & (lanes - 1)) == lanes - 1 || i == len - 1) {  // a scale to a lane
            const int mine = (i & ~(lanes - 1)) + u;
            if (mine <= i) {
              const Place to = places[start + mine];
              if (to.row >= 0) scales[to.scale + scale_head] = my_scale;
            }
          }
        });
  } else {
    constexpr int AHEAD = FP8 ? 8 : 4;
    uint4 x[AHEAD];
    float sc[AHEAD];
    walk<AHEAD>(
        places + start, first + start, len,
        [&](int j, int64_t, const Place& at) {
          x[j] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);  // a row that the cache does not hold is NaN
          if (at.row < 0) return;
          if (FP8) {
            const uint2 q = *reinterpret_cast<const uint2*>(codes + at.row + head);
            x[j].x = q.x;
            x[j].y = q.y;
            sc[j] = scales[at.scale + scale_head];
          } else {
            x[j] = *reinterpret_cast<const uint4*>(cached + at.row + head);
          }
        },
        [&](int j, int, int64_t tok, const Place& at) {
          if (FP8 && at.row >= 0) {
            V8 f = e4m3x8(make_uint2(x[j].x, x[j].y));
#pragma unroll
            for (int e = 0; e < 8; ++e) f.v[e] *= sc[j];
            x[j] = pack8(f);
          }
          if (at.row != -2) *reinterpret_cast<uint4*>(plain + tok * ts) = x[j];
        });
  }
}

template <typename K>
cudaError_t run(K kfn, const KvArgs& a, cudaStream_t st) {
  if (a.tokens <= 0) return cudaSuccess;
  const int groups = kThreads / (a.c.head_dim >> 3), rows = 2 * a.c.n_kv_heads;
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
