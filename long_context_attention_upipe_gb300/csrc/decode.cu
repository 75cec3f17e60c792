// Attention of the newest tokens of many sequences over their cached keys and values.
//
// For query t of the T newest tokens of a sequence of len keys, over the keys j < len - T + 1 + t:
//   s_j = scale q . k_j,   lse = log sum_j exp s_j,   o = sum_j exp(s_j - lse) v_j
// and o = 0, lse = -infinity where no key is seen.
#include "internal.h"
#include "kv_cache.cuh"
#include "quant.cuh"

namespace upipe {

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Running softmax of one query row: maximum (in units of log2), sum and weighted values.
template <int E>
struct Part {
  float m, l, acc[E];
};

// Elements e0 .. e0 + E of a cached row.
template <int E, bool FP8>
__device__ __forceinline__ void load_row(const void* base, int64_t row, int e0, float scale, float (&x)[E]) {
  if (FP8) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + row + e0;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 f = e4m3x2(*reinterpret_cast<const uint16_t*>(p + i));
      x[i] = f.x * scale;
      x[i + 1] = f.y * scale;
    }
  } else {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(reinterpret_cast<const bf16*>(base) + row + e0);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 f = __bfloat1622float2(p[i >> 1]);
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  }
}

// One block for each token and query head; a warp takes every fourth key, its lanes the elements of a row.
template <int D, bool FP8>
__global__ void __launch_bounds__(32 * kWarps) k_decode_simple(const __grid_constant__ DecodeArgs a) {
  constexpr int E = D / 32;
  __shared__ Part<E> part[kWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tok = blockIdx.x;
  const int h = blockIdx.y, hk = h / (a.hq / a.c.n_kv_heads);
  const int b = (int)(tok / a.q_len), t = (int)(tok % a.q_len);
  grid_dep_wait();
  const int64_t len = a.lens[b], seen = len - a.q_len + 1 + t;
  const bool bad = len > (int64_t)a.t.max_pages * a.c.page_size;
  float q[E];
  load_row<E, false>(a.q, h * a.q_head + tok * a.q_tok, lane * E, 1.f, q);
  Part<E> me{-INFINITY, 0.f, {}};
  for (int64_t j = warp; j < seen && !bad; j += kWarps) {
    const KvPlace at = kv_place(a.c, a.t, b, (int)j);
    if (at.page < 0) {
      me.l = NAN;
      break;
    }
    const int64_t row = kv_row(a.c, at, hk), sc = FP8 ? kv_scale(a.c, at, hk) : 0;
    float k[E], v[E];
    load_row<E, FP8>(a.c.k, row, lane * E, FP8 ? a.c.k_scale[sc] : 1.f, k);
    load_row<E, FP8>(a.c.v, row, lane * E, FP8 ? a.c.v_scale[sc] : 1.f, v);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * k[e];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= a.scale * kLog2e;
    const float m = fmaxf(me.m, s), base = m == -INFINITY ? 0.f : m;
    const float keep = exp2f(me.m - base), w = exp2f(s - base);
    me.m = m;
    me.l = me.l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) me.acc[e] = me.acc[e] * keep + w * v[e];
  }
  part[warp][lane] = me;
  __syncthreads();
  if (warp) return;
  for (int w = 1; w < kWarps; ++w) {
    const Part<E>& o = part[w][lane];
    const float m = fmaxf(me.m, o.m), base = m == -INFINITY ? 0.f : m;
    const float x = exp2f(me.m - base), y = exp2f(o.m - base);
    me.m = m;
    me.l = me.l * x + o.l * y;
#pragma unroll
    for (int e = 0; e < E; ++e) me.acc[e] = me.acc[e] * x + o.acc[e] * y;
  }
  if (bad) me.l = NAN;
  float out[E];
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = seen <= 0 ? 0.f : me.acc[e] / me.l;
  bf16* o = a.o + h * a.o_head + tok * a.o_tok + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16(out[e], out[e + 1]);
  if (a.lse && lane == 0)
    a.lse[h * (int64_t)a.t.n_seqs * a.q_len + tok] = seen <= 0 ? -INFINITY : me.m * kLn2 + logf(me.l);
}

}  // namespace

size_t decode_workspace(const DecodeArgs&) { return 16; }

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st) {
  const int64_t tokens = (int64_t)a.t.n_seqs * a.q_len;
  if (tokens <= 0) return cudaSuccess;
  auto kfn = a.c.head_dim == 128 ? (a.c.e4m3 ? k_decode_simple<128, true> : k_decode_simple<128, false>)
                                 : (a.c.e4m3 ? k_decode_simple<64, true> : k_decode_simple<64, false>);
  const cudaError_t e = launch_pdl(kfn, dim3((unsigned)tokens, (unsigned)a.hq), dim3(32 * kWarps), 0, st, a);
  note_launch();
  return e;
}

}  // namespace upipe
