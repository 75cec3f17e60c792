// Global norm of many gradient tensors and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2),   out = g * min(1, max_norm / (norm + 1e-6))
// Two launches: the first sums squares (a partial sum per block, in the workspace), the second adds the
// partial sums up in every block, in the same order, and scales.  No atomics: the norm depends on the
// sizes alone, not on which block comes first.
//
// The tensors are cut into chunks, walked by a fixed number of blocks; a block takes a chunk 4096 elements at
// a time, 16 per thread, with the next 4096 in flight.  A thread squares and adds its 16 elements in fp32 and
// those sums in fp64.  Squares outside fp32's comfortable range (a sum below 1e-20 or above 1e30) are summed
// once more with the elements scaled by a power of two, which is exact, so neither tiny nor huge gradients
// lose their norm.
//
// Bound by HBM: reading twice and writing once, less what the second launch still finds in L2; it walks
// the chunks backwards, so that what was read last is read first.  Only the last 64 MB of the first launch are
// left in L2; everything else is marked to leave it first, stores and second reads too (872 MB of fp32 gradients
// into bf16: 332 us, all left to L2 340 us, nothing 330 us; 361 MB into fp32: 172, 181, 181 us).  The 64 MB are
// counted as fp32 elements and for each list of tensors: 32 MB of bf16 gradients, and of many lists every one's last,
// of which the second pass finds only the last list's.
#include "common.cuh"
#include "internal.h"

namespace upipe {

namespace {

constexpr int kClipThreads = 256;
constexpr int kPer = 16;                     // elements of a thread and step
constexpr int kStep = kClipThreads * kPer;   // 4096
constexpr int kFewTensors = 24, kSomeTensors = 120, kManyTensors = 960;  // tensors of one launch (its parameters hold the list)
constexpr int kClipBlocksPerSm = 4;
constexpr int64_t kKeepBytes = 64 << 20;  // of fp32 gradients left in L2 (129 MB) for the second launch

struct ClipEntry {
  const void* g;
  void* out;
  int64_t n;
  uint32_t chunk0;  // first chunk of this tensor in the launch's list
  uint16_t g_bf16, out_bf16;
};

template <int CAP>
struct ClipList {
  ClipEntry t[CAP];
  int count;
  uint32_t chunks;
  int chunk;     // elements of a chunk, a multiple of kStep
  int in_place;  // every tensor of the list is scaled in place
  uint32_t keep_from;  // first chunk that is to stay in L2 for the second launch
};

template <int CAP>
__device__ __forceinline__ int find_tensor(const ClipList<CAP>& l, uint32_t chunk) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.t[mid].chunk0 <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// 16 elements of this thread out of the kStep at g (`n` of them exist; zeros past that): fp32 in four runs of 4
// neighbours, bf16 in two runs of 8.  LAST: read for the last time.
template <bool LAST>
__device__ __forceinline__ uint4 load16(const void* p) {
  return LAST ? __ldcs(reinterpret_cast<const uint4*>(p)) : *reinterpret_cast<const uint4*>(p);
}
template <bool BF, bool LAST>
__device__ __forceinline__ void load_step(const void* base, int64_t off, int64_t n, uint4 (&q)[4]) {
  constexpr int RUN = BF ? 8 : 4;
#pragma unroll
  for (int i = 0; i < kPer / RUN; ++i) {
    const int at = (i * kClipThreads + threadIdx.x) * RUN;
    q[i] = make_uint4(0, 0, 0, 0);
    if (BF) {
      const bf16* g = reinterpret_cast<const bf16*>(base) + off;
      if (at + 8 <= n) q[i] = load16<LAST>(g + at);
      else if (at < n) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (at + k < n) w[k >> 1] |= (uint32_t)__bfloat16_as_ushort(g[at + k]) << (16 * (k & 1));
        q[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      const float* g = reinterpret_cast<const float*>(base) + off;
      if (at + 4 <= n) q[i] = load16<LAST>(g + at);
      else if (at < n) {
        q[i].x = __float_as_uint(g[at]);
        if (at + 1 < n) q[i].y = __float_as_uint(g[at + 1]);
        if (at + 2 < n) q[i].z = __float_as_uint(g[at + 2]);
      }
    }
  }
}

template <bool BF>
__device__ __forceinline__ void to_floats(const uint4 (&q)[4], float (&v)[kPer]) {
#pragma unroll
  for (int i = 0; i < (BF ? 2 : 4); ++i) {
    if (BF) {
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __bfloat1622float2(h[k]);
        v[8 * i + 2 * k] = f.x;
        v[8 * i + 2 * k + 1] = f.y;
      }
    } else {
      v[4 * i] = __uint_as_float(q[i].x);
      v[4 * i + 1] = __uint_as_float(q[i].y);
      v[4 * i + 2] = __uint_as_float(q[i].z);
      v[4 * i + 3] = __uint_as_float(q[i].w);
    }
  }
}

// A chunk's elements [off, off + n) step by step, the next step's loads in flight while f works on this one's.
template <bool BF, bool LAST, typename F>
__device__ __forceinline__ void walk(const void* base, int64_t off, int n, F&& f) {
  uint4 next[4];
  load_step<BF, LAST>(base, off, n, next);
#pragma unroll 1
  for (int done = 0; done < n; done += kStep) {
    float v[kPer];
    to_floats<BF>(next, v);
    if (done + kStep < n) load_step<BF, LAST>(base, off + done + kStep, n - done - kStep, next);
    f(v, done);
  }
}

__device__ __forceinline__ double sum_squares(const float (&v)[kPer]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) s += v[i] * v[i];
  if (s >= 1e-20f && s <= 1e30f) return (double)s;
  // outside the range in which fp32 squares are exact enough (or zero, infinite, NaN)
  const bool small = s < 1e-20f;
  const float up = small ? 1.2379400392853803e27f : 8.470329472543003e-22f;  // 2^90, 2^-70
  const double back = small ? 6.525304467998525e-55 : 1.3937965749081639e42;  // 2^-180, 2^140
  float s2 = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) s2 += (v[i] * up) * (v[i] * up);
  return (double)s2 * back;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kClipThreads / 32];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < kClipThreads / 32; ++i) v += red[i];
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kClipThreads, kClipBlocksPerSm) k_clip_norm(const __grid_constant__ ClipList<CAP> l, double* part) {
  double total = 0.0;
  grid_dep_wait();
  for (uint32_t c = blockIdx.x; c < l.chunks; c += gridDim.x) {
    const ClipEntry& e = l.t[find_tensor(l, c)];
    const int64_t off = (int64_t)(c - e.chunk0) * l.chunk;
    const int n = (int)min((int64_t)l.chunk, e.n - off);
    auto add = [&](const float (&v)[kPer], int) { total += sum_squares(v); };
    // what the second launch will reach only after L2 has turned over leaves L2 first
    if (c < l.keep_from) {
      if (e.g_bf16) walk<true, true>(e.g, off, n, add);
      else walk<false, true>(e.g, off, n, add);
    } else {
      if (e.g_bf16) walk<true, false>(e.g, off, n, add);
      else walk<false, false>(e.g, off, n, add);
    }
  }
  grid_dep_trigger();
  total = block_sum(total);
  if (threadIdx.x == 0) part[blockIdx.x] = total;
}

template <int CAP>
__global__ void __launch_bounds__(kClipThreads, kClipBlocksPerSm) k_clip_scale(const __grid_constant__ ClipList<CAP> l,
                                                                               const double* part, int n_part, float max_norm,
                                                                               float* norm_out) {
  grid_dep_wait();  // the partial sums are complete and visible
  double total = 0.0;
  for (int i = threadIdx.x; i < n_part; i += kClipThreads) total += part[i];
  const double norm = sqrt(block_sum(total));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  // gradients that hold an infinity or NaN are not scaled: the caller sees it in the norm and skips the step.  Finite
  // ones are, even where their norm is past fp32 and is returned as infinity.
  float coef = 1.f;
  if (norm <= 1.7976931348623157e308) coef = (float)fmin(1.0, (double)max_norm / (norm + 1e-6));
  if (coef == 1.f && l.in_place) return;
  for (uint32_t k = blockIdx.x; k < l.chunks; k += gridDim.x) {
    const uint32_t c = l.chunks - 1 - k;
    const ClipEntry& e = l.t[find_tensor(l, c)];
    if (coef == 1.f && e.out == e.g) continue;
    const int64_t off = (int64_t)(c - e.chunk0) * l.chunk;
    const int n = (int)min((int64_t)l.chunk, e.n - off);
    void* out = e.out;
    const int out_bf16 = e.out_bf16;
    // values i .. i + 3 of a thread are neighbours, from element `at` of the step on
    auto store4 = [&](int64_t at, int64_t left, float a, float b, float cc, float d) {
      if (out_bf16) {
        bf16* dst = reinterpret_cast<bf16*>(out) + off + at;
        if (left >= 4) __stcs(reinterpret_cast<uint2*>(dst), make_uint2(pack_bf16(a, b), pack_bf16(cc, d)));
        else {
          if (left > 0) dst[0] = __float2bfloat16_rn(a);
          if (left > 1) dst[1] = __float2bfloat16_rn(b);
          if (left > 2) dst[2] = __float2bfloat16_rn(cc);
        }
      } else {
        float* dst = reinterpret_cast<float*>(out) + off + at;
        if (left >= 4) __stcs(reinterpret_cast<float4*>(dst), make_float4(a, b, cc, d));
        else {
          if (left > 0) dst[0] = a;
          if (left > 1) dst[1] = b;
          if (left > 2) dst[2] = cc;
        }
      }
    };
    auto scale = [&](const float (&v)[kPer], int done, int run) {
#pragma unroll
      for (int i = 0; i < kPer; i += 4) {
        const int at = done + (i / run * kClipThreads + threadIdx.x) * run + i % run;
        store4(at, n - at, v[i] * coef, v[i + 1] * coef, v[i + 2] * coef, v[i + 3] * coef);
      }
    };
    if (e.g_bf16) walk<true, true>(e.g, off, n, [&](const float (&v)[kPer], int done) { scale(v, done, 8); });
    else walk<false, true>(e.g, off, n, [&](const float (&v)[kPer], int done) { scale(v, done, 4); });
  }
}

int clip_blocks(uint32_t chunks) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(chunks, (int64_t)sm_count() * kClipBlocksPerSm));
}

template <int CAP>
cudaError_t run_clip(const GradTensor* t, const int* idx, int count, float max_norm, float* norm, double* part,
                     cudaStream_t st) {
  // lists of at most CAP tensors and 2^31 chunks each: every list's partial sums, then every list's scaling
  int64_t elements = 0;
  for (int i = 0; i < count; ++i) elements += t[idx[i]].n;
  // Steps per chunk: a chunk's first loads are not hidden behind another step, which costs about a step; the
  // last round of chunks may be short; every tensor may end in a short chunk of its own.
  const int64_t blocks_full = (int64_t)sm_count() * kClipBlocksPerSm, steps = ceil_div(elements, kStep);
  int64_t chunk = kStep, cost = INT64_MAX;
  for (int s = 1; s <= 16; ++s) {
    const int64_t k = ceil_div(ceil_div(steps, s) + count, blocks_full) * (s + 1);
    if (k < cost) { cost = k; chunk = (int64_t)s * kStep; }
  }
  int n_part = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int at = 0, slot = 0;
    bool first = true;
    while (at < count || first) {
      ClipList<CAP> l;
      l.count = 0;
      l.chunks = 0;
      l.chunk = (int)chunk;
      l.in_place = 1;
      while (at < count && l.count < CAP) {
        const GradTensor& g = t[idx[at]];
        const int64_t c = ceil_div(g.n, chunk);
        if (l.count > 0 && (int64_t)l.chunks + c > INT32_MAX) break;
        l.t[l.count++] = ClipEntry{g.grad, g.out, g.n, l.chunks, (uint16_t)g.grad_bf16, (uint16_t)g.out_bf16};
        l.chunks += (uint32_t)c;
        l.in_place &= g.out == g.grad;
        ++at;
      }
      const int64_t kept = kKeepBytes / (chunk * 4);
      l.keep_from = (uint32_t)std::max<int64_t>(0, (int64_t)l.chunks - kept);
      const int blocks = clip_blocks(l.chunks);
      cudaError_t e;
      if (pass == 0) {
        e = launch_pdl(k_clip_norm<CAP>, dim3(blocks), dim3(kClipThreads), 0, st, l, part + slot);
      } else {
        e = launch_pdl(k_clip_scale<CAP>, dim3(blocks), dim3(kClipThreads), 0, st, l, (const double*)part, n_part,
                       max_norm, first ? norm : (float*)nullptr);
      }
      note_launch();
      if (e != cudaSuccess) return e;
      slot += blocks;
      first = false;
    }
    n_part = slot;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_clip_workspace(int count) {
  return (size_t)std::max<int64_t>(1, ceil_div(count, kFewTensors)) * sm_count() * kClipBlocksPerSm * sizeof(double);
}

cudaError_t launch_grad_clip(const GradTensor* t, const int* idx, int count, float max_norm, float* norm, double* part,
                             cudaStream_t st) {
  if (count <= kFewTensors) return run_clip<kFewTensors>(t, idx, count, max_norm, norm, part, st);
  if (count <= kSomeTensors) return run_clip<kSomeTensors>(t, idx, count, max_norm, norm, part, st);
  return run_clip<kManyTensors>(t, idx, count, max_norm, norm, part, st);
}

}  // namespace upipe
