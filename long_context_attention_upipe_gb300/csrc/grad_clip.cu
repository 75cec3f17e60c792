// Global norm of many gradient tensors and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2),   out = g * min(1, max_norm / (norm + 1e-6))
// Two launches: the first sums squares (a partial sum per block, in the workspace), the second adds the
// partial sums up in every block, in the same order, and scales.  No atomics: the norm depends on the
// sizes alone, not on which block comes first.
//
// The tensors are cut into chunks of 8192 elements, walked by a fixed number of blocks, 32 elements of
// a thread in flight at once.  A thread squares and adds its 32 elements in fp32 and the chunks' sums
// in fp64.  Squares outside fp32's comfortable range (a sum below 1e-20 or above 1e30) are summed once
// more with the elements scaled by a power of two, which is exact, so neither tiny nor huge gradients
// lose their norm.
//
// Bound by HBM: reading twice and writing once, less what the second launch still finds in L2; it walks
// the chunks backwards, so that what was read last is read first.
#include "common.cuh"
#include "internal.h"

namespace upipe {

namespace {

constexpr int kClipThreads = 256;
constexpr int kChunk = 8192;
constexpr int kPer = kChunk / kClipThreads;  // 32 elements of a thread
constexpr int kFewTensors = 24, kManyTensors = 960;  // tensors of one launch (its parameters hold the list)

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

// 32 elements of this thread: 4 (fp32) or 8 (bf16) neighbours at a time; zeros past the end.
__device__ __forceinline__ void load32(const ClipEntry& e, int64_t base, int64_t n, float (&v)[kPer]) {
  if (e.g_bf16) {
    const bf16* g = reinterpret_cast<const bf16*>(e.g) + base;
    uint4 q[kPer / 8];
#pragma unroll
    for (int i = 0; i < kPer / 8; ++i) {
      const int at = (i * kClipThreads + threadIdx.x) * 8;
      if (at + 8 <= n) q[i] = *reinterpret_cast<const uint4*>(g + at);
      else {
        uint32_t w[4] = {0, 0, 0, 0};
        for (int k = 0; k < 8; ++k)
          if (at + k < n) w[k >> 1] |= (uint32_t)__bfloat16_as_ushort(g[at + k]) << (16 * (k & 1));
        q[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < kPer / 8; ++i) {
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __bfloat1622float2(h[k]);
        v[8 * i + 2 * k] = f.x;
        v[8 * i + 2 * k + 1] = f.y;
      }
    }
  } else {
    const float* g = reinterpret_cast<const float*>(e.g) + base;
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const int at = (i * kClipThreads + threadIdx.x) * 4;
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      if (at + 4 <= n) q = *reinterpret_cast<const float4*>(g + at);
      else {
        if (at < n) q.x = g[at];
        if (at + 1 < n) q.y = g[at + 1];
        if (at + 2 < n) q.z = g[at + 2];
      }
      v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
    }
  }
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
__global__ void __launch_bounds__(kClipThreads) k_clip_norm(const __grid_constant__ ClipList<CAP> l, double* part) {
  double total = 0.0;
  grid_dep_wait();
  for (uint32_t c = blockIdx.x; c < l.chunks; c += gridDim.x) {
    const ClipEntry& e = l.t[find_tensor(l, c)];
    const int64_t base = (int64_t)(c - e.chunk0) * kChunk;
    float v[kPer];
    load32(e, base, min((int64_t)kChunk, e.n - base), v);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s += v[i] * v[i];
    if (s >= 1e-20f && s <= 1e30f) {
      total += (double)s;
    } else {  // outside the range in which fp32 squares are exact enough (or zero, infinite, NaN)
      const bool small = s < 1e-20f;
      const float up = small ? 1.2379400392853803e27f : 8.470329472543003e-22f;          // 2^90, 2^-70
      const double back = small ? 6.525304467998525e-55 : 1.3937965749081639e42;          // 2^-180, 2^140
      float s2 = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) s2 += (v[i] * up) * (v[i] * up);
      total += (double)s2 * back;
    }
  }
  total = block_sum(total);
  if (threadIdx.x == 0) part[blockIdx.x] = total;
}

template <int CAP>
__global__ void __launch_bounds__(kClipThreads) k_clip_scale(const __grid_constant__ ClipList<CAP> l, const double* part,
                                                             int n_part, float max_norm, float* norm_out) {
  grid_dep_wait();  // the partial sums are complete and visible
  double total = 0.0;
  for (int i = threadIdx.x; i < n_part; i += kClipThreads) total += part[i];
  const double norm = sqrt(block_sum(total));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  // a norm that is not finite scales nothing: the caller sees it and skips the step
  float coef = 1.f;
  if (norm <= 1.7976931348623157e308) coef = (float)fmin(1.0, (double)max_norm / (norm + 1e-6));
  for (uint32_t k = blockIdx.x; k < l.chunks; k += gridDim.x) {
    const uint32_t c = l.chunks - 1 - k;
    const ClipEntry& e = l.t[find_tensor(l, c)];
    if (coef == 1.f && e.out == e.g) continue;
    const int64_t base = (int64_t)(c - e.chunk0) * kChunk, n = min((int64_t)kChunk, e.n - base);
    float v[kPer];
    load32(e, base, n, v);
    // element i of v is element at(i) of the chunk, in runs of `run` neighbours
    const int run = e.g_bf16 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const int at = (i / run * kClipThreads + threadIdx.x) * run + i % run;
      const float4 o = make_float4(v[i] * coef, v[i + 1] * coef, v[i + 2] * coef, v[i + 3] * coef);
      if (e.out_bf16) {
        bf16* dst = reinterpret_cast<bf16*>(e.out) + base;
        if (at + 4 <= n) *reinterpret_cast<uint2*>(dst + at) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
        else {
          if (at < n) dst[at] = __float2bfloat16_rn(o.x);
          if (at + 1 < n) dst[at + 1] = __float2bfloat16_rn(o.y);
          if (at + 2 < n) dst[at + 2] = __float2bfloat16_rn(o.z);
        }
      } else {
        float* dst = reinterpret_cast<float*>(e.out) + base;
        if (at + 4 <= n) *reinterpret_cast<float4*>(dst + at) = o;
        else {
          if (at < n) dst[at] = o.x;
          if (at + 1 < n) dst[at + 1] = o.y;
          if (at + 2 < n) dst[at + 2] = o.z;
        }
      }
    }
  }
}

int clip_blocks(uint32_t chunks) { return (int)std::max<int64_t>(1, std::min<int64_t>(chunks, (int64_t)sm_count() * 4)); }

template <int CAP>
cudaError_t run_clip(const GradTensor* t, const int* idx, int count, float max_norm, float* norm, double* part,
                     cudaStream_t st) {
  // lists of at most CAP tensors and 2^31 chunks each: every list's partial sums, then every list's scaling
  int n_part = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int at = 0, slot = 0;
    bool first = true;
    while (at < count || first) {
      ClipList<CAP> l;
      l.count = 0;
      l.chunks = 0;
      while (at < count && l.count < CAP) {
        const GradTensor& g = t[idx[at]];
        const int64_t c = ceil_div(g.n, kChunk);
        if (l.count > 0 && (int64_t)l.chunks + c > INT32_MAX) break;
        l.t[l.count++] = ClipEntry{g.grad, g.out, g.n, l.chunks, (uint16_t)g.grad_bf16, (uint16_t)g.out_bf16};
        l.chunks += (uint32_t)c;
        ++at;
      }
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
  return (size_t)std::max<int64_t>(1, ceil_div(count, kFewTensors)) * sm_count() * 4 * sizeof(double);
}

cudaError_t launch_grad_clip(const GradTensor* t, const int* idx, int count, float max_norm, float* norm, double* part,
                             cudaStream_t st) {
  return count <= kFewTensors ? run_clip<kFewTensors>(t, idx, count, max_norm, norm, part, st)
                              : run_clip<kManyTensors>(t, idx, count, max_norm, norm, part, st);
}

}  // namespace upipe
