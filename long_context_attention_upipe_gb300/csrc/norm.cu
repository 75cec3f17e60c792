// Root-mean-square norm with the residual's addition (forward in bf16 or e4m3, backward), and the
// e4m3 block quantiser.
//
// Forward, per row of d elements:
//   h = bf16(x + r)                        (without a residual h = x, nothing written)
//   rstd = (mean(h^2) + eps)^(-1/2),  y = h * rstd * w
//   y rounded to bf16, or per block of 128 columns  s = max|y| fp32(1 / 448),  q = e4m3(fp32(y / s))
// h is normalised as it is stored, so the backward pass, which reads the stored h, differentiates
// exactly the function that ran.  Backward, with t = dy * w:
//   dx = rstd * (t - h * rstd^2 * mean(t * h)) [+ dres],   dw = sum over rows of dy * h * rstd
// All sums are fp32; each output is rounded once.
//
// A row belongs to a group of `tpr` threads, 8 elements (one 16-byte vector) per thread and step, V
// steps, kept in registers between the statistics and the output: one read and one write of each
// tensor, which is what bounds these kernels (HBM: 32768 x 4096 into e4m3 149 us, 6.3 TB/s; 16381 x 5120
// backward 105 us, 6.4 TB/s).  A 128-column block is 16 neighbouring lanes, so
// its maximum is four shuffles; maxima are compared as the bits of |y|, which orders NaN above every
// number, so a NaN reaches its block's scale.
#include "internal.h"
#include "quant.cuh"
#include "tc_common.cuh"

namespace upipe {

namespace {

constexpr int kMaxNormThreads = 1024;
constexpr int kRingBytes = 216 * 1024;
constexpr int kMaxRing = 8;  // rows in flight of the ring kernel

// Maximum over the 16 lanes that hold a 128-column block.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

// Sum over a group of tpr threads (16, or a multiple of 32), the same for every thread of it.  `red`
// holds a float per warp of the block; callers alternate between two of them, so one barrier is enough.
__device__ __forceinline__ float group_sum(float v, int tpr, float* red) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (tpr == 16) return v;
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  if (tpr == 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = tpr >> 5;
  const int first = warp / nw * nw;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < nw ? red[first + lane] : 0.f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

struct NormShape {
  int64_t rows;
  int d, tpr, rpb;  // columns; threads per row; rows per block
};

// PF: the next row's loads are issued as soon as the current row's registers are free, before the row's
// reduction, so every block always has a row in flight.
template <int V, bool FP8, int MAXT, int MINB, bool PF>
__global__ void __launch_bounds__(MAXT, MINB) k_rms_fwd(NormShape n, float eps, const bf16* x, const bf16* res,
                                                        const bf16* __restrict__ w, bf16* h, bf16* y, uint8_t* q,
                                                        float* scales, float* rstd_out) {
  __shared__ float red[2][32];
  const int g = threadIdx.x / n.tpr, t = threadIdx.x - g * n.tpr;
  const int nvec = n.d >> 3;
  grid_dep_wait();
  uint4 wv[V], xv[V], rv[V];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * n.tpr;
      const bool ok = row < n.rows && c < nvec;
      xv[i] = ok ? *reinterpret_cast<const uint4*>(x + row * n.d + c * 8) : make_uint4(0, 0, 0, 0);
      if (res) rv[i] = ok ? *reinterpret_cast<const uint4*>(res + row * n.d + c * 8) : make_uint4(0, 0, 0, 0);
    }
  };
  const int64_t step = (int64_t)gridDim.x * n.rpb;
  int64_t row = (int64_t)blockIdx.x * n.rpb + g;
  if (PF) load(row);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * n.tpr;
    wv[i] = c < nvec ? *reinterpret_cast<const uint4*>(w + c * 8) : make_uint4(0, 0, 0, 0);
  }
  int par = 0;
  // every group of the block makes the same number of turns (group_sum holds a barrier)
  for (int64_t r0 = (int64_t)blockIdx.x * n.rpb; r0 < n.rows; r0 += step, row += step, par ^= 1) {
    const bool row_ok = row < n.rows;
    if (!PF) load(row);
    V8 f[V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * n.tpr;
      f[i] = unpack8(xv[i]);
      if (res) {
        const V8 b = unpack8(rv[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[i].v[k] += b.v[k];
        const uint4 hv = pack8(f[i]);
        if (row_ok && c < nvec) *reinterpret_cast<uint4*>(h + row * n.d + c * 8) = hv;
        f[i] = unpack8(hv);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) ss += f[i].v[k] * f[i].v[k];
    }
    if (PF) load(row + step);
    ss = group_sum(ss, n.tpr, red[par]);
    const float rstd = rsqrtf(ss / (float)n.d + eps);
    if (rstd_out && row_ok && t == 0) rstd_out[row] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * n.tpr;
      const bool ok = row_ok && c < nvec;
      const int64_t at = row * n.d + c * 8;
      const V8 wf = unpack8(wv[i]);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 o = __fmul2_rn(__fmul2_rn(make_float2(f[i].v[k], f[i].v[k + 1]), make_float2(rstd, rstd)),
                                    make_float2(wf.v[k], wf.v[k + 1]));
        f[i].v[k] = o.x;
        f[i].v[k + 1] = o.y;
      }
      if (!FP8 || y) {
        if (ok) *reinterpret_cast<uint4*>(y + at) = pack8(f[i]);
      }
      if (FP8) {
        // columns past d of the last block hold zeros (x and w were read as zeros there), unless
        // rstd is not finite; they must not reach the block's maximum then either
        const float s = block_scale(max16(ok ? amax_bits(f[i]) : 0u));
        const Divisor by = divisor(s);
        if (ok) *reinterpret_cast<uint2*>(q + at) = by.doubt ? quant8_divided(f[i], s) : quant8(f[i], by);
        if (ok && (t & 15) == 0) scales[(int64_t)(c >> 4) * n.rows + row] = s;
      }
    }
  }
}

// The next row's loads are issued before the current row's reduction.
template <int V, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_rms_bwd(NormShape n, const bf16* dy, const bf16* h,
                                                        const bf16* __restrict__ w, const float* __restrict__ rstd_in,
                                                        const bf16* dres, bf16* dx, float* part) {
  __shared__ float red[2][32];
  const int g = threadIdx.x / n.tpr, t = threadIdx.x - g * n.tpr;
  const int nvec = n.d >> 3;
  grid_dep_wait();
  uint4 wv[V], nd[V], nh[V], nr[V];
  float rstd_next = 0.f;
  auto load = [&](int64_t row) {
    rstd_next = row < n.rows ? rstd_in[row] : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * n.tpr;
      const bool ok = row < n.rows && c < nvec;
      const int64_t at = row * n.d + c * 8;
      nd[i] = ok ? *reinterpret_cast<const uint4*>(dy + at) : make_uint4(0, 0, 0, 0);
      nh[i] = ok ? *reinterpret_cast<const uint4*>(h + at) : make_uint4(0, 0, 0, 0);
      nr[i] = ok && dres ? *reinterpret_cast<const uint4*>(dres + at) : make_uint4(0, 0, 0, 0);
    }
  };
  const int64_t step = (int64_t)gridDim.x * n.rpb;
  int64_t row = (int64_t)blockIdx.x * n.rpb + g;
  load(row);
  V8 dw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * n.tpr;
    wv[i] = c < nvec ? *reinterpret_cast<const uint4*>(w + c * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i].v[k] = 0.f;
  }
  int par = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * n.rpb; r0 < n.rows; r0 += step, row += step, par ^= 1) {
    const bool row_ok = row < n.rows;
    uint4 dv[V], hv[V], rv[V];
    const float rstd = rstd_next;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dv[i] = nd[i];
      hv[i] = nh[i];
      rv[i] = nr[i];
    }
    load(row + step);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const V8 a = unpack8(dv[i]), b = unpack8(hv[i]), wf = unpack8(wv[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dot += a.v[k] * wf.v[k] * b.v[k];
        dw[i].v[k] += a.v[k] * (b.v[k] * rstd);
      }
    }
    dot = group_sum(dot, n.tpr, red[par]);
    const float m = dot / (float)n.d * rstd * rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * n.tpr;
      if (!row_ok || c >= nvec) continue;
      const V8 a = unpack8(dv[i]), b = unpack8(hv[i]), wf = unpack8(wv[i]), r = unpack8(rv[i]);
      V8 o;
#pragma unroll
      for (int k = 0; k < 8; ++k) o.v[k] = r.v[k] + rstd * (a.v[k] * wf.v[k] - b.v[k] * m);
      *reinterpret_cast<uint4*>(dx + row * n.d + c * 8) = pack8(o);
    }
  }
  // this group's share of dw: row `group` of the partial sums
  float* dst = part + ((int64_t)blockIdx.x * n.rpb + g) * n.d;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * n.tpr;
    if (c >= nvec) continue;
    *reinterpret_cast<float4*>(dst + c * 8) = make_float4(dw[i].v[0], dw[i].v[1], dw[i].v[2], dw[i].v[3]);
    *reinterpret_cast<float4*>(dst + c * 8 + 4) = make_float4(dw[i].v[4], dw[i].v[5], dw[i].v[6], dw[i].v[7]);
  }
}

// The same for longer rows, whose next row would not fit into registers without leaving SMs short of threads
// (see bwd_ring): a producer warp copies whole rows (dy, h, dres) ahead into a ring in shared memory, tpr
// threads work on one row after the other.  One block per SM.  A thread whose wait runs out (wait_ns) gives up for good
// and hands no stage back; the rows of dx that its block has not finished, and dw, become NaN.
template <int V>
__global__ void __launch_bounds__(V == 2 ? 512 : 544, 1) k_rms_bwd_ring(NormShape n, const bf16* dy, const bf16* h, const bf16* __restrict__ w,
                                                         const float* __restrict__ rstd_in, const bf16* dres, bf16* dx,
                                                         float* part, int stages, uint64_t wait_ns) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxRing], empty[kMaxRing];
  __shared__ float red[2][32];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nvec = n.d >> 3, nw = n.tpr >> 5;
  const uint32_t row_bytes = (uint32_t)n.d * 2, stage_bytes = row_bytes * (dres ? 3 : 2);
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], nw);
    }
    abort_word = 0;
    tc::fence_mbar_init();
  }
  __syncthreads();
  grid_dep_wait();
  int s = 0;
  bool ok = true;
  if (warp == 0) {
    const bool leader = tc::elect_one();
    uint32_t ph = 1, turns = 0;  // parity of the stage's previous release: the first turn needs none
    for (int64_t row = blockIdx.x; row < n.rows && __all_sync(0xffffffffu, ok); row += gridDim.x) {
      ok = tc::mbar_wait_addr(smem_u32(&empty[s]), ph, abort_flag, wait_ns) && ok;
      if (leader && ok) {
        ++turns;
        uint8_t* st = ring + s * stage_bytes;
        tc::mbar_arrive_expect_tx(&full[s], stage_bytes);
        tc::bulk_load(st, dy + row * n.d, row_bytes, &full[s]);
        tc::bulk_load(st + row_bytes, h + row * n.d, row_bytes, &full[s]);
        if (dres) tc::bulk_load(st + 2 * row_bytes, dres + row * n.d, row_bytes, &full[s]);
      }
      __syncwarp();
      if (++s == stages) { s = 0; ph ^= 1; }
    }
    if (leader) tc::drain_ring(smem_u32(full), turns, stages);
    return;
  }
  const int t = threadIdx.x - 32;
  // two vectors per thread stay in registers between the sum and the output; four are read from the ring again
  constexpr bool kHold = V == 2;
  uint4 wv[kHold ? V : 1];
  V8 dw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * n.tpr;
    if (kHold) wv[i] = c < nvec ? *reinterpret_cast<const uint4*>(w + c * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i].v[k] = 0.f;
  }
  uint32_t ph = 0;
  int par = 0;
  float rstd_next = blockIdx.x < n.rows ? rstd_in[blockIdx.x] : 0.f;
  for (int64_t row = blockIdx.x; row < n.rows; row += gridDim.x, par ^= 1) {
    const float rstd = rstd_next;
    if (row + gridDim.x < n.rows) rstd_next = rstd_in[row + gridDim.x];
    ok = tc::mbar_wait_addr(smem_u32(&full[s]), ph, abort_flag, wait_ns) && ok;
    const uint8_t* st = ring + s * stage_bytes;
    uint4 dv[V], hv[V], rv[V];
    auto read = [&](int i, int c) {
      dv[i] = hv[i] = rv[i] = make_uint4(0, 0, 0, 0);
      if (c < nvec) {
        dv[i] = *reinterpret_cast<const uint4*>(st + c * 16);
        hv[i] = *reinterpret_cast<const uint4*>(st + row_bytes + c * 16);
        if (dres) rv[i] = *reinterpret_cast<const uint4*>(st + 2 * row_bytes + c * 16);
      }
    };
    auto weight = [&](int i, int c) {
      return kHold ? wv[i] : c < nvec ? *reinterpret_cast<const uint4*>(w + c * 8) : make_uint4(0, 0, 0, 0);
    };
    auto release = [&]() {
      __syncwarp();
      if (lane == 0 && ok) tc::mbar_arrive(&empty[s]);
      if (++s == stages) { s = 0; ph ^= 1; }
    };
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * n.tpr;
      read(i, c);
      const V8 a = unpack8(dv[i]), b = unpack8(hv[i]), wf = unpack8(weight(i, c));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dot += a.v[k] * wf.v[k] * b.v[k];
        dw[i].v[k] += a.v[k] * (b.v[k] * rstd);
      }
    }
    if (kHold) release();
    if (!ok) dot = __int_as_float(0x7fc00000);  // through the sum, the whole row becomes NaN
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if (lane == 0) red[par][warp - 1] = dot;
    tc::named_bar_sync(1, n.tpr);
    dot = lane < nw ? red[par][lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    const float m = dot / (float)n.d * rstd * rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * n.tpr;
      if (c >= nvec) continue;
      if (!kHold) read(i, c);
      const V8 a = unpack8(dv[i]), b = unpack8(hv[i]), wf = unpack8(weight(i, c)), r = unpack8(rv[i]);
      V8 o;
#pragma unroll
      for (int k = 0; k < 8; ++k) o.v[k] = r.v[k] + rstd * (a.v[k] * wf.v[k] - b.v[k] * m);
      *reinterpret_cast<uint4*>(dx + row * n.d + c * 8) = pack8(o);
    }
    if (!kHold) release();
  }
  float* dst = part + (int64_t)blockIdx.x * n.d;
  tc::named_bar_sync(1, n.tpr);
  const float bad = *abort_flag ? __int_as_float(0x7fc00000) : 0.f;  // rows are missing from every column's sum
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * n.tpr;
    if (c >= nvec) continue;
    *reinterpret_cast<float4*>(dst + c * 8) = make_float4(dw[i].v[0] + bad, dw[i].v[1] + bad, dw[i].v[2] + bad, dw[i].v[3] + bad);
    *reinterpret_cast<float4*>(dst + c * 8 + 4) = make_float4(dw[i].v[4] + bad, dw[i].v[5] + bad, dw[i].v[6] + bad, dw[i].v[7] + bad);
  }
}

// The same for rows of more than 16384 columns (1024 threads at 64 registers), whose vectors do not fit into
// registers beside the sums of dw: the row is read twice, the second time from L1 or L2 (3.9 TB/s at d 32768,
// where spilled registers left 1.5; at d 16384 the kernel above runs at 6.3, this one at 4.3).
__global__ void __launch_bounds__(kMaxNormThreads, 1) k_rms_bwd_long(NormShape n, const bf16* dy, const bf16* h,
                                                                     const bf16* __restrict__ w,
                                                                     const float* __restrict__ rstd_in, const bf16* dres,
                                                                     bf16* dx, float* part) {
  constexpr int V = 4;
  __shared__ float red[2][32];
  const int t = threadIdx.x, nvec = n.d >> 3;
  grid_dep_wait();
  V8 dw[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i].v[k] = 0.f;
  int par = 0;
  for (int64_t row = blockIdx.x; row < n.rows; row += gridDim.x, par ^= 1) {
    const float rstd = rstd_in[row];
    const bf16 *dyr = dy + row * n.d, *hr = h + row * n.d, *rr = dres ? dres + row * n.d : nullptr;
    bf16* dxr = dx + row * n.d;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * n.tpr;
      if (c >= nvec) continue;
      const V8 a = unpack8(*reinterpret_cast<const uint4*>(dyr + c * 8)), b = unpack8(*reinterpret_cast<const uint4*>(hr + c * 8));
      const V8 wf = unpack8(*reinterpret_cast<const uint4*>(w + c * 8));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dot += a.v[k] * wf.v[k] * b.v[k];
        dw[i].v[k] += a.v[k] * (b.v[k] * rstd);
      }
    }
    dot = group_sum(dot, n.tpr, red[par]);
    const float m = dot / (float)n.d * rstd * rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * n.tpr;
      if (c >= nvec) continue;
      const V8 a = unpack8(*reinterpret_cast<const uint4*>(dyr + c * 8)), b = unpack8(*reinterpret_cast<const uint4*>(hr + c * 8));
      const V8 wf = unpack8(*reinterpret_cast<const uint4*>(w + c * 8));
      const V8 r = unpack8(rr ? *reinterpret_cast<const uint4*>(rr + c * 8) : make_uint4(0, 0, 0, 0));
      V8 o;
#pragma unroll
      for (int k = 0; k < 8; ++k) o.v[k] = r.v[k] + rstd * (a.v[k] * wf.v[k] - b.v[k] * m);
      *reinterpret_cast<uint4*>(dxr + c * 8) = pack8(o);
    }
  }
  float* dst = part + (int64_t)blockIdx.x * n.d;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * n.tpr;
    if (c >= nvec) continue;
    *reinterpret_cast<float4*>(dst + c * 8) = make_float4(dw[i].v[0], dw[i].v[1], dw[i].v[2], dw[i].v[3]);
    *reinterpret_cast<float4*>(dst + c * 8 + 4) = make_float4(dw[i].v[4], dw[i].v[5], dw[i].v[6], dw[i].v[7]);
  }
}

// dw[c] = sum over p of part[p][c], in an order that depends on the shape alone: 32 columns per block, 32
// warps that each take every 32nd partial row (4 loads in flight), then the warps in turn.
__global__ void __launch_bounds__(1024) k_dw_reduce(const float* __restrict__ part, int p_rows, int d, float* dw) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  grid_dep_wait();
  float v = 0.f;
  if (c < d) {
    int p = warp;
    for (; p + 96 < p_rows; p += 128) {
      const float a0 = part[(int64_t)p * d + c], a1 = part[(int64_t)(p + 32) * d + c];
      const float a2 = part[(int64_t)(p + 64) * d + c], a3 = part[(int64_t)(p + 96) * d + c];
      v += (a0 + a1) + (a2 + a3);
    }
    for (; p < p_rows; p += 32) v += part[(int64_t)p * d + c];
  }
  s[warp][lane] = v;
  __syncthreads();
  v = s[lane][warp];  // column `warp` of the block, warp `lane`'s share
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  const int cw = blockIdx.x * 32 + warp;
  if (lane == 0 && cw < d) dw[cw] = v;
}

// One scale per row and 128 columns: 16 lanes per block, blocks of a row side by side, four blocks of a
// 16-lane group in flight at once (32768 x 4096: 75 us, 5.4 TB/s; one block in flight 94 us).
__global__ void __launch_bounds__(256, 4) k_quant_rows(int64_t rows, int d, int nb, const bf16* __restrict__ x, uint8_t* q,
                                                    float* scales) {
  constexpr int U = 4;
  const int64_t total = rows * nb;  // (row, block) pairs
  const int64_t step = (int64_t)gridDim.x * 16;
  const int lane16 = threadIdx.x & 15;
  const int64_t first = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t turns = ceil_div(total, step * U);  // the same for every lane: the shuffles need them all
  // the pair `step` further on, without a division per pair
  const int64_t step_row = step / nb;
  const int step_b = (int)(step - step_row * nb);
  int64_t row = first / nb;
  int b = (int)(first - row * nb);
  grid_dep_wait();
  for (int64_t k = 0; k < turns; ++k) {
    uint4 v[U];
    int64_t rw[U];
    int bl[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rw[u] = row;
      bl[u] = b;
      const int c = b * 128 + lane16 * 8;
      v[u] = row < rows && c < d ? *reinterpret_cast<const uint4*>(x + row * d + c) : make_uint4(0, 0, 0, 0);
      row += step_row;
      b += step_b;
      if (b >= nb) { b -= nb; ++row; }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const V8 f = unpack8(v[u]);
      const float s = block_scale(max16(pair_bits(amax2(v[u]))));
      const Divisor by = divisor(s);
      const int c = bl[u] * 128 + lane16 * 8;
      if (rw[u] < rows && c < d) *reinterpret_cast<uint2*>(q + rw[u] * d + c) = by.doubt ? quant8_divided(f, s) : quant8(f, by);
      if (rw[u] < rows && lane16 == 0) scales[(int64_t)bl[u] * rows + rw[u]] = s;
    }
  }
}

// One scale per 128 x 128 block: a block of threads per tile, 8 vectors per thread in registers.  Four blocks
// of threads per SM (64 registers): 28672 x 4096 in 54 us, 6.5 TB/s, where two took 68.
__global__ void __launch_bounds__(256, 4) k_quant_tiles(int64_t rows, int d, int nb, const bf16* __restrict__ x, uint8_t* q,
                                                     float* scales) {
  __shared__ uint32_t red[8];
  const int64_t tile = blockIdx.x;
  const int64_t tr = tile / nb;
  const int b = (int)(tile - tr * nb);
  uint4 v[8];
  uint32_t m = 0;
  grid_dep_wait();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int id = threadIdx.x + 256 * i;
    const int64_t row = tr * 128 + (id >> 4);
    const int c = b * 128 + (id & 15) * 8;
    v[i] = row < rows && c < d ? *reinterpret_cast<const uint4*>(x + row * d + c) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = amax2(m, amax2(v[i]));
  m = pair_bits(m);
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, red[i]);
  const float s = block_scale(m);
  const Divisor by = divisor(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int id = threadIdx.x + 256 * i;
    const int64_t row = tr * 128 + (id >> 4);
    const int c = b * 128 + (id & 15) * 8;
    if (row < rows && c < d) {
      const V8 f = unpack8(v[i]);
      *reinterpret_cast<uint2*>(q + row * d + c) = by.doubt ? quant8_divided(f, s) : quant8(f, by);
    }
  }
  if (threadIdx.x == 0) scales[tr * nb + b] = s;
}

// Threads per row and vectors per thread.  Rows of up to 32 vectors take half a warp or a warp with one
// vector per thread; longer rows two vectors per thread, up to 512 threads (d 8192), then four.
NormShape norm_shape(int64_t rows, int d, int& V) {
  const int nvec = d / 8;
  NormShape n{rows, d, 0, 1};
  if (nvec <= 32) {
    V = 1;
    n.tpr = nvec <= 16 ? 16 : 32;
  } else {
    V = nvec <= 1024 ? 2 : 4;
    n.tpr = (int)ceil_div(ceil_div(nvec, V), 32) * 32;
  }
  n.rpb = std::max(1, 256 / n.tpr);
  return n;
}

// The backward pass holds a row's vectors twice (the next row's are in flight) and the sums of dw: at two
// vectors per thread it takes 128 registers (at 96 it spills and runs at half the speed), so an SM holds 512
// threads.  Between 4096 and 16384 columns the rows in flight lie in shared memory instead (d 5120: 5.5 TB/s in
// registers, 6.5 in shared memory; 16384: 4.8, 6.3), but for 7688 to 8192, which fill 512 threads (8192: 6.1, 5.8).
bool bwd_ring(int d) { return (d > 4096 && d <= 7680) || (d > 8192 && d <= 16384); }
NormShape bwd_shape(int64_t rows, int d, int& V) {
  NormShape n = norm_shape(rows, d, V);
  if (bwd_ring(d)) {  // with its producer warp at most 16 warps at two vectors per thread: 128 registers
    V = d <= 7680 ? 2 : 4;
    n.tpr = (int)ceil_div(d / 8, 32 * V) * 32;
    n.rpb = 1;
  }
  return n;
}

int64_t norm_blocks(const NormShape& n, int per_sm_threads) {
  const int threads = n.tpr * n.rpb;
  const int64_t most = (int64_t)sm_count() * std::max(1, per_sm_threads / threads);
  return std::max<int64_t>(1, std::min<int64_t>(ceil_div(n.rows, n.rpb), most));
}

// resident threads per SM that the launch bounds below leave room for
constexpr int kFwdThreadsPerSm = 1024, kBwdThreadsPerSm = 512, kBwdThreadsPerSmNarrow = 768;

int bwd_threads(int d, int V) { return bwd_ring(d) ? 0 : V == 1 ? kBwdThreadsPerSmNarrow : kBwdThreadsPerSm; }

}  // namespace

int sm_count() {
  static int sms = 0;
  if (sms == 0) {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
      v = 152;
    sms = v;
  }
  return sms;
}

template <int V, int MAXT, int MINB, bool PF>
static cudaError_t run_rms_fwd(const NormShape& n, const RmsNormArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)norm_blocks(n, kFwdThreadsPerSm)), block(n.tpr * n.rpb);
  const cudaError_t e = launch_pdl(a.q ? k_rms_fwd<V, true, MAXT, MINB, PF> : k_rms_fwd<V, false, MAXT, MINB, PF>, grid, block, 0,
                                   st, n, a.eps, a.x, a.res, a.w, a.h, a.y, a.q, a.scales, a.rstd);
  note_launch();
  return e;
}

cudaError_t launch_rms_fwd(const RmsNormArgs& a, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  int V = 1;
  const NormShape n = norm_shape(a.rows, a.d, V);
  if (V == 1) return run_rms_fwd<1, 320, 3, true>(n, a, st);
  if (V == 2 && n.tpr <= 320) return run_rms_fwd<2, 320, 3, true>(n, a, st);
  if (V == 2) return run_rms_fwd<2, 512, 2, true>(n, a, st);
  if (n.tpr <= 512) return run_rms_fwd<4, 512, 1, true>(n, a, st);
  return run_rms_fwd<4, kMaxNormThreads, 1, false>(n, a, st);
}

size_t rms_bwd_workspace(int64_t rows, int d) {
  int V = 1;
  const NormShape n = bwd_shape(std::max<int64_t>(rows, 1), d, V);
  return (size_t)norm_blocks(n, bwd_threads(n.d, V)) * n.rpb * d * sizeof(float);
}

template <int V, int MAXT, int MINB>
static cudaError_t run_rms_bwd(const NormShape& n, const RmsNormBwdArgs& a, float* part, cudaStream_t st) {
  const dim3 grid((unsigned)norm_blocks(n, bwd_threads(n.d, V))), block(n.tpr * n.rpb);
  const cudaError_t e = launch_pdl(k_rms_bwd<V, MAXT, MINB>, grid, block, 0, st, n, a.dy, a.h, a.w, a.rstd, a.dres, a.dx, part);
  note_launch();
  return e;
}

template <int V>
static cudaError_t run_rms_bwd_ring(const NormShape& n, const RmsNormBwdArgs& a, float* part, cudaStream_t st) {
  const int stage = n.d * 2 * (a.dres ? 3 : 2);
  const int stages = std::min(kMaxRing, kRingBytes / stage);
  cudaError_t e = cudaFuncSetAttribute(k_rms_bwd_ring<V>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_rms_bwd_ring<V>, dim3((unsigned)norm_blocks(n, 0)), dim3(32 + n.tpr), (size_t)stages * stage, st, n,
                 a.dy, a.h, a.w, a.rstd, a.dres, a.dx, part, stages, wait_limit_ns());
  note_launch();
  return e;
}

cudaError_t launch_rms_bwd(const RmsNormBwdArgs& a, float* part, cudaStream_t st) {
  int p_rows = 0;
  if (a.rows > 0) {
    int V = 1;
    const NormShape n = bwd_shape(a.rows, a.d, V);
    p_rows = (int)norm_blocks(n, bwd_threads(n.d, V)) * n.rpb;
    cudaError_t e;
    if (bwd_ring(a.d)) e = V == 2 ? run_rms_bwd_ring<2>(n, a, part, st) : run_rms_bwd_ring<4>(n, a, part, st);
    else if (V == 4) {
      e = launch_pdl(k_rms_bwd_long, dim3((unsigned)norm_blocks(n, bwd_threads(n.d, V))), dim3(n.tpr), 0, st, n, a.dy, a.h, a.w, a.rstd,
                     a.dres, a.dx, part);
      note_launch();
    } else if (V == 1) e = run_rms_bwd<1, 256, 3>(n, a, part, st);
    else if (n.tpr <= 256) e = run_rms_bwd<2, 256, 2>(n, a, part, st);
    else e = run_rms_bwd<2, 512, 1>(n, a, part, st);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_pdl(k_dw_reduce, dim3((unsigned)ceil_div(a.d, 32)), dim3(1024), 0, st, (const float*)part, p_rows,
                                   a.d, a.dw);
  note_launch();
  return e;
}

cudaError_t launch_quantize(int64_t rows, int d, int block_rows, const bf16* x, uint8_t* q, float* scales,
                            cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  const int nb = (int)ceil_div(d, 128);
  cudaError_t e;
  if (block_rows == 1) {
    const int64_t blocks = std::min<int64_t>(ceil_div(rows * nb, 16), (int64_t)sm_count() * 4);
    e = launch_pdl(k_quant_rows, dim3((unsigned)blocks), dim3(256), 0, st, rows, d, nb, x, q, scales);
  } else {
    e = launch_pdl(k_quant_tiles, dim3((unsigned)(ceil_div(rows, 128) * nb)), dim3(256), 0, st, rows, d, nb, x, q, scales);
  }
  note_launch();
  return e;
}

}  // namespace upipe
