// 8-bit matrix product with a scale for each block of 128 (tcgen05 kind::f8f6f4, TMEM, TMA).
//
//   C[m, n] = sum_kb sa[kb][m] * sb[n / 128][kb] * sum_{k in block kb} A[m, k] B[n, k]
// with e4m3 A (activations: a scale per row and 128 columns) and B (weights: a scale per 128 x 128
// block), fp32 scales.  The tensor core sums one 128-wide block of K exactly as given (four MMAs of
// K 32); the block's scales then multiply that sum on its way from TMEM into fp32 registers, where the
// blocks are added up.  Blocks alternate between two TMEM accumulators, so the tensor core works on
// one while the other is scaled.
//
// Few rows of A (decode): the weights take the 128 rows of the MMA and the tokens its N side (TN = 16
// ... 128 of them), so the tensor core's rows are full whatever the batch.  One CTA per 128 weight rows
// and TN tokens, 6 warps: 0 TMA producer, 1 MMA issuer, 2-5 scaling (one weight row per thread).
#include <cstring>

#include "internal.h"
#include "tc_common.cuh"

namespace upipe {

namespace {

constexpr int kBlk = 128;  // K block of a scale, and a stage of the operand ring

struct Fp8Params {
  int64_t M, N, K;
  int nkb;
  const float* sa;
  int64_t lds;
  const float* sb;
  void* c;
  int64_t ldc;
  int c_bf16;
  uint64_t wait_ns;
};

// ------------------------------------------------------------------------------------------------
// weights on the MMA's rows, TN tokens on its columns
// ------------------------------------------------------------------------------------------------
template <int TN>
struct SwapLayout {
  static constexpr int STAGES = TN <= 32 ? 6 : 5;
  static constexpr uint32_t W = 128 * 128, T = TN * 128, STAGE = W + T;
  static constexpr uint32_t SC = STAGES * STAGE;               // two rows of TN scales
  static constexpr uint32_t BAR = SC + 2 * TN * 4;
  static constexpr uint32_t BYTES = BAR + 256;
  static constexpr uint32_t TMEM = 2 * TN < 32 ? 32 : 2 * TN;  // power of two
};

constexpr int kSwapThreads = 192;

template <int TN>
__global__ void __launch_bounds__(kSwapThreads) k_gemm_fp8_swap(const __grid_constant__ CUtensorMap tw,
                                                                const __grid_constant__ CUtensorMap tt, Fp8Params p) {
  using L = SwapLayout<TN>;
  constexpr int ST = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sc = reinterpret_cast<float*>(smem + L::SC);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR);
  uint64_t* full = bars;               // [ST]
  uint64_t* empty = bars + ST;         // [ST]
  uint64_t* acc_full = bars + 2 * ST;  // [2]
  uint64_t* acc_empty = acc_full + 2;  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(acc_empty + 3);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n0 = (int64_t)blockIdx.x * 128, m0 = (int64_t)blockIdx.y * TN;
  const int nkb = p.nkb;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&acc_full[i], 1);
      tc::mbar_init(&acc_empty[i], 128);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, L::TMEM);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      tc::prefetch_tmap(&tw);
      tc::prefetch_tmap(&tt);
      for (int kb = 0; kb < nkb; ++kb) {
        const int s = kb % ST;
        if (kb >= ST && !tc::mbar_wait(&empty[s], ((kb / ST) - 1) & 1, abort_flag, nullptr, p.wait_ns)) break;
        tc::mbar_arrive_expect_tx(&full[s], L::STAGE);
        tc::tma_load_2d(smem + s * L::STAGE, &tw, &full[s], kb * kBlk, (int)n0);
        tc::tma_load_2d(smem + s * L::STAGE + L::W, &tt, &full[s], kb * kBlk, (int)m0);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = tc::idesc_e4m3(128, TN);
      const uint64_t w0 = tc::sdesc_sw128(smem_u32(smem), 16, 1024), t0 = tc::sdesc_add(w0, L::W);
      for (int kb = 0; kb < nkb; ++kb) {
        const int s = kb % ST, buf = kb & 1;
        if (kb >= 2 && !tc::mbar_wait(&acc_empty[buf], ((kb >> 1) - 1) & 1, abort_flag, nullptr, p.wait_ns)) break;
        if (!tc::mbar_wait(&full[s], (kb / ST) & 1, abort_flag, nullptr, p.wait_ns)) break;
        tc::fence_after_sync();
        const uint64_t wd = tc::opaque(tc::sdesc_add(w0, s * L::STAGE)), td = tc::opaque(tc::sdesc_add(t0, s * L::STAGE));
#pragma unroll
        for (int k = 0; k < kBlk / 32; ++k)
          tc::mma_ss_f8(tmem + buf * TN, tc::sdesc_add(wd, k * 32), tc::sdesc_add(td, k * 32), idesc, k > 0);
        tc::mma_commit(&empty[s]);
        tc::mma_commit(&acc_full[buf]);
      }
    }
    __syncwarp();
  } else {
    // scaling warps: one weight row (TMEM lane) per thread, TN token columns
    const int t = threadIdx.x - 64;
    const int64_t n = n0 + 32 * (warp & 3) + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    // token t's scale times the weight block's, loaded PF blocks ahead
    constexpr int PF = 4;
    const float* sb = p.sb + (int64_t)blockIdx.x * nkb;
    const bool has = t < TN && m0 + t < p.M;
    auto scale_of = [&](int kb) { return has && kb < nkb ? p.sa[(int64_t)kb * p.lds + m0 + t] * sb[kb] : 0.f; };
    float ahead[PF];
#pragma unroll
    for (int i = 0; i < PF; ++i) ahead[i] = scale_of(i);
    float acc[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i) acc[i] = 0.f;
    bool ok = true;
    for (int kb0 = 0; kb0 < nkb; kb0 += PF) {
#pragma unroll
      for (int u = 0; u < PF; ++u) {
        const int kb = kb0 + u;
        if (kb >= nkb) break;
        const int buf = kb & 1;
        if (t < TN) sc[buf * TN + t] = ahead[u];
        ahead[u] = scale_of(kb + PF);
        tc::named_bar_sync(1, 128);  // never skipped, so that a thread that gave up holds nobody up
        if (ok) ok = tc::mbar_wait(&acc_full[buf], (kb >> 1) & 1, abort_flag, nullptr, p.wait_ns);
        __syncwarp();
        tc::fence_after_sync();
#pragma unroll
        for (int ch = 0; ch < TN / 16; ++ch) {
          uint32_t v[16];
          tc::tmem_ld16(lane_addr + buf * TN + ch * 16, v);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 s4 = *reinterpret_cast<const float4*>(&sc[buf * TN + ch * 16 + i]);
            acc[ch * 16 + i] += __uint_as_float(v[i]) * s4.x;
            acc[ch * 16 + i + 1] += __uint_as_float(v[i + 1]) * s4.y;
            acc[ch * 16 + i + 2] += __uint_as_float(v[i + 2]) * s4.z;
            acc[ch * 16 + i + 3] += __uint_as_float(v[i + 3]) * s4.w;
          }
        }
        tc::fence_before_sync();
        tc::mbar_arrive(&acc_empty[buf]);
      }
    }
    // neighbouring lanes hold neighbouring columns of C
    if (ok && n < p.N) {
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        if (m0 + i < p.M) {
          const int64_t at = (m0 + i) * p.ldc + n;
          if (p.c_bf16) reinterpret_cast<bf16*>(p.c)[at] = __float2bfloat16_rn(acc[i]);
          else reinterpret_cast<float*>(p.c)[at] = acc[i];
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::TMEM);
  }
}

template <int TN>
cudaError_t run_swap(const Fp8GemmArgs& a, const Fp8Params& p, cudaStream_t st) {
  using L = SwapLayout<TN>;
  CUtensorMap tw, tt;
  if (!make_tmap_2d_u8(&tw, a.B, a.K, a.N, a.ldb, kBlk, 128) || !make_tmap_2d_u8(&tt, a.A, a.K, a.M, a.lda, kBlk, TN))
    return cudaErrorInvalidValue;
  auto kfn = k_gemm_fp8_swap<TN>;
  const size_t smem = L::BYTES + 1024;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kfn<<<dim3((unsigned)ceil_div(a.N, 128), (unsigned)ceil_div(a.M, TN)), kSwapThreads, smem, st>>>(tw, tt, p);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_fp8(const Fp8GemmArgs& a, cudaStream_t st) {
  if (a.M <= 0) return cudaSuccess;
  Fp8Params p{a.M, a.N, a.K, (int)ceil_div(a.K, kBlk), a.sa, a.lds, a.sb, a.C, a.ldc, a.c_bf16, wait_limit_ns()};
  if (a.M <= 16) return run_swap<16>(a, p, st);
  if (a.M <= 32) return run_swap<32>(a, p, st);
  if (a.M <= 64) return run_swap<64>(a, p, st);
  return run_swap<128>(a, p, st);
}

}  // namespace upipe
