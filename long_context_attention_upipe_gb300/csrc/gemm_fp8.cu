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
// ... 128 of them), so the tensor core's rows are full whatever the batch.
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

// Shared memory from its next multiple of 1024.  An offset, not a rounded address: a pointer that comes from an integer
// has lost its address space, and every access through it goes by the generic path (8192 x 28672 x 4096: 1 to 2%,
// 1000 x 5120 x 8192 40.4 -> 38.0 us, 128 x 5120 x 8192 19.0 -> 16.4).
__device__ __forceinline__ uint8_t* align_smem(uint8_t* p) { return p + ((0u - smem_u32(p)) & 1023); }

// ------------------------------------------------------------------------------------------------
// few rows of A: weights on the MMA's rows, TN tokens on its columns, K split over a cluster
// ------------------------------------------------------------------------------------------------
// One CTA per 128 weight rows, TN tokens and share of K:
//   warp 0      TMA producer over a ring of ST stages (128 x 128 weights, TN x 128 tokens)
//   warp 1      MMA issuer: 4 MMAs (M128 N TN K32) per block of K into one of NBUF TMEM accumulators
//   warps 2-3   the blocks' scales (token's times weight block's), four blocks of K at a time
//   warps 4..   scaling: one weight row (TMEM lane) per thread, its tokens' sums in registers
// Bound by the weights' bytes: enough CTAs have to stream at once, so K is split over a cluster of up to 8
// CTAs while that fits on the SMs at once.  Each CTA then sends its sums to the CTAs that own the tokens
// (token i belongs to CTA i % splits) through distributed shared memory, and the owners add them in the order
// of the shares.  The accumulators are narrow here, so there are 4 to 8 of them: the chain from an MMA to its
// accumulator's release (about 900 clocks) is long against the block's MMA (2 TN clocks), and its bytes
// arrive every 800.
template <int TN>
struct SwapLayout {
  static constexpr int STAGES = TN == 16 ? 5 : TN == 64 ? 3 : 4;
  static constexpr int NBUF = TN <= 32 ? 8 : 4;
  static constexpr int WARPS = TN <= 32 ? 4 : 8;   // scaling warps
  static constexpr int CT = TN * 4 / WARPS;        // tokens of a scaling thread
  static constexpr int THREADS = 128 + 32 * WARPS;
  static constexpr uint32_t W = 128 * 128, T = TN * 128, STAGE = W + T;
  static constexpr uint32_t SC = STAGES * STAGE;   // per group: 4 rows of TN scales
  static constexpr uint32_t SCSLOT = 4 * TN * 4;
  static constexpr uint32_t RED = SC + 4 * SCSLOT;  // [splits][ceil(TN / splits)][128] sums for the owned tokens
  static constexpr uint32_t BAR = RED + (TN + 6) * 128 * 4;
  static constexpr uint32_t BYTES = BAR + 512;
  static constexpr uint32_t TMEM = NBUF * TN;       // 128 ... 512, a power of two
};

template <int TN>
__global__ void __launch_bounds__(SwapLayout<TN>::THREADS)
    k_gemm_fp8_swap(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tt, Fp8Params p, int splits) {
  using L = SwapLayout<TN>;
  constexpr int ST = L::STAGES, NB = L::NBUF, CT = L::CT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR);
  uint64_t* full = bars;                // [ST]
  uint64_t* empty = bars + ST;          // [ST]
  uint64_t* acc_full = bars + 2 * ST;   // [NB]
  uint64_t* acc_empty = acc_full + NB;  // [NB]
  uint64_t* sc_full = acc_empty + NB;   // [4]
  uint64_t* sc_empty = sc_full + 4;     // [4]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sc_empty + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sc_empty + 5);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = splits > 1 ? (int)tc::cluster_ctarank() : 0;
  const int tile = blockIdx.x / splits;
  const int64_t n0 = (int64_t)tile * 128, m0 = (int64_t)blockIdx.y * TN;
  // this CTA's blocks of K: [kb0, kb0 + nkb), shares that differ by one block at most
  const int kb0 = (int)((int64_t)p.nkb * rank / splits), nkb = (int)((int64_t)p.nkb * (rank + 1) / splits) - kb0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) {
      tc::mbar_init(&acc_full[i], 1);
      tc::mbar_init(&acc_empty[i], L::WARPS);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&sc_full[i], 64);
      tc::mbar_init(&sc_empty[i], L::WARPS);
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
  if (splits > 1) tc::cluster_arrive();  // (A) this CTA runs: its shared memory may be written
  grid_dep_wait();

  float acc[CT];
  bool ok = true;
  const int t0 = warp >= 4 ? ((warp - 4) >> 2) * CT : 0;  // first token of a scaling thread
  const int wrow = 32 * (warp & 3) + lane;                // its weight row
  if (warp == 0) {
    tc::prefetch_tmap(&tw);
    tc::prefetch_tmap(&tt);
    const bool leader = tc::elect_one();
    const uint32_t emptya = smem_u32(empty);
    int s = 0;
    uint32_t ph = 1, turns = 0;  // parity of the stage's previous release: the first turn needs none
#pragma unroll 1
    for (int kb = 0; kb < nkb; ++kb) {
      ok = tc::mbar_wait_addr(emptya + s * 8, ph, abort_flag, p.wait_ns) && ok;
      if (leader && ok) {
        ++turns;
        uint8_t* st = smem + s * L::STAGE;
        tc::mbar_arrive_expect_tx(&full[s], L::STAGE);
        tc::tma_load_2d(st, &tw, &full[s], (kb0 + kb) * kBlk, (int)n0);
        tc::tma_load_2d(st + L::W, &tt, &full[s], (kb0 + kb) * kBlk, (int)m0);
      }
      __syncwarp();
      if (++s == ST) { s = 0; ph ^= 1; }
    }
    if (leader) tc::drain_ring(smem_u32(full), turns, ST);
  } else if (warp == 1) {
    constexpr uint32_t idesc = tc::idesc_e4m3(128, TN);
    const uint64_t w0 = tc::sdesc_sw128(smem_u32(smem), 16, 1024), x0 = tc::sdesc_add(w0, L::W);
    const uint32_t fulla = smem_u32(full), acce = smem_u32(acc_empty);
    const bool leader = tc::elect_one();
    int s = 0, buf = 0;
    uint32_t ph = 0, eph = 1, turns = 0;
#pragma unroll 1
    for (int kb = 0; kb < nkb; ++kb) {
      ok = tc::mbar_wait_addr(acce + buf * 8, eph, abort_flag, p.wait_ns) && ok;
      ok = tc::mbar_wait_addr(fulla + s * 8, ph, abort_flag, p.wait_ns) && ok;
      tc::fence_after_sync();
      const uint64_t wd = tc::sdesc_add(w0, s * L::STAGE), xd = tc::sdesc_add(x0, s * L::STAGE);
      const uint32_t d = tmem + buf * TN;
      if (leader && ok) {
        ++turns;
#pragma unroll
        for (int k = 0; k < kBlk / 32; ++k)
          tc::mma_ss_f8(d, tc::sdesc_add(wd, k * 32), tc::sdesc_add(xd, k * 32), idesc, k > 0);
        tc::mma_commit(&acc_full[buf]);
        tc::mma_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == ST) { s = 0; ph ^= 1; }
      if (++buf == NB) { buf = 0; eph ^= 1; }
    }
    if (leader) {
      tc::drain_ring(smem_u32(empty), turns, ST);
      tc::drain_ring(smem_u32(acc_full), turns, NB);
    }
  } else if (warp < 4) {
    // tokens j and j + 64
    const int j = threadIdx.x - 64;
    const float* sb = p.sb + (int64_t)tile * p.nkb + kb0;
    const bool in0 = j < TN && m0 + j < p.M, in1 = j + 64 < TN && m0 + j + 64 < p.M;
    const float* sa = p.sa + (int64_t)kb0 * p.lds + m0 + j;
    float v0[4], v1[4];
    auto fetch = [&](int kb) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = kb + u < nkb;
        const float w = in ? sb[kb + u] : 0.f;
        v0[u] = in && in0 ? sa[(int64_t)(kb + u) * p.lds] * w : 0.f;
        v1[u] = in && in1 ? sa[(int64_t)(kb + u) * p.lds + 64] * w : 0.f;
      }
    };
    fetch(0);
    int slot = 0;
    uint32_t ph = 1;
    for (int kb = 0; kb < nkb; kb += 4) {
      ok = tc::mbar_wait(&sc_empty[slot], ph, abort_flag, nullptr, p.wait_ns) && ok;
      if (!ok) break;
      float* dst = reinterpret_cast<float*>(smem + L::SC + slot * L::SCSLOT);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (j < TN) dst[u * TN + j] = v0[u];
        if (j + 64 < TN) dst[u * TN + j + 64] = v1[u];
      }
      tc::mbar_arrive(&sc_full[slot]);
      fetch(kb + 4);
      if (++slot == 4) { slot = 0; ph ^= 1; }
    }
  } else {
#pragma unroll
    for (int i = 0; i < CT; ++i) acc[i] = 0.f;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + t0;
    const uint32_t scf = smem_u32(sc_full), sce = smem_u32(sc_empty), accf = smem_u32(acc_full), acce = smem_u32(acc_empty);
    int slot = 0, buf = 0;
    uint32_t sph = 0, aph = 0;
#pragma unroll 1
    for (int kb = 0; kb < nkb; ++kb) {
      const int u = kb & 3;
      if (u == 0) ok = tc::mbar_wait_addr(scf + slot * 8, sph, abort_flag, p.wait_ns) && ok;
      const float4* sc = reinterpret_cast<const float4*>(smem + L::SC + slot * L::SCSLOT + (u * TN + t0) * 4);
      ok = tc::mbar_wait_addr(accf + buf * 8, aph, abort_flag, p.wait_ns) && ok;
      __syncwarp();
      tc::fence_after_sync();
#pragma unroll
      for (int g = 0; g < CT / 16; ++g) {
        uint32_t v[16];
        tc::tmem_ld16_wait(lane_addr + buf * TN + g * 16, v);
        if (g == CT / 16 - 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0 && ok) tc::mbar_arrive_addr(acce + buf * 8);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 s4 = sc[(g * 16 + i) / 4];
          acc[g * 16 + i] += __uint_as_float(v[i]) * s4.x;
          acc[g * 16 + i + 1] += __uint_as_float(v[i + 1]) * s4.y;
          acc[g * 16 + i + 2] += __uint_as_float(v[i + 2]) * s4.z;
          acc[g * 16 + i + 3] += __uint_as_float(v[i + 3]) * s4.w;
        }
      }
      if (++buf == NB) { buf = 0; aph ^= 1; }
      if (u == 3) {
        __syncwarp();
        if (lane == 0 && ok) tc::mbar_arrive_addr(sce + slot * 8);
        if (++slot == 4) { slot = 0; sph ^= 1; }
      }
    }
  }
  __syncwarp();
  grid_dep_trigger();

  auto store = [&](int token, int64_t n, float v) {  // neighbouring lanes hold neighbouring columns of C
    const int64_t at = (m0 + token) * p.ldc + n;
    if (p.c_bf16) reinterpret_cast<bf16*>(p.c)[at] = __float2bfloat16_rn(v);
    else reinterpret_cast<float*>(p.c)[at] = v;
  };
  if (splits == 1) {
    if (warp >= 4 && n0 + wrow < p.N) {
#pragma unroll
      for (int i = 0; i < CT; ++i)
        if (m0 + t0 + i < p.M) store(t0 + i, n0 + wrow, ok ? acc[i] : __int_as_float(0x7fc00000));
    }
  } else {
    const int per = (TN + splits - 1) / splits;  // tokens of an owner
    tc::cluster_wait();                          // (A)
    if (warp >= 4) {
      const uint32_t red = smem_u32(smem + L::RED) + (rank * per * 128 + wrow) * 4;
      int owner = t0 % splits, slot = t0 / splits;
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        // NaN marks the sums of a CTA that gave up
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::mapa_cluster(red + slot * 512, owner)),
                     "f"(ok ? acc[i] : __int_as_float(0x7fc00000))
                     : "memory");
        if (++owner == splits) { owner = 0; ++slot; }
      }
    }
    tc::cluster_sync();  // all sums have arrived; no CTA touches another's shared memory after this
    const float* red = reinterpret_cast<const float*>(smem + L::RED) + (threadIdx.x & 127);
    const int64_t n = n0 + (threadIdx.x & 127);
    if (n < p.N) {
      for (int slot = threadIdx.x >> 7; slot < per; slot += L::THREADS >> 7) {
        const int token = slot * splits + rank;
        if (token >= TN || m0 + token >= p.M) break;
        float v = 0.f;
        for (int r = 0; r < splits; ++r) v += red[(r * per + slot) * 128];
        store(token, n, v);
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

// Shares of K: as many as let every CTA run at once, one per SM, with at least two blocks of K each.  TN 128
// fills an SM's shared memory, and clusters do not pack all SMs of a GPC then: seven eighths of the SMs.
int swap_splits(int64_t ctas, int nkb, int tn) {
  const int64_t room = tn == 128 ? sm_count() * 7 / 8 : sm_count();
  return (int)std::max<int64_t>(1, std::min<int64_t>({8, room / ctas, nkb / 2}));
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
  const int64_t tiles = ceil_div(a.N, 128), mt = ceil_div(a.M, TN);
  const int splits = swap_splits(tiles * mt, p.nkb, TN);
  e = launch_pdl_cluster(kfn, dim3((unsigned)(tiles * splits), (unsigned)mt), dim3(L::THREADS), smem, st, splits, tw, tt, p, splits);
  note_launch();
  return e;
}

// ------------------------------------------------------------------------------------------------
// CTA pairs: 256 rows of A x BN = 32 NCH columns
// ------------------------------------------------------------------------------------------------
// 12 warps per CTA, persistent, one CTA per SM, a pair (cluster of two) per tile:
//   warp 0      TMA producer: this CTA's 128 rows of A and its half of B's BN columns, ring of 5 or 6 stages
//   warp 1      in the even CTA the MMA issuer: 4 MMAs (M256 BN K32, cta_group::2) per block of K into one of the
//               512 / BN TMEM accumulators, which both CTAs hold for their rows
//   warps 2-3   the blocks' scales, eight blocks of K at a time, into a ring in shared memory (cp.async)
//   warps 4-11  scaling: TMEM lanes 32 * (warp % 4), one half of the columns each, the sums in registers
// A wait that runs out (p.wait_ns) makes its thread give up for good: it loads, issues and arrives no more, so that
// whoever depends on it gives up in turn, and a sum to which every wait came through is a right one; all others leave
// as NaN.
// One commit per block of K says both that its accumulator is ready and that its stage may be filled again:
// the scaling warps wait on the stages' ring.  Block b's stage completes again with block b + STAGES, whose MMAs wait
// for block b + STAGES - ACCS to be handed back, and ACCS <= STAGES: every scaling warp has seen b by then, so none
// can miss a phase.
//
// What bounds it is the scaling warps' own path, about 720 clocks per block of K at BN 256 where its MMAs take 512:
// the wait (120, though the block is ready), the loads and sums (385 until the accumulator is handed back, of which
// 256 are the sums') and the rest.  With neither loads of operands nor MMAs the kernel took 75% of its time; a
// free-running loop of the same loads and sums takes 320, with waits and arrivals 490.  On the way here: an
// arrive.release.cluster waits for every load in flight, so the accumulator is released by a relaxed arrive
// (tcgen05.fence orders the reads of TMEM before it) and the scales are fetched by warps of their own; a one-lane
// issuing loop moves every descriptor into uniform registers, so the whole warp walks it (elect_one); the
// accumulator is released as soon as its last columns are in registers.  Loops are kept short, one block of K per
// turn: the issuer's unrolled over the ring took 12% more, the scaling loop's unrolled by eight 4% (by two, with
// spills, 30%).  An MMA per CTA with the columns multicast to both frees its accumulators without the other CTA,
// but writes half as many bytes again to shared memory: 5% slower.  C leaves by TMA from small boxes: a tile's
// output took 3300 clocks with 16-byte stores, of which 2300 were instructions, and cost 3 to 4% more in all.
// us at 1000 x 5120 x 8192 / 8192 x 28672 x 4096, each step beside the last on a GPU that was not at its power limit:
// one commit and short loops 46.8 -> 42.7 / 735 -> 703, C by TMA -> 40.4 / 684 (with three boxes of 16 columns and a
// sixth stage 3% more), shared addressing -> 38 / 662.  The large size runs at the limit after some seconds (1760 of
// 2070 MHz) and takes 730 to 750 then, 2560 to 2640 TFLOP/s; the other 40 to 41 with cold operands.
// Sixteen scaling warps of a quarter of the columns each: 763.  Tokens on the columns, the kernel above: 171 / 2550 us.
constexpr int kTileThreads = 384;
constexpr int kScSlots = 2, kScGroup = 8;  // ring of scales: groups of eight blocks of K
constexpr int kScRow = 128 + 4;            // a block's scales: of each row, and of 2 x 2 column blocks

// Four bytes (or, with `bytes` 0, a zero) to shared memory without a register in between.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// One arrival of this thread's once its copies so far are there.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int NCH>
struct TileLayout {
  static constexpr int BN = 32 * NCH, CW = BN / 2;  // CW: columns of a scaling warp
  static constexpr uint32_t A = 128 * 128, B = CW * 128, STAGE = A + B;
  static constexpr int STAGES = NCH == 8 ? 5 : 6;  // what fits
  static constexpr int ACCS = 512 / BN;  // accumulators in TMEM
  static constexpr uint32_t SC = STAGES * STAGE;
  static constexpr uint32_t SCSLOT = kScGroup * kScRow * 4;
  static constexpr uint32_t OUT = (SC + kScSlots * SCSLOT + 1023) / 1024 * 1024;
  static constexpr int BC = NCH % 2 ? 16 : 32;      // columns of a box of C in bf16 (a warp's are a multiple); 16 in fp32
  static constexpr uint32_t BOX = 32 * 64;          // 32 rows
  static constexpr uint32_t OUTBOX = 2 * BOX;       // per scaling warp
  static constexpr uint32_t BAR = OUT + 8 * OUTBOX;
  static constexpr uint32_t BYTES = BAR + 256;
};

struct TileSched {
  int tiles_mp, tiles_n, m_fast;  // pairs of 128-row tiles, column tiles, and which of the two is the fast index
};

template <int NCH>
__global__ void __launch_bounds__(kTileThreads, 1)
    k_gemm_fp8_tile(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                    const __grid_constant__ CUtensorMap tcm, Fp8Params p, TileSched sch) {
  using L = TileLayout<NCH>;
  constexpr int ST = L::STAGES, BN = L::BN, CW = L::CW;
  constexpr bool kStraddle = CW % 64 != 0;  // a warp's columns may lie in two weight blocks
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR);
  uint64_t* full = bars;               // [ST]
  uint64_t* empty = bars + ST;                 // [ST]: the stage's MMAs are done, in both CTAs
  uint64_t* acc_empty = bars + 2 * ST;         // [ACCS]
  uint64_t* sc_full = acc_empty + L::ACCS;     // [kScSlots]
  uint64_t* sc_empty = sc_full + kScSlots;    // [kScSlots]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sc_empty + kScSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sc_empty + kScSlots + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = (int)tc::cluster_ctarank();
  const int cid = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
  const int n_tiles = sch.tiles_mp * sch.tiles_n;
  const int nkb = p.nkb;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < L::ACCS; ++i) tc::mbar_init(&acc_empty[i], 16);  // even CTA: both CTAs' 8 scaling warps
    for (int i = 0; i < kScSlots; ++i) {
      tc::mbar_init(&sc_full[i], 64);
      tc::mbar_init(&sc_empty[i], 8);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(tmem_slot, 512);
    tc::tmem_relinquish_pair();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();

  auto decode = [&](int t, int& tm, int& tn) {
    if (sch.m_fast) {
      tm = 2 * (t % sch.tiles_mp) + crank;
      tn = t / sch.tiles_mp;
    } else {
      tm = 2 * (t / sch.tiles_n) + crank;
      tn = t % sch.tiles_n;
    }
  };

  // Launched with 168 registers per thread; the scaling warps rise to 216 (128 of them sums), the others
  // drop to 72: 4 x 72 + 8 x 216 = 12 x 168.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n" ::: "memory");
    if (warp == 0) {
      tc::prefetch_tmap(&ta);
      tc::prefetch_tmap(&tb);
      const bool leader = tc::elect_one();
      const uint32_t emptya = smem_u32(empty), full0 = tc::mapa_cluster(smem_u32(full), 0);
      int s = 0;
      uint32_t ph = 1, turns = 0;  // parity of the stage's previous release: the first turn needs none
      bool ok = true;
      for (int t = cid; t < n_tiles && __all_sync(0xffffffffu, ok); t += n_clusters) {
        int tm, tn;
        decode(t, tm, tn);
#pragma unroll 1
        for (int kb = 0; kb < nkb; ++kb) {
          ok = tc::mbar_wait_addr(emptya + s * 8, ph, abort_flag, p.wait_ns) && ok;
          uint8_t* sa = smem + s * L::STAGE;
          if (leader && ok) {
            ++turns;
            if (crank == 0) tc::mbar_arrive_expect_tx(&full[s], 2 * L::STAGE);  // both CTAs' halves
            tc::tma_load_2d_pair(sa, &ta, full0 + s * 8, kb * kBlk, tm * 128);
            tc::tma_load_2d_pair(sa + L::A, &tb, full0 + s * 8, kb * kBlk, tn * BN + crank * CW);
          }
          __syncwarp();
          if (++s == ST) { s = 0; ph ^= 1; }
        }
      }
      // a stage whose MMAs are done holds neither CTA's loads any more; one whose MMAs never come holds loads that
      // land in microseconds, the limit's second later
      if (leader) tc::drain_ring(emptya, turns, ST);
    } else if (warp == 1 && crank == 0) {
      constexpr uint32_t idesc = tc::idesc_e4m3(256, BN);
      const uint64_t a0 = tc::sdesc_sw128(smem_u32(smem), 16, 1024), b0 = tc::sdesc_add(a0, L::A);
      const uint32_t fulla = smem_u32(full), acce = smem_u32(acc_empty);
      const bool leader = tc::elect_one();
      int s = 0, buf = 0;
      uint32_t ph = 0, eph = 1;
      bool ok = true;
      for (int t = cid; t < n_tiles && __all_sync(0xffffffffu, ok); t += n_clusters) {
#pragma unroll 1
        for (int kb = 0; kb < nkb; ++kb) {
          const bool f = tc::mbar_try_wait_addr(fulla + s * 8, ph), e = tc::mbar_try_wait_addr(acce + buf * 8, eph);
          if (!f) ok = tc::mbar_wait_addr(fulla + s * 8, ph, abort_flag, p.wait_ns) && ok;
          if (!e) ok = tc::mbar_wait_addr(acce + buf * 8, eph, abort_flag, p.wait_ns) && ok;
          tc::fence_after_sync();
          const uint64_t ad = tc::sdesc_add(a0, s * L::STAGE), bd = tc::sdesc_add(b0, s * L::STAGE);
          const uint32_t d = tmem + buf * BN;
          if (leader && ok) {
#pragma unroll
            for (int k = 0; k < kBlk / 32; ++k)
              tc::mma_ss_pair_f8(d, tc::sdesc_add(ad, k * 32), tc::sdesc_add(bd, k * 32), idesc, k > 0);
            tc::mma_commit_pair(&empty[s]);
          }
          __syncwarp();
          if (++s == ST) { s = 0; ph ^= 1; }
          if (++buf == L::ACCS) { buf = 0; eph ^= 1; }
        }
      }
    } else if (warp >= 2) {
      // rows j and j + 64 of this CTA's 128, and (4 threads) the weight blocks under both column halves
      const int j = threadIdx.x - 64;
      const int nblocks = (int)ceil_div(p.N, kBlk);
      int slot = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int t = cid; t < n_tiles && ok; t += n_clusters) {
        int tm, tn;
        decode(t, tm, tn);
        const int64_t ma = (int64_t)tm * 128 + j, mb = ma + 64;
        const float* pa = p.sa + (ma < p.M ? ma : 0);
        const float* pb = p.sa + (mb < p.M ? mb : 0);
        const int blk = (int)(((int64_t)tn * BN + (j >> 1 & 1) * CW) / kBlk) + (j & 1);
        const float* ps = p.sb + (int64_t)min(blk, nblocks - 1) * nkb;
        const uint32_t na = ma < p.M ? 4 : 0, nb = mb < p.M ? 4 : 0, ns = j < 4 ? 4 : 0;  // bytes: 0 writes a zero
#pragma unroll 1
        for (int kb0 = 0; kb0 < nkb; kb0 += kScGroup) {
          ok = tc::mbar_wait_addr(smem_u32(&sc_empty[slot]), ph, abort_flag, p.wait_ns) && ok;
          if (!ok) break;
          uint32_t dst = smem_u32(smem + L::SC + slot * L::SCSLOT) + j * 4;
          const int n = min(kScGroup, nkb - kb0);
#pragma unroll 1
          for (int u = 0; u < n; ++u, dst += kScRow * 4) {
            cp_async4(dst, pa, na);
            cp_async4(dst + 256, pb, nb);
            if (j < 4) cp_async4(dst + 512, ps, ns);
            pa += p.lds;
            pb += p.lds;
            ++ps;
          }
          cp_async_arrive(smem_u32(&sc_full[slot]));
          if (++slot == kScSlots) { slot = 0; ph ^= 1; }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n" ::: "memory");
    const int half = (warp - 4) >> 2;
    const int r = 32 * (warp & 3) + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + half * CW;
    int slot = 0, buf = 0;
    uint32_t sph = 0, aph = 0;
    const uint32_t scf = smem_u32(sc_full), sce = smem_u32(sc_empty), done = smem_u32(empty);
    int st = 0, ob = 0;
    const uint32_t acc0 = tc::mapa_cluster(smem_u32(acc_empty), 0);  // the even CTA's
    bool ok = true;
    for (int t = cid; t < n_tiles; t += n_clusters) {
      int tm, tn;
      decode(t, tm, tn);
      const int64_t n0 = (int64_t)tn * BN + half * CW;
      // the warp's columns lie in one weight block up to chunk `cut` (16 columns each), then in the next
      const int cut = (int)((kBlk - n0 % kBlk) / 16);
      float2 acc[CW / 2];
#pragma unroll
      for (int i = 0; i < CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      ok = __all_sync(0xffffffffu, ok);  // a warp that gave up only fills the rest of its tiles
      const int blocks = ok ? nkb : 0;
#pragma unroll 1
      for (int kb = 0; kb < blocks; ++kb) {
        const int u = kb % kScGroup;
        if (u == 0) ok = tc::mbar_wait_addr(scf + slot * 8, sph, abort_flag, p.wait_ns) && ok;
        const float* sc = reinterpret_cast<const float*>(smem + L::SC + slot * L::SCSLOT) + u * kScRow;
        const float sa = sc[r], sb0 = sc[128 + 2 * half], sb1 = kStraddle ? sc[129 + 2 * half] : 0.f;
        ok = tc::mbar_wait_addr(done + st * 8, aph, abort_flag, p.wait_ns) && ok;
        if (++st == ST) { st = 0; aph ^= 1; }
        __syncwarp();
        tc::fence_after_sync();
        const uint32_t src = lane_addr + buf * BN;
        uint32_t v[2][16];  // the next 16 columns are loaded while these are scaled
        tc::tmem_ld16(src, v[0]);
        const float f0 = sa * sb0, f1 = kStraddle ? sa * sb1 : f0;
        if (u == kScGroup - 1 || kb + 1 == nkb) {
          __syncwarp();
          if (lane == 0 && ok) tc::mbar_arrive_addr(sce + slot * 8);
          if (++slot == kScSlots) { slot = 0; sph ^= 1; }
        }
#pragma unroll
        for (int g = 0; g < NCH; ++g) {
          tc::tmem_ld16_ready(v[g & 1]);
          if (g + 1 < NCH) tc::tmem_ld16(src + (g + 1) * 16, v[(g + 1) & 1]);
          else {
            // everything is in registers: the accumulator may be written again while these are scaled
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0 && ok) tc::mbar_arrive_cluster_relaxed(acc0 + buf * 8);
          }
          const float f = kStraddle && g >= cut ? f1 : f0;
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc[g * 8 + i] = __ffma2_rn(make_float2(__uint_as_float(v[g & 1][2 * i]), __uint_as_float(v[g & 1][2 * i + 1])), f2,
                                        acc[g * 8 + i]);
        }
        if (++buf == L::ACCS) buf = 0;
      }
      if (!ok) {  // a wait that ran out leaves NaN
#pragma unroll
        for (int i = 0; i < CW / 2; ++i) acc[i] = make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
      }
      // C leaves through shared memory by TMA, which drops what lies outside, two boxes per warp in turn; 16-byte chunk j
      // of row r lies at chunk j ^ (r / 2 % 4) of a row of 64 bytes, j ^ (r / 4 % 2) of one of 32 (the map's swizzle,
      // which keeps the writes free of bank conflicts)
      uint8_t* box = smem + L::OUT + (warp - 4) * L::OUTBOX;
      const int mw = tm * 128 + 32 * (warp & 3);
      auto room = [&]() {
        if (lane == 0) tc::bulk_wait_read<1>();
        __syncwarp();
        return box + ob * L::BOX;
      };
      auto leave = [&](const uint8_t* from, int64_t n) {
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (mw < p.M && n < p.N) tc::tma_store_2d(&tcm, from, (int)n, mw);
          tc::bulk_commit();
        }
        ob ^= 1;
      };
      if (p.c_bf16) {
        constexpr int BC = L::BC;
        const int sw = BC == 32 ? (lane >> 1) & 3 : (lane >> 2) & 1;
#pragma unroll
        for (int c = 0; c < CW; c += BC) {
          uint8_t* to = room();
#pragma unroll
          for (int j = 0; j < BC / 8; ++j) {
            const float2* v = &acc[(c + 8 * j) / 2];
            *reinterpret_cast<uint4*>(to + lane * (BC * 2) + ((j ^ sw) << 4)) =
                make_uint4(tc::pack_bf16x2(v[0].x, v[0].y), tc::pack_bf16x2(v[1].x, v[1].y), tc::pack_bf16x2(v[2].x, v[2].y),
                           tc::pack_bf16x2(v[3].x, v[3].y));
          }
          leave(to, n0 + c);
        }
      } else {
        const int sw = (lane >> 1) & 3;
#pragma unroll
        for (int c = 0; c < CW; c += 16) {
          uint8_t* to = room();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2* v = &acc[(c + 4 * j) / 2];
            *reinterpret_cast<float4*>(to + lane * 64 + ((j ^ sw) << 4)) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
          }
          leave(to, n0 + c);
        }
      }
    }
    if (lane == 0) tc::bulk_wait_all();
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // the peer's loads and commits reach into this CTA until it is done too
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, 512);
  }
}

template <int NCH>
cudaError_t run_tile(const Fp8GemmArgs& a, const Fp8Params& p, cudaStream_t st) {
  using L = TileLayout<NCH>;
  CUtensorMap ta, tb, tcm;
  if (!make_tmap_2d_u8(&ta, a.A, a.K, a.M, a.lda, kBlk, 128) || !make_tmap_2d_u8(&tb, a.B, a.K, a.N, a.ldb, kBlk, L::CW) ||
      !make_tmap_2d_out(&tcm, a.C, a.c_bf16, a.N, a.M, a.ldc, a.c_bf16 ? L::BC : 16))
    return cudaErrorInvalidValue;
  auto kfn = k_gemm_fp8_tile<NCH>;
  const size_t smem = L::BYTES + 1024;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  // the fast index sweeps the smaller operand, so the larger one is read from DRAM about once
  const TileSched sch{(int)ceil_div(a.M, 256), (int)ceil_div(a.N, L::BN), a.N > a.M};
  const int64_t units = (int64_t)sch.tiles_mp * sch.tiles_n;
  const unsigned grid = (unsigned)(2 * std::max<int64_t>(1, std::min<int64_t>(units, sm_count() / 2)));
  e = launch_pdl_cluster(kfn, dim3(grid), dim3(kTileThreads), smem, st, 2, ta, tb, tcm, p, sch);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_gemm_fp8(const Fp8GemmArgs& a, cudaStream_t st) {
  if (a.M <= 0) return cudaSuccess;
  Fp8Params p{a.M, a.N, a.K, (int)ceil_div(a.K, kBlk), a.sa, a.lds, a.sb, a.C, a.ldc, a.c_bf16, wait_limit_ns()};
  if (a.M <= 16) return run_swap<16>(a, p, st);
  if (a.M <= 32) return run_swap<32>(a, p, st);
  if (a.M <= 64) return run_swap<64>(a, p, st);
  // The modelled clocks of both kernels.  Tile kernel: the column width whose rounds over all clusters take the
  // least; a block of K takes about 130 + 90 NCH (510 measured at 128 columns, 570 at 160, 850 at 256, each with
  // its share of a tile's ends), a tile's output about 200 NCH.  Tokens on the columns: about 1000 for a block of
  // K, and about 12500 for the ends and the output of every round of CTAs, which is not persistent.  Measured on both
  // sides (us, tile kernel / tokens on the columns): 100 x 1024 x 4096 10.4 / 7.6, 128 x 4096 x 4096 11.4 / 10.6,
  // 128 x 5120 x 8192 18.1 / 16.4; 128 x 28672 x 4096 27.7 / 36.8, 200 x 6144 x 4096 11.8 / 17.9, 256 x 5120 x 8192
  // 18.2 / 34.7; one or two blocks of K: 8192 x 28672 x 128 105 / 518, 4096 x 4096 x 128 11.8 / 39.3, 8192 x 28672 x 256
  // 123 / 567, 128 x 28672 x 256 9.4 / 12.6, 1000 x 512 x 128 and 1024 x 1024 x 256 8.5 / 8.5.
  const int64_t clusters = sm_count() / 2, tm = ceil_div(a.M, 256);
  int best = 8;
  int64_t cost = INT64_MAX;
  for (int c = 8; c >= 4; --c) {
    const int64_t rounds = ceil_div(tm * ceil_div(a.N, 32 * c), clusters);
    const int64_t k = rounds * ((int64_t)p.nkb * (130 + 90 * c) + 200 * c);
    if (k < cost) { cost = k; best = c; }
  }
  const int64_t ctas = ceil_div(a.N, 128) * ceil_div(a.M, 128);
  const int splits = swap_splits(ctas, p.nkb, 128);
  if (ceil_div(a.M, 128) <= 65535 && ceil_div(ctas * splits, sm_count()) * (12500 + ceil_div(p.nkb, splits) * 1000) < 8000 + cost)
    return run_swap<128>(a, p, st);
  switch (best) {
    case 4: return run_tile<4>(a, p, st);
    case 5: return run_tile<5>(a, p, st);
    case 6: return run_tile<6>(a, p, st);
    case 7: return run_tile<7>(a, p, st);
    default: return run_tile<8>(a, p, st);
  }
}

}  // namespace upipe
