// Rotary positions with several axes (text: one; images: height, width; video: time, height, width)
// between the projection and the attention core, forward and (by the negative angle) backward.
//
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),   t = position[axis(j)] * inv_freq(j)
// for the rotary pairs j of every head's row: elements (j, j + R/2), or (2j, 2j + 1).
//
// The angle is reduced in integers.  The host turns inv_freq / 2 pi into a 64-bit fraction of a turn, so
// position * fraction modulo 2^64 is one integer product whose high half is the angle within its
// turn, however far the position.  Its high 32 bits become x in [-1, 1), the angle over pi, for sincospif.  The
// angle is off by at most 2^-26 of a turn (x in fp32) plus 2^-52 of the turns made (the 53-bit frequency: 2^-23 of a
// turn at position 2^31 and a radian per position), where an fp32 product of a position of five million
// would be off by whole radians.
//
// A thread owns 16 elements of a row (8 pairs, two 16-byte vectors) of one token and walks over heads:
// the sines and cosines, which all heads of a token share, are computed once.  Rows are read and
// written through their own head and token strides, so the kernel reads the projection's output token
// by token and writes the attention core's operand head by head (or back) in the same pass.  Bound by
// HBM: 4 bytes per element.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace upipe {

namespace {

struct RopeSide {
  const bf16* in;
  bf16* out;
  int64_t in_head, in_tok, out_head, out_tok;
};

struct RopeParams {
  RopeSide s[2];  // queries, keys
  int n_q, n_all;
  int units, rot_units;  // 16-element units of a row, and those of them that are rotated
  int half;              // rotary pairs
  int adjacent;
  int heads_per_block;
  int64_t tokens;
  const int32_t* pos;    // [n_axes][tokens]
  uint64_t frac[kRopeMaxPairs];  // inv_freq / 2 pi, in units of 2^-64 turns
  uint8_t axis[kRopeMaxPairs];
};

struct F16 {
  float a[8], b[8];
};

__device__ __forceinline__ void unpack(const uint4& q, float (&f)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

__global__ void __launch_bounds__(256) k_rope(const __grid_constant__ RopeParams p) {
  const int per_block = blockDim.x / p.units;  // tokens
  const int tl = threadIdx.x / p.units, u = threadIdx.x - tl * p.units;
  const int64_t tok = (int64_t)blockIdx.x * per_block + tl;
  grid_dep_wait();  // before any thread leaves: this grid must not complete before the one that it follows
  if (tl >= per_block || tok >= p.tokens) return;
  const bool rot = u < p.rot_units;
  // the unit's two vectors: (j.., j + R/2..) of a split row, 16 neighbours otherwise
  const bool split = rot && !p.adjacent;
  const int e0 = split ? 8 * u : 16 * u, e1 = split ? p.half + 8 * u : 16 * u + 8;
  float cs[8], sn[8];
  if (rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = 8 * u + i;
      const int32_t pv = p.pos[(int64_t)p.axis[j] * p.tokens + tok];
      const uint32_t turn = (uint32_t)(((uint64_t)(int64_t)pv * p.frac[j]) >> 32);
      sincospif((float)(int32_t)turn * 4.656612873077393e-10f, &sn[i], &cs[i]);  // * 2^-31
    }
  }
  const int h0 = blockIdx.y * p.heads_per_block, h1 = min(p.n_all, h0 + p.heads_per_block);
  // two heads at a time, their loads in flight together (110 -> 106.7 us at 32768 tokens of 32 + 8 heads, 6.3 TB/s)
  for (int hb = h0; hb < h1; hb += 2) {
    uint4 v0[2], v1[2];
    bf16* dst[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int h = hb + k;
      if (h < h1) {
        const RopeSide& s = p.s[h >= p.n_q];
        const int hl = h >= p.n_q ? h - p.n_q : h;
        const bf16* src = s.in + hl * s.in_head + tok * s.in_tok;
        dst[k] = s.out + hl * s.out_head + tok * s.out_tok;
        v0[k] = *reinterpret_cast<const uint4*>(src + e0);
        v1[k] = *reinterpret_cast<const uint4*>(src + e1);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (hb + k < h1) {
        if (rot) {
          float a[8], b[8];
          unpack(v0[k], a);
          unpack(v1[k], b);
          if (split) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x = a[i], y = b[i];
              a[i] = x * cs[i] - y * sn[i];
              b[i] = y * cs[i] + x * sn[i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = a[2 * i], y = a[2 * i + 1];
              a[2 * i] = x * cs[i] - y * sn[i];
              a[2 * i + 1] = y * cs[i] + x * sn[i];
              const float z = b[2 * i], t = b[2 * i + 1];
              b[2 * i] = z * cs[4 + i] - t * sn[4 + i];
              b[2 * i + 1] = t * cs[4 + i] + z * sn[4 + i];
            }
          }
          v0[k] = pack(a);
          v1[k] = pack(b);
        }
        *reinterpret_cast<uint4*>(dst[k] + e0) = v0[k];
        *reinterpret_cast<uint4*>(dst[k] + e1) = v1[k];
      }
    }
  }
}

// inv_freq as a fraction of a turn in units of 2^-64 (modulo whole turns, which integer positions
// do not see).
uint64_t turn_fraction(double inv_freq) {
  const double turns = inv_freq / 6.283185307179586476925;
  double f = turns - std::floor(turns);
  if (!(f < 1.0)) f = 0.0;
  const double scaled = f * 4294967296.0, hi = std::floor(scaled);  // powers of two and their differences are exact
  return ((uint64_t)hi << 32) | (uint64_t)((scaled - hi) * 4294967296.0);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
  if (a.tokens <= 0 || a.side[0].heads + a.side[1].heads <= 0) return cudaSuccess;
  RopeParams p{};
  for (int i = 0; i < 2; ++i) {
    const RopeTensor& t = a.side[i];
    p.s[i] = RopeSide{t.in, t.out, t.in_head, t.in_tok, t.out_head, t.out_tok};
  }
  p.n_q = a.side[0].heads;
  p.n_all = p.n_q + a.side[1].heads;
  p.units = a.head_dim / 16;
  p.rot_units = a.rotary_dim / 16;
  p.half = a.rotary_dim / 2;
  p.adjacent = a.adjacent;
  p.tokens = a.tokens;
  p.pos = a.pos;
  for (int j = 0; j < p.half; ++j) {
    const uint64_t f = turn_fraction(a.inv_freq[j]);
    p.frac[j] = a.inverse ? 0 - f : f;
    p.axis[j] = a.axis[j];
  }
  const int per_block = 256 / p.units;
  const int64_t bx = ceil_div(a.tokens, per_block);
  // few tokens: the heads are spread over blocks too, until there are about 8 blocks per SM
  const int64_t want = ceil_div((int64_t)sm_count() * 8, bx);
  p.heads_per_block = (int)ceil_div(p.n_all, std::min<int64_t>(want, p.n_all));
  const dim3 grid((unsigned)bx, (unsigned)ceil_div(p.n_all, p.heads_per_block));
  const cudaError_t e = launch_pdl(k_rope, grid, dim3(per_block * p.units), 0, st, p);
  note_launch();
  return e;
}

}  // namespace upipe
