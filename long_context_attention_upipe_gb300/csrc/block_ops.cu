// C-ABI entry points of the operators around the attention layer and the MLP: argument checks on the
// host, then one or two launches.  Nothing throws: the only allocation is the sort of grad_clip's
// ranges, and its failure becomes a status.
#include <cmath>
#include <new>
#include <algorithm>
#include <vector>

#include "checks.h"
#include "common.cuh"
#include "internal.h"

using namespace upipe;

namespace {

constexpr int64_t kMaxNormCols = 32768;

upipe_status_t check_norm(int64_t rows, int64_t d) {
  if (rows < 0 || rows > INT32_MAX || d <= 0) return UPIPE_ERR_INVALID_ARG;
  if (d % 8 || d > kMaxNormCols) return UPIPE_ERR_UNSUPPORTED;
  return UPIPE_OK;
}

upipe_status_t check_rope_side(const upipe_rope_tensor_t* t, int64_t tokens, int head_dim, HeadRows& in, HeadRows& out) {
  if (t->n_heads < 0) return UPIPE_ERR_INVALID_ARG;
  if (t->n_heads == 0) return UPIPE_OK;
  if (!t->in || !t->out) return UPIPE_ERR_INVALID_ARG;
  in = rows_of(t->in, t->n_heads, tokens, t->in_head_stride, t->in_token_stride, head_dim);
  out = rows_of(t->out, t->n_heads, tokens, t->out_head_stride, t->out_token_stride, head_dim);
  if (in.hs < 0 || in.ts < 0 || out.hs < 0 || out.ts < 0) return UPIPE_ERR_INVALID_ARG;
  if (!rows_disjoint(out.heads, tokens, out.hs, out.ts, head_dim)) return UPIPE_ERR_INVALID_ARG;
  if (in.hs % 8 || in.ts % 8 || out.hs % 8 || out.ts % 8) return UPIPE_ERR_UNSUPPORTED;
  if (!aligned16(t->in) || !aligned16(t->out)) return UPIPE_ERR_ALIGNMENT;
  if (!in.same(out) && rows_may_meet(in, out)) return UPIPE_ERR_INVALID_ARG;
  return UPIPE_OK;
}

RopeTensor rope_side(const upipe_rope_tensor_t* t) {
  if (!t || t->n_heads == 0) return RopeTensor{};
  return RopeTensor{reinterpret_cast<const bf16*>(t->in), reinterpret_cast<bf16*>(t->out), t->in_head_stride,
                    t->in_token_stride, t->out_head_stride, t->out_token_stride, t->n_heads};
}

}  // namespace

extern "C" {

upipe_status_t upipe_attn_rms_norm_fwd(int64_t rows, int64_t d, float eps, const uint16_t* x, const uint16_t* residual,
                                       const uint16_t* w, uint16_t* h, uint16_t* y, uint8_t* q, float* scales,
                                       float* rstd, void* stream) {
  upipe_status_t s = check_norm(rows, d);
  if (s != UPIPE_OK) return s;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return UPIPE_ERR_INVALID_ARG;
  if (rows == 0) return UPIPE_OK;  // buffers of no elements may be NULL
  if (!x || !w || (!y && !q) || (!q != !scales) || (!residual != !h)) return UPIPE_ERR_INVALID_ARG;
  if (q && d % 16) return UPIPE_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(w) || !aligned16(h) || !aligned16(y) || !aligned16(q) ||
      !aligned16(scales) || !aligned16(rstd))
    return UPIPE_ERR_ALIGNMENT;
  const int64_t n = rows * d * 2;
  const int64_t sb = (d + 127) / 128 * rows * 4;
  if (!outputs_apart({{h, n, true}, {y, n, true}, {q, n / 2}, {scales, sb}, {rstd, rows * 4}},
                     {{x, n, true}, {residual, n, true}, {w, d * 2}}))
    return UPIPE_ERR_INVALID_ARG;
  RmsNormArgs a{rows, (int)d, eps, reinterpret_cast<const bf16*>(x), reinterpret_cast<const bf16*>(residual),
                reinterpret_cast<const bf16*>(w), reinterpret_cast<bf16*>(h), reinterpret_cast<bf16*>(y), q, scales, rstd};
  return finish(launch_rms_fwd(a, (cudaStream_t)stream));
}

upipe_status_t upipe_attn_rms_norm_workspace_size(int64_t rows, int64_t d, size_t* bytes) {
  upipe_status_t s = check_norm(rows, d);
  if (s != UPIPE_OK) return s;
  if (!bytes) return UPIPE_ERR_INVALID_ARG;
  *bytes = rms_bwd_workspace(rows, (int)d);
  return UPIPE_OK;
}

upipe_status_t upipe_attn_rms_norm_bwd(int64_t rows, int64_t d, const uint16_t* dy, const uint16_t* h, const uint16_t* w,
                                       const float* rstd, const uint16_t* dres, uint16_t* dx, float* dw, void* ws,
                                       size_t ws_bytes, void* stream) {
  upipe_status_t s = check_norm(rows, d);
  if (s != UPIPE_OK) return s;
  if (!w || !dw || !ws || (rows && (!dy || !h || !rstd || !dx))) return UPIPE_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(h) || !aligned16(w) || !aligned16(rstd) || !aligned16(dres) || !aligned16(dx) ||
      !aligned16(dw) || !aligned16(ws))
    return UPIPE_ERR_ALIGNMENT;
  const size_t need = rms_bwd_workspace(rows, (int)d);
  if (ws_bytes < need) return UPIPE_ERR_WORKSPACE_TOO_SMALL;
  const int64_t n = rows * d * 2;
  if (!outputs_apart({{dx, n, true}, {dw, d * 4}, {ws, (int64_t)need}},
                     {{dy, n, true}, {h, n, true}, {dres, n, true}, {w, d * 2}, {rstd, rows * 4}}))
    return UPIPE_ERR_INVALID_ARG;
  RmsNormBwdArgs a{rows, (int)d, reinterpret_cast<const bf16*>(dy), reinterpret_cast<const bf16*>(h),
                   reinterpret_cast<const bf16*>(w), rstd, reinterpret_cast<const bf16*>(dres),
                   reinterpret_cast<bf16*>(dx), dw};
  return finish(launch_rms_bwd(a, reinterpret_cast<float*>(ws), (cudaStream_t)stream));
}

upipe_status_t upipe_attn_fp8_quantize(int64_t rows, int64_t cols, int32_t block_rows, const uint16_t* x, uint8_t* q,
                                       float* scales, void* stream) {
  if (rows < 0 || rows > INT32_MAX || cols <= 0 || cols > INT32_MAX - 128) return UPIPE_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != 128) return UPIPE_ERR_INVALID_ARG;
  if (cols % 16) return UPIPE_ERR_UNSUPPORTED;
  if (rows == 0) return UPIPE_OK;
  if (!x || !q || !scales) return UPIPE_ERR_INVALID_ARG;
  if (ceil_div(rows, 128) * ceil_div(cols, 128) > INT32_MAX) return UPIPE_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scales)) return UPIPE_ERR_ALIGNMENT;
  const int64_t sb = ceil_div(rows, (int64_t)block_rows) * ceil_div(cols, 128) * 4;
  if (!outputs_apart({{q, rows * cols}, {scales, sb}}, {{x, 2 * rows * cols}})) return UPIPE_ERR_INVALID_ARG;
  return finish(launch_quantize(rows, (int)cols, block_rows, reinterpret_cast<const bf16*>(x), q, scales,
                                     (cudaStream_t)stream));
}

upipe_status_t upipe_attn_rope(const upipe_rope_desc_t* desc, int64_t tokens, const int32_t* positions,
                               const upipe_rope_tensor_t* q, const upipe_rope_tensor_t* k, void* stream) {
  if (!desc || !q || tokens < 0 || tokens > INT32_MAX) return UPIPE_ERR_INVALID_ARG;
  const int R = desc->rotary_dim;
  if (desc->head_dim <= 0 || R <= 0 || R > desc->head_dim || desc->n_axes < 1 || desc->n_axes > 4 ||
      (desc->adjacent != 0 && desc->adjacent != 1) || (desc->inverse != 0 && desc->inverse != 1))
    return UPIPE_ERR_INVALID_ARG;
  if (desc->head_dim % 16 || R % 16 || desc->head_dim > 2 * kRopeMaxPairs) return UPIPE_ERR_UNSUPPORTED;
  for (int j = 0; j < R / 2; ++j)
    if (!std::isfinite(desc->inv_freq[j]) || desc->axis[j] >= desc->n_axes) return UPIPE_ERR_INVALID_ARG;
  if (tokens == 0) return UPIPE_OK;
  if (!positions) return UPIPE_ERR_INVALID_ARG;
  HeadRows rows[4] = {};
  upipe_status_t s = check_rope_side(q, tokens, desc->head_dim, rows[0], rows[1]);
  if (s == UPIPE_OK && k) s = check_rope_side(k, tokens, desc->head_dim, rows[2], rows[3]);
  if (s != UPIPE_OK) return s;
  // one launch: neither output may touch the other tensor
  if (k && q->n_heads && k->n_heads &&
      (rows_may_meet(rows[1], rows[2]) || rows_may_meet(rows[1], rows[3]) || rows_may_meet(rows[0], rows[3])))
    return UPIPE_ERR_INVALID_ARG;
  if (q->n_heads > 65535 - (k ? k->n_heads : 0)) return UPIPE_ERR_UNSUPPORTED;
  if (!aligned16(positions)) return UPIPE_ERR_ALIGNMENT;
  for (int i = 1; i < 4; i += 2)
    if (rows[i].base && overlaps(rows[i].base, rows[i].bytes(), positions, 4 * tokens * desc->n_axes))
      return UPIPE_ERR_INVALID_ARG;
  RopeArgs a{};
  a.head_dim = desc->head_dim;
  a.rotary_dim = R;
  a.n_axes = desc->n_axes;
  a.adjacent = desc->adjacent;
  a.inverse = desc->inverse;
  a.inv_freq = desc->inv_freq;
  a.axis = desc->axis;
  a.tokens = tokens;
  a.pos = positions;
  a.side[0] = rope_side(q);
  a.side[1] = rope_side(k);
  return finish(launch_rope(a, (cudaStream_t)stream));
}

upipe_status_t upipe_attn_grad_clip_workspace_size(int32_t count, size_t* bytes) {
  if (count < 0 || !bytes) return UPIPE_ERR_INVALID_ARG;
  *bytes = grad_clip_workspace(count);
  return UPIPE_OK;
}

upipe_status_t upipe_attn_grad_clip(const upipe_grad_tensor_t* tensors, int32_t count, float max_norm, float* norm,
                                    void* ws, size_t ws_bytes, void* stream) {
  if (count < 0 || (count > 0 && !tensors) || !norm || !ws || !(max_norm > 0.f)) return UPIPE_ERR_INVALID_ARG;
  if (!aligned16(norm) || !aligned16(ws)) return UPIPE_ERR_ALIGNMENT;
  if (ws_bytes < grad_clip_workspace(count)) return UPIPE_ERR_WORKSPACE_TOO_SMALL;
  try {
    struct Range { uintptr_t lo, hi; };
    std::vector<GradTensor> t((size_t)count);
    std::vector<int> idx;
    std::vector<Range> r;
    idx.reserve((size_t)count);
    r.reserve(2 * (size_t)count + 2);
    const uintptr_t pn = reinterpret_cast<uintptr_t>(norm), pw = reinterpret_cast<uintptr_t>(ws);
    r.push_back(Range{pn, pn + sizeof(float)});
    r.push_back(Range{pw, pw + grad_clip_workspace(count)});
    for (int i = 0; i < count; ++i) {
      const upipe_grad_tensor_t& e = tensors[i];
      if (e.n < 0 || e.n > (int64_t)1 << 42 || e.grad_dtype < 0 || e.grad_dtype > 1 || e.out_dtype < 0 || e.out_dtype > 1)
        return UPIPE_ERR_INVALID_ARG;
      if (e.n == 0) continue;
      void* out = e.out ? e.out : const_cast<void*>(e.grad);
      const int out_dtype = e.out ? e.out_dtype : e.grad_dtype;
      if (!e.grad || (out == e.grad && out_dtype != e.grad_dtype)) return UPIPE_ERR_INVALID_ARG;
      if (!aligned16(e.grad) || !aligned16(out)) return UPIPE_ERR_ALIGNMENT;
      t[i] = GradTensor{e.grad, out, e.n, e.grad_dtype, out_dtype};
      idx.push_back(i);
      const uintptr_t g = reinterpret_cast<uintptr_t>(e.grad), o = reinterpret_cast<uintptr_t>(out);
      r.push_back(Range{g, g + (uintptr_t)(e.n * (e.grad_dtype ? 2 : 4))});
      if (o != g) r.push_back(Range{o, o + (uintptr_t)(e.n * (out_dtype ? 2 : 4))});
    }
    // a tensor listed twice would be scaled twice, by blocks that race; so would one over the workspace
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    for (size_t i = 1; i < r.size(); ++i)
      if (r[i].lo < r[i - 1].hi) return UPIPE_ERR_INVALID_ARG;
    return finish(launch_grad_clip(t.data(), idx.data(), (int)idx.size(), max_norm, norm,
                                        reinterpret_cast<double*>(ws), (cudaStream_t)stream));
  } catch (const std::bad_alloc&) {
    return cuda_status(cudaErrorMemoryAllocation);
  }
}

upipe_status_t upipe_attn_gemm_fp8_nt(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda,
                                      const float* a_scale, int64_t a_scale_ld, const uint8_t* B, int64_t ldb,
                                      const float* b_scale, void* C, int64_t ldc, int32_t c_dtype, void* stream) {
  if (M < 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX || lda < K || ldb < K || ldc < N ||
      a_scale_ld < M || (c_dtype != 0 && c_dtype != 1))
    return UPIPE_ERR_INVALID_ARG;
  if (K % 16 || N % 8 || lda % 16 || ldb % 16 || ldc % 8) return UPIPE_ERR_UNSUPPORTED;
  if (ceil_div(M, 256) * ceil_div(N, 128) > INT32_MAX / 2) return UPIPE_ERR_UNSUPPORTED;  // tiles are counted in 32 bits
  if (M == 0) return UPIPE_OK;
  if (!A || !a_scale || !B || !b_scale || !C) return UPIPE_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(B) || !aligned16(C) || !aligned16(a_scale) || !aligned16(b_scale))
    return UPIPE_ERR_ALIGNMENT;
  const int64_t c_bytes = ((M - 1) * ldc + N) * (c_dtype ? 2 : 4);
  const int64_t nkb = ceil_div(K, 128);
  if (overlaps(C, c_bytes, A, (M - 1) * lda + K) || overlaps(C, c_bytes, B, (N - 1) * ldb + K) ||
      overlaps(C, c_bytes, a_scale, ((nkb - 1) * a_scale_ld + M) * 4) || overlaps(C, c_bytes, b_scale, ceil_div(N, 128) * nkb * 4))
    return UPIPE_ERR_INVALID_ARG;
  const Fp8GemmArgs g{M, N, K, A, lda, a_scale, a_scale_ld, B, ldb, b_scale, C, ldc, c_dtype};
  return finish(launch_gemm_fp8(g, (cudaStream_t)stream));
}

}  // extern "C"
