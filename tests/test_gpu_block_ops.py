"""Operators around the two blocks against plain 64-bit arithmetic.

Tolerances count roundings.  u = 2^-24 is fp32's, 2^-8 bf16's, 2^-4 e4m3's relative half step (2^-10 absolute
below e4m3's smallest normal number).  A chain of n fp32 additions of terms t_i is off by at most
n u sum|t_i|; the kernels' chains are at most 8 V <= 32 terms of a thread plus 10 levels of a tree, so a
row's sum of squares is within 48 u of itself (all terms positive), 1 / rms within 24 u + 4 u (the reciprocal
root and the division), and y = h * rstd * w within 32 u < 2^-18 before its own rounding.
"""
import math

import pytest
import torch

import long_context_attention_upipe_gb300 as up

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
BF_TINY = 2.0 ** -133      # half of bf16's smallest subnormal step
ROW = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def nan_like(shape, dtype):
    if dtype == torch.float8_e4m3fn:
        return torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda").view(dtype)
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def within(got, want, tol):
    """got (any type) against want and tol (fp64): finite and no element further off than its tolerance."""
    got = got.double()
    assert bool(torch.isfinite(got).all())
    over = (got - want).abs() - tol
    assert float(over.max()) <= 0.0, f"{float(over.max())} over at {int(over.argmax())}"


# ------------------------------------------------------------------------------------------------
# norm
# ------------------------------------------------------------------------------------------------

def norm_ref(x, res, w, eps):
    h = x.double() if res is None else (x.double() + res.double()).bfloat16().double()
    rstd = (h.square().mean(1) + eps).rsqrt()
    return h, rstd, h * rstd[:, None] * w.double()


def scale_ref(y, br=1):
    """Block maxima of |y| over br rows and 128 columns, spread back over the elements."""
    r, c = y.shape
    p = torch.nn.functional.pad(y.abs(), (0, -c % 128, 0, -r % br))
    return p.view(-1, br, p.shape[1] // 128, 128).amax((1, 3))


def spread(s, br, shape):
    return s.repeat_interleave(br, 0)[: shape[0]].repeat_interleave(128, 1)[:, : shape[1]]


def check_q(q, s, y, br, rel):
    """Codes q and scales s [row blocks, column blocks] of the fp64 values y (known within rel)."""
    amax = scale_ref(y, br)
    want = torch.where(amax < 2.0 ** -100, torch.ones_like(amax), amax / 448)
    within(s, want, want * (rel + 4 * U))
    v = y / spread(want, br, y.shape)
    # v / s is known within rel (the values) + rel + 8 u (the scale and its reciprocal); then one rounding
    off = v.abs() * (2 * rel + 8 * U)
    within(q, v, torch.maximum((v.abs() + off) * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) + off)


# rows that end within each step of the threads per row and vectors per thread
SHAPES = [(1, 8), (3, 64), (17, 128), (33, 136), (5, 256), (2, 264), (7, 1040), (130, 4096), (3, 4112), (3, 5120), (3, 5136), (2, 8192),
          (3, 8208), (2, 10240), (2, 10256), (1, 16384), (2, 16400), (1, 32768), (0, 256)]


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_forward(rows, d, residual):
    g = gen(rows * 7 + d)
    x = (3 * randn(g, rows, d)).bfloat16()
    res = randn(g, rows, d).bfloat16() if residual else None
    w = (1 + randn(g, d)).bfloat16()
    eps = 1e-5
    h, rstd, y = norm_ref(x, res, w, eps)
    out, ho, ro = nan_like((rows, d), torch.bfloat16), nan_like((rows, d), torch.bfloat16) if residual else None, nan_like((rows,), torch.float32)
    up.rms_norm_fwd(x, w, out, ro, residual=res, h=ho, eps=eps)
    if rows == 0:
        return
    if residual:
        assert torch.equal(ho.double(), h)
    within(ro, rstd, rstd * ROW)
    within(out, y, y.abs() * (BF + ROW) + BF_TINY)
    if d % 16 == 0:
        q, s, h2 = nan_like((rows, d), torch.float8_e4m3fn), nan_like((-(-d // 128), rows), torch.float32), None if ho is None else torch.empty_like(ho)
        y2 = nan_like((rows, d), torch.bfloat16)
        up.rms_norm_fwd_fp8(x, w, q, s, residual=res, h=h2, eps=eps, y=y2)
        check_q(q, s.t(), y, 1, ROW)
        assert torch.equal(y2, out) and (h2 is None or torch.equal(h2, ho))


def test_norm_in_place_and_zero_rows():
    g = gen(3)
    x, r, w = randn(g, 40, 512).bfloat16(), randn(g, 40, 512).bfloat16(), randn(g, 512).bfloat16()
    x[7] = 0
    r[7] = 0
    y, h = torch.empty_like(x), torch.empty_like(x)
    up.rms_norm_fwd(x, w, y, residual=r, h=h, eps=1e-6)
    assert bool((y[7] == 0).all())                       # a row of zeros: rstd = eps^-1/2, y = 0
    x2, r2 = x.clone(), r.clone()
    up.rms_norm_fwd(x2, w, x2, residual=r2, h=r2, eps=1e-6)  # y over x, the residual stream updated in place
    assert torch.equal(x2, y) and torch.equal(r2, h)
    q, s = nan_like((40, 512), torch.float8_e4m3fn), nan_like((4, 40), torch.float32)
    up.rms_norm_fwd_fp8(x, w, q, s, residual=r, h=h, eps=0.0)
    assert bool((s[:, 8:].isfinite()).all())


def test_norm_keeps_nan_and_infinity_in_their_rows():
    g = gen(4)
    x, w = randn(g, 6, 384).bfloat16(), torch.ones(384, device="cuda").bfloat16()
    x[1, 130] = float("nan")
    x[3, 5] = float("inf")
    y, q, s = torch.empty_like(x), nan_like((6, 384), torch.float8_e4m3fn), nan_like((3, 6), torch.float32)
    up.rms_norm_fwd_fp8(x, w, q, s, y=y)
    assert bool(y[1].isnan().all()) and bool(s[:, 1].isnan().all()) and bool(q[1].float().isnan().all())
    assert bool(y[3, 5].isnan()) and bool((y[3, :5] == 0).all())     # rstd is 0 in a row that holds an infinity
    assert bool(s[0, 3].isnan()) and bool((q[3, 128:].float() == 0).all()) and bool((s[1:, 3] == 1).all())
    for i in (0, 2, 4, 5):
        assert bool(y[i].isfinite().all()) and bool(s[:, i].isfinite().all()) and bool(q[i].float().isfinite().all())


@pytest.mark.parametrize("rows,d", [(1, 8), (3, 64), (300, 128), (33, 136), (5, 256), (2, 264), (7, 1040), (1000, 4096),
                                    (3, 4112), (3, 5120), (3, 5136), (3, 7680), (3, 7688), (2, 8192), (3, 8208), (2, 10240), (2, 10256),
                                    (1, 16384), (2, 16400), (1, 32768), (0, 256),
                                    (2500, 4104), (700, 16384), (2000, 200)])   # more rows than are in flight
@pytest.mark.parametrize("dres", [False, True])
def test_norm_backward(rows, d, dres):
    g = gen(rows + 3 * d)
    h = (2 * randn(g, rows, d)).bfloat16()
    dy, w = randn(g, rows, d).bfloat16(), (1 + randn(g, d)).bfloat16()
    r = randn(g, rows, d).bfloat16() if dres else None
    eps = 1e-5
    rstd = (h.double().square().mean(1) + eps).rsqrt()
    rs = rstd.float()
    dx, dw = nan_like((rows, d), torch.bfloat16), nan_like((d,), torch.float32)
    ws = torch.full((up.rms_norm_workspace_bytes(rows, d),), 255, dtype=torch.uint8, device="cuda")
    up.rms_norm_bwd(dy, h, w, rs, dx, dw, ws, dres=r)
    hd, dyd, R = h.double(), dy.double(), rs.double()[:, None]
    t = dyd * w.double()
    mean = (t * hd).mean(1, keepdim=True) if rows else t[:, :1]
    want = R * (t - hd * R * R * mean) + (r.double() if dres else 0)
    mag = R * (t.abs() + hd.abs() * R * R * ((t * hd).abs().mean(1, keepdim=True) if rows else 0))
    if rows:
        # the dot product is within 48 u of its terms' magnitudes, the rest a handful of roundings of `mag`
        within(dx, want, want.abs() * BF + mag * 64 * U * (1 + BF) + (r.double().abs() * 2 * U if dres else 0) + BF_TINY)
    terms = dyd * hd * R
    within(dw, terms.sum(0), terms.abs().sum(0) * (rows + 64) * U)   # at most rows + 64 additions in any order
    dx2, dw2 = dy.clone(), torch.empty_like(dw)
    up.rms_norm_bwd(dx2, h, w, rs, dx2, dw2, ws, dres=r)             # dx in dy's place, the same sums
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_norm_backward_agrees_with_differences():
    """The gradient of sum(c * y) along random directions against central differences of the 64-bit forward."""
    g = gen(11)
    rows, d, eps = 4, 320, 1e-5
    x, w, c = randn(g, rows, d).bfloat16(), (1 + 0.2 * randn(g, d)).bfloat16(), randn(g, rows, d).bfloat16()
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    up.rms_norm_fwd(x, w, y, rstd, eps=eps)
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(up.rms_norm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    up.rms_norm_bwd(c, x, w, rstd, dx, dw, ws)

    def f(xx, ww):
        return float((c.double() * (xx * (xx.square().mean(1, keepdim=True) + eps).rsqrt() * ww)).sum())

    for seed in range(4):
        vx, vw = randn(gen(100 + seed), rows, d).double(), randn(gen(200 + seed), d).double()
        e = 1e-5
        num = (f(x.double() + e * vx, w.double() + e * vw) - f(x.double() - e * vx, w.double() - e * vw)) / (2 * e)
        got = float((dx.double() * vx).sum() + (dw.double() * vw).sum())
        # dx is rounded to bf16: each term of the sum by 2^-8 of it; the differences' own error is O(e^2)
        assert abs(got - num) <= float((dx.double() * vx).abs().sum()) * BF + 1e-4, (got, num)


# ------------------------------------------------------------------------------------------------
# quantiser and product
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (129, 256), (200, 1040), (1000, 4096), (0, 128)])
@pytest.mark.parametrize("block", [1, 128])
def test_quantize(rows, cols, block):
    g = gen(rows + cols + block)
    x = (randn(g, rows, cols) * torch.exp(2 * randn(g, 1, cols))).bfloat16()
    if rows > 2:
        x[1] = 0
        x[2, :16] = 2.0 ** -120     # its block's maximum is below 2^-100 if nothing else is in it
        x[2, 16:] = 0
    nb = -(-cols // 128)
    q = nan_like((rows, cols), torch.float8_e4m3fn)
    s = nan_like((nb, rows) if block == 1 else (-(-rows // 128), nb), torch.float32)
    up.fp8_quantize(x, q, s, block_rows=block)
    if rows:
        check_q(q, s.t() if block == 1 else s, x.double(), block, 0.0)
        if rows > 2 and block == 1:
            assert bool((s[:, 1:3] == 1).all()) and bool((q[1:3].float() == 0).all())


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_marks_only_the_blocks_that_hold_nan_or_infinity(block):
    x = randn(gen(5), 256, 384).bfloat16()
    x[3, 130], x[200, 300] = float("nan"), float("-inf")
    q = nan_like((256, 384), torch.float8_e4m3fn)
    s = nan_like((3, 256) if block == 1 else (2, 3), torch.float32)
    up.fp8_quantize(x, q, s, block_rows=block)
    per = spread(s.t() if block == 1 else s, block, x.shape)
    bad = torch.zeros_like(x, dtype=torch.bool)
    if block == 1:
        bad[3, 128:256] = bad[200, 256:] = True
    else:
        bad[:128, 128:256] = bad[128:, 256:] = True
    assert bool((per.isfinite() == ~bad).all()) and bool(q.float()[~bad].isfinite().all())
    assert bool(q[3, 130].float().isnan()) and bool(q[200, 300].float().isnan())


def fp8_operands(g, M, N, K, spread_a=1.0):
    a = randn(g, M, K) * torch.exp(spread_a * randn(g, 1, K))
    A = a.clamp(-448, 448).to(torch.float8_e4m3fn)
    B = (8 * randn(g, N, K)).clamp(-448, 448).to(torch.float8_e4m3fn)
    nkb = -(-K // 128)
    sa = torch.exp(randn(g, nkb, M))
    sb = torch.exp(randn(g, -(-N // 128), nkb))
    return A, sa, B, sb


def gemm_ref(A, sa, B, sb):
    """C and the sum of the magnitudes of its terms, in 64 bits."""
    (M, K), N = A.shape, B.shape[0]
    a = A.double() * sa.double().t().repeat_interleave(128, 1)[:, :K]
    b = B.double() * sb.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return a @ b.t(), a.abs() @ b.abs().t()


def check_gemm(C, A, sa, B, sb):
    want, mag = gemm_ref(A, sa, B, sb)
    K = A.shape[1]
    # e4m3 products are exact in fp32.  The tensor core adds 32 of them per instruction to an accumulator of at
    # least 23 bits, truncating: at most 2^-22 of the terms' magnitudes for each of a block's 4 instructions;
    # the blocks' sums are scaled (2 roundings) and added (one each).
    tol = mag * (4 * 2.0 ** -22 + (3 + -(-K // 128)) * U)
    if C.dtype == torch.bfloat16:
        tol = tol * (1 + BF) + want.abs() * BF + BF_TINY
    within(C, want, tol)


@pytest.mark.parametrize("M,N,K", [
    (1, 8, 16), (1, 128, 128), (2, 136, 144), (16, 256, 384), (17, 128, 4096), (33, 520, 1040), (64, 1000, 2064), (65, 256, 256),
    (127, 384, 512), (128, 136, 128), (129, 256, 640), (200, 2048, 1008), (255, 384, 128), (256, 1000, 528), (300, 520, 272),
    (513, 4104, 400), (1000, 776, 1040), (1024, 2560, 256), (0, 128, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_fp8(M, N, K, dtype):
    A, sa, B, sb = fp8_operands(gen(M + N + K), M, N, K)
    C = nan_like((M, N), dtype)
    up.gemm_fp8_nt(A, sa, B, sb, C)
    if M:
        check_gemm(C, A, sa, B, sb)


@pytest.mark.parametrize("M", [5, 100, 700])
def test_gemm_fp8_reads_slices_and_writes_into_a_slice(M):
    g = gen(M)
    N, K = 264, 272
    A0, sa0, B, sb = fp8_operands(g, M + 9, N, K + 32)
    A, sa = A0[4: 4 + M, 16: 16 + K], sa0[: -(-K // 128), 4: 4 + M]
    B, sb = B[:, :K], sb[:, : -(-K // 128)].contiguous()
    big = nan_like((M + 2, N + 16), torch.bfloat16)
    up.gemm_fp8_nt(A, sa, B, sb, big[1: M + 1, 8: 8 + N])
    check_gemm(big[1: M + 1, 8: 8 + N], A, sa, B, sb)
    outside = torch.ones_like(big, dtype=torch.bool)
    outside[1: M + 1, 8: 8 + N] = False
    assert bool(big[outside].isnan().all())              # nothing else was written


@pytest.mark.parametrize("M", [3, 80, 400])
def test_gemm_fp8_keeps_nan_and_infinity_in_their_rows_and_columns(M):
    g = gen(M)
    A, sa, B, sb = fp8_operands(g, M, 296, 160)
    A.view(torch.uint8)[1, 150] = 0x7f                   # a NaN in the last, short block of K
    sa[0, 2] = float("inf")
    C = nan_like((M, 304), torch.float32)[:, :296]
    up.gemm_fp8_nt(A, sa, B, sb, C)
    assert bool(C[1].isnan().all()) and not bool(C[2].isfinite().any())
    keep = [i for i in range(M) if i not in (1, 2)]
    assert bool(C[keep].isfinite().all())


# ------------------------------------------------------------------------------------------------
# rotary positions
# ------------------------------------------------------------------------------------------------

def rope_ref(x, pos, inv_freq, axis, adjacent, inverse):
    """x [heads, tokens, dh] in 64 bits, and the magnitude of each output's two terms."""
    n = len(inv_freq)
    angle = pos.double()[torch.tensor(axis, device="cuda")].t() * torch.tensor(inv_freq, dtype=torch.float64, device="cuda")
    c, s = angle.cos(), angle.sin() * (-1 if inverse else 1)
    x = x.double()
    y, mag = x.clone(), x.abs()
    i0 = torch.arange(n, device="cuda") * (2 if adjacent else 1)
    i1 = i0 + (1 if adjacent else n)
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    mag[..., i0] = mag[..., i1] = a.abs() + b.abs()
    return y, mag


def check_rope(got, x, pos, inv_freq, axis, adjacent, inverse):
    y, mag = rope_ref(x, pos, inv_freq, axis, adjacent, inverse)
    # the angle is off by at most |pos| 2^-52 turns (frequency) + 2^-25 half turns (its 24-bit argument), with the
    # reference's own 2^-53 |pos inv_freq|: below 2^-20 for |pos| < 2^31; sine, cosine and the products: 2^-21
    within(got, y, y.abs() * BF + mag * 2.0 ** -19 + BF_TINY)


@pytest.mark.parametrize("dh,rot,axes,adjacent,inverse", [
    (128, 128, 1, False, False), (128, 128, 3, False, True), (128, 64, 3, True, False), (64, 64, 2, True, True), (64, 32, 1, False, False),
    (80, 80, 2, False, False), (80, 16, 1, True, False), (16, 16, 4, False, False), (256, 256, 3, True, True), (256, 240, 2, False, False)])
@pytest.mark.parametrize("hq,hkv,tokens", [(1, 0, 1), (8, 2, 1), (3, 1, 77), (32, 8, 300)])
def test_rope(dh, rot, axes, adjacent, inverse, hq, hkv, tokens):
    g = gen(dh + rot + hq + tokens)
    n = rot // 2
    inv_freq = [500000.0 ** (-j / n) for j in range(n)]
    axis = [(j * 7 + j // 3) % axes for j in range(n)]
    axis[0] = axes - 1
    desc = up.make_rope_desc(dh, inv_freq, axis, adjacent=adjacent)
    pos = torch.randint(-2 ** 31, 2 ** 31, (axes, tokens), generator=g, device="cuda").int()
    pos[:, 0] = torch.tensor([0, -(2 ** 31), 2 ** 31 - 1, 5], device="cuda")[:axes].int()
    qkv = randn(g, tokens, hq + 2 * hkv, dh).bfloat16()
    heads = qkv.transpose(0, 1)                          # token-major, as the projection writes it
    q, k = heads[:hq], heads[hq: hq + hkv] if hkv else None
    qo = nan_like((hq, tokens, dh), torch.bfloat16)
    ko = nan_like((hkv, tokens, dh), torch.bfloat16) if hkv else None
    up.rope(desc, q, k, pos, qo, ko, inverse=inverse)
    check_rope(qo, q, pos, inv_freq, axis, adjacent, inverse)
    if hkv:
        check_rope(ko, k, pos, inv_freq, axis, adjacent, inverse)
    # in place in the token-major buffer: the same values, V untouched
    v = qkv[:, hq + hkv:].clone()
    up.rope(desc, q, k, pos, q, k, inverse=inverse)
    assert torch.equal(q, qo) and (not hkv or torch.equal(k, ko)) and torch.equal(qkv[:, hq + hkv:], v)
    assert desc.inverse == 0                             # the caller's description is left as it was


def test_rope_and_its_inverse_cancel():
    g = gen(9)
    inv_freq = [10000.0 ** (-j / 64) for j in range(64)]
    desc = up.make_rope_desc(128, inv_freq)
    pos = (torch.arange(500, device="cuda")[None] + 4_999_000).int()
    x = randn(g, 4, 500, 128).bfloat16()
    y, z = torch.empty_like(x), torch.empty_like(x)
    up.rope(desc, x, None, pos, y, None)
    up.rope(desc, y, None, pos, z, None, inverse=True)
    n = torch.hypot(x[..., :64].double(), x[..., 64:].double()).repeat(1, 1, 2)
    # each turn rounds both elements of a pair by 2^-8 of at most the pair's length, the first turn's two
    # roundings reach each element of the second with |cos| + |sin| <= sqrt 2
    within(z, x.double(), n * (BF * (1 + 2 ** 0.5) * (1 + BF) + 2.0 ** -18))


def test_rope_takes_shared_rows():
    """One row of keys for all tokens (stride 0 of the input), and strides longer than a row."""
    g = gen(21)
    inv_freq = [100.0 ** (-j / 32) for j in range(32)]
    desc = up.make_rope_desc(64, inv_freq)
    pos = torch.arange(90, device="cuda").int()[None]
    x = randn(g, 3, 1, 64).bfloat16().expand(3, 90, 64)
    out = nan_like((90, 3, 72), torch.bfloat16)
    up.rope(desc, x, None, pos, out.transpose(0, 1)[..., :64], None)
    check_rope(out.transpose(0, 1)[..., :64], x, pos, inv_freq, [0] * 32, False, False)
    assert bool(out[..., 64:].isnan().all())


# ------------------------------------------------------------------------------------------------
# gradient clipping
# ------------------------------------------------------------------------------------------------

def norm_of(grads):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in grads))


@pytest.mark.parametrize("sizes,dtypes", [
    ([1], "f"), ([0, 3, 0], "b"), ([8191, 8192, 8193, 7], "fb"), ([100_003, 64, 1, 5000], "bf"), ([300_000] * 3, "f"),
    ([17] * 30, "fb"), ([1000 + i for i in range(1100)], "fb"), ([3_000_001], "b"), ([], "f")])
@pytest.mark.parametrize("into", [None, "f", "b"])
def test_grad_clip(sizes, dtypes, into):
    kind = {"f": torch.float32, "b": torch.bfloat16}
    g = gen(len(sizes) + sum(sizes))
    grads = [(0.01 * randn(g, n)).to(kind[dtypes[i % len(dtypes)]]) for i, n in enumerate(sizes)]
    before = [t.clone() for t in grads]
    outs = None if into is None else [nan_like((n,), kind[into]) for n in sizes]
    total = norm_of(grads)
    clip = up.GradClip(grads, outs)
    for max_norm in ((1e30, 0.5 * total) if total else (1.0,)):
        got = clip(max_norm)
        coef = min(1.0, max_norm / (total + 1e-6))
        # 32 squares added in fp32: the sum within 33 u, the norm within 17 u and its own rounding
        assert abs(float(got) - total) <= total * 20 * U
        for src, dst in zip(before, grads if outs is None else outs):
            if not src.numel():
                continue
            want = src.double() * coef
            half = {torch.float32: U, torch.bfloat16: BF}[dst.dtype]
            within(dst, want, want.abs() * (half + 24 * U) + (BF_TINY if dst.dtype == torch.bfloat16 else 2.0 ** -150))
        if outs is not None:
            assert all(torch.equal(a, b) for a, b in zip(before, grads))
    assert math.isclose(float(clip(math.inf)), norm_of(grads), rel_tol=20 * U)


@pytest.mark.parametrize("size", [1e-30, 1e-38, 1e-44, 1e25, 3e38])
def test_grad_clip_norm_of_tiny_and_huge_gradients(size):
    """Squares below and above fp32's range; a tensor of ordinary values beside them changes nothing."""
    g = gen(1)
    t = randn(g, 20_000).clamp(-1, 1) * torch.tensor(size, device="cuda")
    total = norm_of([t])
    clip = up.GradClip([t])
    if total < 3.4e38:
        assert abs(float(clip(math.inf)) - total) <= total * 20 * U + 2.0 ** -149
    else:
        assert math.isinf(float(clip(math.inf)))          # the norm itself is past fp32; the factor is still right
        before = t.clone()
        clip(1e38)
        within(t, before.double() * (1e38 / total), before.double().abs() * (1e38 / total) * 24 * U)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_grad_clip_leaves_gradients_alone_when_the_norm_is_not_finite(bad):
    g = gen(2)
    grads = [randn(g, 5000), randn(g, 9000).bfloat16()]
    grads[1][8500] = bad
    before = [t.clone() for t in grads]
    norm = float(up.GradClip(grads)(1.0))
    assert math.isnan(norm) if bad != bad else math.isinf(norm)
    assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(grads, before))
    outs = [torch.zeros_like(t) for t in grads]
    up.GradClip(grads, outs)(1.0)
    assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(outs, before))


def test_grad_clip_refuses_a_tensor_listed_twice():
    t = torch.zeros(100, device="cuda")
    with pytest.raises(up.UpipeError):
        up.GradClip([t, t])(1.0)
    with pytest.raises(up.UpipeError):
        up.GradClip([t, t[48:]])(1.0)
    with pytest.raises(up.UpipeError):
        up.GradClip([t[1:]])(1.0)                         # not 16-byte aligned
    with pytest.raises(ValueError):
        up.GradClip([t.view(10, 10).t()])


# ------------------------------------------------------------------------------------------------
# refusals of the binding, streams, graphs, offsets past 32 bits
# ------------------------------------------------------------------------------------------------

def test_binding_refuses_wrong_tensors():
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(256, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    q, s = nan_like((4, 256), torch.float8_e4m3fn), nan_like((2, 4), torch.float32)
    bad = [lambda: up.rms_norm_fwd(x.float(), w, y), lambda: up.rms_norm_fwd(x, w[:128], y), lambda: up.rms_norm_fwd(x.cpu(), w, y),
           lambda: up.rms_norm_fwd(torch.zeros(256, 4, dtype=torch.bfloat16, device="cuda").t(), w, y), lambda: up.rms_norm_fwd(x[0], w, y),
           lambda: up.rms_norm_fwd_fp8(x, w, q, s.t()), lambda: up.rms_norm_fwd_fp8(x, w, q.view(torch.uint8), s),
           lambda: up.fp8_quantize(x, q, s.t()), lambda: up.fp8_quantize(x, q, s, block_rows=64), lambda: up.gemm_fp8_nt(q, s, q, s, y),
           lambda: up.gemm_fp8_nt(q, s, q, s[:1], y.half()),
           lambda: up.gemm_fp8_nt(q[:1].expand(4, 256), s, q, s[:1, :2].contiguous(), y[:, :4]),   # rows that overlap
           lambda: up.gemm_fp8_nt(q, s[:, :1].expand(2, 4), q, s[:1, :2].contiguous(), y[:, :4]),
           lambda: up.gemm_fp8_nt(q, s, q, s[:1, :2].contiguous(), y[:1, :4].expand(4, 4)), lambda: up.rope(up.make_rope_desc(64, [0.1] * 32), y[None], None, s, y[None], None)]
    n = up.launch_count()
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(up.UpipeError):
        up.rms_norm_fwd(x, w, y, residual=x)              # a residual without h
    d, pos, z = up.make_rope_desc(64, [0.1] * 32), torch.zeros(1, 4, dtype=torch.int32, device="cuda"), y.view(4, 4, 64)
    for q_out, k_out in ((y.view(4, 4, 64), y.view(4, 4, 64)), (z[:1].expand(4, 4, 64), x.view(4, 4, 64))):
        with pytest.raises(up.UpipeError):
            up.rope(d, x.view(4, 4, 64), x.view(4, 4, 64), pos, q_out, k_out)
    with pytest.raises(up.UpipeError):
        up.rms_norm_bwd(x, x, w, s.view(-1)[:4].contiguous(), y, s.new_empty(256), torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert up.launch_count() == n


def block_state(seed, rows=300, d=512):
    g = gen(seed)
    hq, hkv, dh = 4, 2, 64
    s = dict(x=randn(g, rows, d).bfloat16(), r=randn(g, rows, d).bfloat16(), w=(1 + 0.1 * randn(g, d)).bfloat16(),
             W=(0.05 * randn(g, (hq + 2 * hkv) * dh, d)).bfloat16(), pos=torch.arange(rows, device="cuda").int()[None] + 1000,
             dq=randn(g, hq, rows, dh).bfloat16(), dk=randn(g, hkv, rows, dh).bfloat16())
    n = (hq + 2 * hkv) * dh
    f8 = torch.float8_e4m3fn
    s.update(h=nan_like((rows, d), torch.bfloat16), q8=nan_like((rows, d), f8), sx=nan_like((-(-d // 128), rows), torch.float32),
             rstd=nan_like((rows,), torch.float32), W8=nan_like((n, d), f8), sw=nan_like((-(-n // 128), -(-d // 128)), torch.float32),
             qkv=nan_like((rows, hq + 2 * hkv, dh), torch.bfloat16), q=nan_like((hq, rows, dh), torch.bfloat16),
             k=nan_like((hkv, rows, dh), torch.bfloat16), dqkv=torch.zeros(rows, hq + 2 * hkv, dh, dtype=torch.bfloat16, device="cuda"),
             dx=nan_like((rows, d), torch.bfloat16), dw=nan_like((d,), torch.float32),
             ws=torch.empty(up.rms_norm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda"),
             desc=up.make_rope_desc(dh, [10000.0 ** (-j / 32) for j in range(32)]), hq=hq, hkv=hkv)
    s["clip"] = up.GradClip([s["dw"]], [nan_like((d,), torch.float32)])
    return s


def block_pass(s, stream=None):
    """Norm to 8 bits, weights quantised, product, rotary and back, norm backward, clip."""
    hq, hkv = s["hq"], s["hkv"]
    rows = s["x"].shape[0]
    up.rms_norm_fwd_fp8(s["x"], s["w"], s["q8"], s["sx"], s["rstd"], residual=s["r"], h=s["h"], stream=stream)
    up.fp8_quantize(s["W"], s["W8"], s["sw"], block_rows=128, stream=stream)
    up.gemm_fp8_nt(s["q8"], s["sx"], s["W8"], s["sw"], s["qkv"].view(rows, -1), stream=stream)
    t = s["qkv"].transpose(0, 1)
    up.rope(s["desc"], t[:hq], t[hq: hq + hkv], s["pos"], s["q"], s["k"], stream=stream)
    t = s["dqkv"].transpose(0, 1)
    up.rope(s["desc"], s["dq"], s["dk"], s["pos"], t[:hq], t[hq: hq + hkv], inverse=True, stream=stream)
    up.rms_norm_bwd(s["x"], s["h"], s["w"], s["rstd"], s["dx"], s["dw"], s["ws"], dres=s["r"], stream=stream)
    s["clip"](0.5, stream=stream)
    return [s[k] for k in ("h", "q8", "sx", "rstd", "W8", "sw", "qkv", "q", "k", "dqkv", "dx", "dw")] + s["clip"].outs + [s["clip"].norm]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x,
                           y.view(torch.uint8) if y.dtype == torch.float8_e4m3fn else y) for x, y in zip(a, b))


def test_operators_on_another_stream_and_in_graphs():
    """Every operator on a side stream, then captured; the graph replayed on new inputs, twice, and two graphs that
    share their workspaces replayed one after the other on one stream: bit for bit what eager calls give."""
    a, b = block_state(1), block_state(2)
    b["ws"], b["clip"].ws = a["ws"], a["clip"].ws
    want_a = [t.clone() for t in block_pass(a)]
    want_b = [t.clone() for t in block_pass(b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = block_pass(a, stream=side)
    side.synchronize()
    assert same(out, want_a)
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = block_pass(s)
        graphs.append((g, outs))
    for t in graphs[0][1]:
        t.view(torch.uint8).zero_()
    for _ in range(2):
        for g, _o in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert same(graphs[0][1], want_a) and same(graphs[1][1], want_b)
    a["x"].copy_(b["x"])                                  # new inputs in the captured buffers
    for k in ("r", "w", "W", "dq", "dk", "pos"):
        a[k].copy_(b[k])
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert same(graphs[0][1], want_b)


def test_two_streams_at_once():
    """Runs of every operator on two streams that overlap, products of every kernel among them, beside the attention
    core: each result is the one of a run alone."""
    states = [block_state(s, rows=r) for s, r in ((5, 9), (6, 700), (7, 40), (8, 257))]
    core = up.make_desc(1024, 256, 4, 2, 128)
    g = gen(9)
    q, k, v = (randn(g, h, 1024, 128).bfloat16() for h in (4, 2, 2))
    table = torch.empty(up.tile_table_bytes(core), dtype=torch.uint8, device="cuda")
    up.build_tile_table(core, None, table)
    o, lse = torch.empty_like(q), torch.empty(4, 1024, device="cuda")
    up.core_fwd(core, q, k, v, None, table, o, lse)
    want_o = o.clone()
    want = [[t.clone() for t in block_pass(s)] for s in states]
    for t in [o] + [x for s in states for x in (s["qkv"], s["dx"], s["q8"], s["q"])]:
        t.view(torch.uint8).zero_()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(states):
            block_pass(s, stream=streams[i % 2])
        up.core_fwd(core, q, k, v, None, table, o, lse, stream=streams[2])
    torch.cuda.synchronize()
    assert torch.equal(o, want_o) and up.device_status(table) == 0
    for s, w in zip(states, want):
        assert same([s[k] for k in ("h", "q8", "sx", "rstd", "W8", "sw", "qkv", "q", "k", "dqkv", "dx", "dw")] + s["clip"].outs
                    + [s["clip"].norm], w)


def test_norm_and_rope_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows are right and the first were not overwritten."""
    rows, d = 530_000, 4096                               # 2.17e9 elements, 4.3 GB each
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    x[:3], x[-3:] = randn(gen(1), 3, d).bfloat16(), randn(gen(2), 3, d).bfloat16()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    up.rms_norm_fwd(x, w, y)
    small = torch.empty(6, d, dtype=torch.bfloat16, device="cuda")
    up.rms_norm_fwd(torch.cat([x[:3], x[-3:]]), w, small)
    assert torch.equal(torch.cat([y[:3], y[-3:]]), small) and not bool(y[1000].any())
    tokens = rows * d // (32 * 128)
    heads = x.view(tokens, 32, 128).transpose(0, 1)
    pos = torch.arange(tokens, device="cuda").int()[None]
    desc = up.make_rope_desc(128, [10000.0 ** (-j / 64) for j in range(64)])
    out = y.view(32, tokens, 128)
    up.rope(desc, heads, None, pos, out, None)
    some = [0, 1, 2, tokens - 3, tokens - 2, tokens - 1]
    ref = torch.empty(32, 6, 128, dtype=torch.bfloat16, device="cuda")
    up.rope(desc, heads[:, some].contiguous(), None, pos[:, some].contiguous(), ref, None)
    assert torch.equal(out[:, some], ref)


def test_gemm_offsets_past_32_bits():
    M, N, K = 150_000, 14_400, 128                        # C of 2.16e9 elements
    g = gen(6)
    A, sa, B, sb = fp8_operands(g, M, N, K)
    C = nan_like((M, N), torch.bfloat16)
    up.gemm_fp8_nt(A, sa, B, sb, C)
    rows = torch.tensor([0, 1, 127, M // 2, M - 130, M - 1], device="cuda")
    check_gemm(C[rows], A.view(torch.uint8)[rows].view(A.dtype), sa[:, rows], B, sb)
    for part in C.split(10_000):
        assert bool(part.isfinite().all())


# ------------------------------------------------------------------------------------------------
# a run of them, as a block uses them
# ------------------------------------------------------------------------------------------------

def test_attention_block_in_8_bits():
    """residual + norm -> e4m3 -> QKV product -> rotary -> attention core, forward and backward -> gradients turned
    back: each stage against the 64-bit result of what the stage before it wrote."""
    g = gen(77)
    rows, d, hq, hkv, dh = 700, 512, 4, 2, 128
    x, r = randn(g, rows, d).bfloat16(), randn(g, rows, d).bfloat16()
    w, W = (1 + 0.1 * randn(g, d)).bfloat16(), (0.04 * randn(g, (hq + 2 * hkv) * dh, d)).bfloat16()
    h, q8, sx, rstd = torch.empty_like(x), nan_like((rows, d), torch.float8_e4m3fn), torch.empty(d // 128, rows, device="cuda"), torch.empty(rows, device="cuda")
    up.rms_norm_fwd_fp8(x, w, q8, sx, rstd, residual=r, h=h)
    check_q(q8, sx.t(), norm_ref(x, r, w, 1e-5)[2], 1, ROW)
    W8, sw = nan_like(W.shape, torch.float8_e4m3fn), torch.empty(W.shape[0] // 128, d // 128, device="cuda")
    up.fp8_quantize(W, W8, sw, block_rows=128)
    check_q(W8, sw, W.double(), 128, 0.0)
    qkv = nan_like((rows, hq + 2 * hkv, dh), torch.bfloat16)
    up.gemm_fp8_nt(q8, sx, W8, sw, qkv.view(rows, -1))
    check_gemm(qkv.view(rows, -1), q8, sx, W8, sw)
    inv_freq, axis = [10000.0 ** (-j / 64) for j in range(64)], [j // 22 for j in range(64)]
    desc = up.make_rope_desc(dh, inv_freq, axis)
    t = torch.arange(rows, device="cuda")
    pos = torch.stack([t // 96, t // 12 % 8, t % 12]).int()
    heads = qkv.transpose(0, 1)
    q, k = nan_like((hq, rows, dh), torch.bfloat16), nan_like((hkv, rows, dh), torch.bfloat16)
    up.rope(desc, heads[:hq], heads[hq: hq + hkv], pos, q, k)
    check_rope(q, heads[:hq], pos, inv_freq, axis, False, False)
    check_rope(k, heads[hq: hq + hkv], pos, inv_freq, axis, False, False)
    v = heads[hq + hkv:].contiguous()
    core = up.make_desc(rows, d, hq, hkv, dh)
    table = torch.empty(up.tile_table_bytes(core), dtype=torch.uint8, device="cuda")
    up.build_tile_table(core, None, table)
    o, lse = torch.empty_like(q), torch.empty(hq, rows, device="cuda")
    up.core_fwd(core, q, k, v, None, table, o, lse)
    do = randn(g, hq, rows, dh).bfloat16()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    up.core_bwd(core, q, k, v, do, lse, None, table, dq, dk, dv)
    assert up.device_status(table) == 0
    qd, kd, vd = q.double(), k.double().repeat_interleave(2, 0), v.double().repeat_interleave(2, 0)
    p = (qd @ kd.transpose(1, 2) * dh ** -0.5).masked_fill(torch.ones(rows, rows, device="cuda").triu(1).bool(), -math.inf).softmax(-1)
    assert float((o.double() - p @ vd).norm() / (p @ vd).norm()) <= 5e-3   # the attention core's own bars
    ds = p * (do.double() @ vd.transpose(1, 2) - (do.double() * (p @ vd)).sum(-1, keepdim=True)) * dh ** -0.5
    assert float((dq.double() - ds @ kd).norm() / (ds @ kd).norm()) <= 1e-2
    dqkv = nan_like((rows, hq + 2 * hkv, dh), torch.bfloat16)
    t = dqkv.transpose(0, 1)
    up.rope(desc, dq, dk, pos, t[:hq], t[hq: hq + hkv], inverse=True)
    t[hq + hkv:].copy_(dv)
    check_rope(t[:hq], dq, pos, inv_freq, axis, False, True)
    check_rope(t[hq: hq + hkv], dk, pos, inv_freq, axis, False, True)


def test_training_step_of_a_block():
    """residual + norm -> attention layer -> its backward -> norm backward -> clipped gradients."""
    g = gen(78)
    rows, d, hq, hkv, dh = 384, 256, 4, 2, 64
    x, r, dres = (randn(g, rows, d).bfloat16() for _ in range(3))
    w = (1 + 0.1 * randn(g, d)).bfloat16()
    Wqkv, Wo = (0.05 * randn(g, (hq + 2 * hkv) * dh, d)).bfloat16(), (0.05 * randn(g, d, hq * dh)).bfloat16()
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    up.rms_norm_fwd(x, w, y, rstd, residual=r, h=h)
    layer = up.Layer(up.make_desc(rows, d, hq, hkv, dh, 2))
    Y, lse = layer.forward(y, Wqkv, Wo)
    dX, dWqkv, dWo = layer.backward(y, Wqkv, Wo, None, dres, lse)
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(up.rms_norm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    up.rms_norm_bwd(dX, h, w, rstd, dx, dw, ws, dres=dres)   # dres: the residual stream's own gradient
    grads = [dWqkv, dWo, dw]
    total = norm_of(grads)
    before = [t.clone() for t in grads]
    norm = up.GradClip(grads)(0.1 * total)
    assert abs(float(norm) - total) <= total * 20 * U
    for a, b in zip(grads, before):
        want = b.double() * (0.1 * total / (total + 1e-6))
        within(a, want, want.abs() * 32 * U)
    # gradients of sum(dres * (h + attention(norm(h)))) in 64 bits
    hd = h.double().requires_grad_()
    wd, Wq, Wp = (t.double().requires_grad_() for t in (w, Wqkv, Wo))
    yd = hd * (hd.square().mean(1, keepdim=True) + 1e-5).rsqrt() * wd
    qkv = (yd @ Wq.t()).view(rows, hq + 2 * hkv, dh).transpose(0, 1)
    q, k, v = qkv[:hq], qkv[hq: hq + hkv].repeat_interleave(2, 0), qkv[hq + hkv:].repeat_interleave(2, 0)
    p = (q @ k.transpose(1, 2) * dh ** -0.5).masked_fill(torch.ones(rows, rows, device="cuda").triu(1).bool(), -math.inf).softmax(-1)
    out = (p @ v).transpose(0, 1).reshape(rows, -1) @ Wp.t() + hd
    (out * dres.double()).sum().backward()
    for got, want in ((dx, hd.grad), (before[2], wd.grad), (before[0], Wq.grad), (before[1], Wp.grad)):
        assert float((got.double() - want).norm() / want.norm()) <= 1e-2   # the layer's gradient bar
