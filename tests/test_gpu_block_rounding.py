"""The e4m3 outputs of the norm and of the block quantiser, bit for bit.

A block's scale is s = max|y| * fp32(1 / 448) (1 below 2^-100), its codes are e4m3(fp32(y / s)): one fp32 product,
one fp32 division and one rounding to nearest even, each exactly rounded, so the oracle below repeats them in fp32 on
the CPU and no tolerance is needed.  bf16 values over a shared scale meet e4m3's ties often (y = 17 m over a largest
value of 7 m is one), and an inexact quotient sends them to either side.
"""
import pytest
import torch

import long_context_attention_upipe_gb300 as up

pytestmark = pytest.mark.gpu

C448 = torch.tensor(1.0) / torch.tensor(448.0)   # rounded to fp32 once
TINY = 2.0 ** -100


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


def oracle(y, br):
    """Codes (as bytes) and scales [row blocks, column blocks] of fp32 y on the CPU."""
    rows, cols = y.shape
    p = torch.nn.functional.pad(y, (0, -cols % 128, 0, -rows % br))
    b = p.view(p.shape[0] // br, br, p.shape[1] // 128, 128)
    amax = b.abs().amax((1, 3))
    s = torch.where(amax < TINY, torch.ones_like(amax), amax * C448)
    v = (b / s[:, None, :, None]).reshape(p.shape)[:rows, :cols]
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def same_codes(q, want):
    """Equal bytes; a NaN may carry either sign."""
    q = q.cpu().view(torch.uint8)
    nan = (want & 0x7f) == 0x7f
    bad = torch.where(nan, (q & 0x7f) != 0x7f, q != want)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} codes differ, the first at {int(bad.flatten().int().argmax())}"


def same_scales(s, want):
    assert torch.equal(s.cpu().nan_to_num(-1.0), want.nan_to_num(-1.0))


def values(kind, rows, cols):
    g = torch.Generator().manual_seed(rows + cols + len(kind))
    x = torch.randn(rows, cols, generator=g)
    if kind == "wide":          # columns of very different strength
        x = x * torch.exp(3 * torch.randn(1, cols, generator=g))
    if kind == "ties":          # every block's largest value is 7 m 2^k, the others are odd 5-bit numbers times m
        m = torch.randint(1, 16, (rows, 1), generator=g).float()
        x = (2 * torch.randint(8, 16, (rows, cols), generator=g) + 1).float() * m * torch.randint(0, 2, (rows, cols), generator=g).mul(2).sub(1)
        x[:, ::128] = 7 * m * 8
        if cols > 128:
            x[:, 128::256] *= 2
    if kind == "far":           # scales from 2^-108 to 2^118
        x = x * torch.exp2(torch.linspace(-100, 126, rows).floor())[:, None]
    if kind == "codes":         # every e4m3 boundary and its neighbours in bf16 steps, scale a power of two
        x = torch.arange(rows * cols).view(rows, cols).remainder(65536).to(torch.int32)
        x = (x << 16).view(torch.float32)
        x = torch.where(x.isfinite() & (x.abs() <= 448), x, torch.full_like(x, 448.0))
        x[:, ::128] = 448.0
    return x.bfloat16()


@pytest.mark.parametrize("kind", ["plain", "wide", "ties", "far", "codes"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 144), (129, 272), (1001, 1040), (600, 4096)])
@pytest.mark.parametrize("block", [1, 128])
def test_quantiser_codes(kind, rows, cols, block):
    x = values(kind, rows, cols)
    nb = -(-cols // 128)
    q = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((nb, rows) if block == 1 else (-(-rows // 128), nb), -7.0, device="cuda")
    up.fp8_quantize(x.cuda(), q, s, block_rows=block)
    want_q, want_s = oracle(x.float(), block)
    same_scales(s.t() if block == 1 else s, want_s)
    same_codes(q, want_q)


@pytest.mark.parametrize("block", [1, 128])
def test_quantiser_codes_of_blocks_with_nan_and_infinity(block):
    x = values("wide", 256, 400)
    x[3, 130], x[200, 300], x[77, 399], x[9, 0] = float("nan"), float("-inf"), float("inf"), 3.38e38
    q = torch.full((256, 400), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((4, 256) if block == 1 else (2, 4), -7.0, device="cuda")
    up.fp8_quantize(x.cuda(), q, s, block_rows=block)
    want_q, want_s = oracle(x.float(), block)
    same_scales(s.t() if block == 1 else s, want_s)
    same_codes(q, want_q)


@pytest.mark.parametrize("kind", ["plain", "wide", "ties"])
@pytest.mark.parametrize("rows,d", [(1, 16), (5, 272), (300, 1040), (1000, 4096), (200, 5120), (60, 8208), (20, 16400)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_codes(kind, rows, d, residual):
    """From the h and rstd that the kernel wrote, y = (h * rstd) * w is two fp32 products."""
    x = values(kind, rows, d)
    g = torch.Generator().manual_seed(d)
    w = (torch.ones(d) if kind == "ties" else 1 + 0.3 * torch.randn(d, generator=g)).bfloat16()
    r = values("plain", rows, d).cuda() if residual else None
    h = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda") if residual else None
    q = torch.full((rows, d), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s, rstd = torch.full((-(-d // 128), rows), -7.0, device="cuda"), torch.empty(rows, device="cuda")
    up.rms_norm_fwd_fp8(x.cuda(), w.cuda(), q, s, rstd, residual=r, h=h)
    hf = (x if h is None else h.cpu()).float()
    want_q, want_s = oracle(hf * rstd.cpu()[:, None] * w.float(), 1)
    same_scales(s.t(), want_s)
    same_codes(q, want_q)
