"""Operators around the two blocks where their kernels go round: more tiles, rows or blocks than the device works on at
once, and rings of stages, accumulators and scales that wrap.  Every instantiation of the product is reached; which
shape reaches which is restated below from the product's rule, so that a change of the rule shows here.  Tolerances are
those of test_gpu_block_ops.py, which counts the roundings.
"""
import pytest
import torch

import long_context_attention_upipe_gb300 as up
from test_gpu_block_ops import BF, BF_TINY, ROW, check_gemm, check_q, fp8_operands, gen, nan_like, norm_ref, randn, within
from test_gpu_block_rounding import oracle, same_codes, same_scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


def cdiv(a, b):
    return -(-a // b)


def splits(ctas, nkb, tn, sms):
    return max(1, min(8, (sms * 7 // 8 if tn == 128 else sms) // ctas, nkb // 2))


def kernel_of(M, N, K, sms):
    """("few", tokens per CTA, shares of K) or ("pair", 32 columns per tile, rounds of tiles)."""
    nkb = cdiv(K, 128)
    for tn in (16, 32, 64):
        if M <= tn:
            return "few", tn, splits(cdiv(N, 128), nkb, tn, sms)
    clusters, tm = sms // 2, cdiv(M, 256)
    cost, best = min((cdiv(tm * cdiv(N, 32 * c), clusters) * (nkb * (130 + 90 * c) + 200 * c), -c) for c in range(4, 9))
    ctas = cdiv(N, 128) * cdiv(M, 128)
    s = splits(ctas, nkb, 128, sms)
    if cdiv(M, 128) <= 65535 and cdiv(ctas * s, sms) * (12500 + cdiv(nkb, s) * 1000) < 8000 + cost:
        return "few", 128, s
    return "pair", -best, tm * cdiv(N, -32 * best) / clusters


SHAPES = [  # kernel, width, (M, N, K)
    ("pair", 4, (1281, 3088, 1360)), ("pair", 4, (3438, 1952, 2384)), ("pair", 5, (515, 6432, 1360)), ("pair", 5, (1774, 3296, 2736)),
    ("pair", 6, (514, 8152, 1360)), ("pair", 6, (3318, 2984, 1616)), ("pair", 7, (773, 7336, 1360)), ("pair", 7, (3723, 3160, 1360)),
    ("pair", 8, (775, 8560, 1360)), ("pair", 8, (875, 8592, 2128)), ("few", 16, (16, 256, 4096)), ("few", 16, (9, 1000, 2064)),
    ("few", 16, (16, 19464, 2064)), ("few", 32, (32, 256, 4096)), ("few", 32, (29, 19464, 2064)), ("few", 64, (64, 256, 4112)),
    ("few", 64, (40, 20000, 2064)), ("few", 128, (128, 4096, 4096)), ("few", 128, (100, 1024, 4096)), ("few", 128, (65, 256, 4112))]


@pytest.mark.parametrize("kind,width,shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_of_many_turns(kind, width, shape, dtype):
    M, N, K = shape
    got = kernel_of(M, N, K, torch.cuda.get_device_properties(0).multi_processor_count)
    assert got[:2] == (kind, width) and (kind == "few" or got[2] > 1)
    A, sa, B, sb = fp8_operands(gen(M + N + K), M, N, K)
    C = nan_like((M, N), dtype)
    up.gemm_fp8_nt(A, sa, B, sb, C)
    check_gemm(C, A, sa, B, sb)
    D = nan_like((M, N), dtype)
    up.gemm_fp8_nt(A, sa, B, sb, D)
    assert torch.equal(C, D)


def test_product_of_few_rows_reaches_every_number_of_shares():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seen = set()
    for N in (128, 2432, 3200, 3840, 4864, 6400, 9728, 12800):
        M, K = 16, 2064
        seen.add(kernel_of(M, N, K, sms)[2])
        A, sa, B, sb = fp8_operands(gen(N), M, N, K)
        C = nan_like((M, N), torch.bfloat16)
        up.gemm_fp8_nt(A, sa, B, sb, C)
        check_gemm(C, A, sa, B, sb)
    assert seen >= {1, 2, 3, 4, 5, 6, 8}


def test_product_of_one_block_of_k_takes_no_longer_than_of_two():
    """By the kernel of few rows it took four times as long."""
    def us(K):
        A, sa, B, sb = fp8_operands(gen(K), 8192, 14336, K)
        C = nan_like((8192, 14336), torch.bfloat16)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for i in range(13):
            if i == 3:
                start.record()
            up.gemm_fp8_nt(A, sa, B, sb, C)
        end.record()
        torch.cuda.synchronize()
        check_gemm(C[-300:], A.view(torch.uint8)[-300:].view(A.dtype), sa[:, -300:], B, sb)
        return start.elapsed_time(end)
    assert us(128) < 2 * us(256)


def test_tiled_product_offsets_past_32_bits():
    M, N, K = 150_000, 14_400, 400                        # C of 2.16e9 elements, by the kernel of many rows
    assert kernel_of(M, N, K, torch.cuda.get_device_properties(0).multi_processor_count)[0] == "pair"
    A, sa, B, sb = fp8_operands(gen(7), M, N, K)
    C = nan_like((M, N), torch.bfloat16)
    up.gemm_fp8_nt(A, sa, B, sb, C)
    rows = torch.tensor([0, 1, 127, 128, 255, M // 2, 149_130, 149_131, M - 130, M - 1], device="cuda")
    check_gemm(C[rows], A.view(torch.uint8)[rows].view(A.dtype), sa[:, rows], B, sb)
    for part in C.split(10_000):
        assert bool(part.isfinite().all())


# more rows than are in flight, for every instantiation of the forward kernel
@pytest.mark.parametrize("rows,d", [(30_001, 128), (12_003, 256), (4_001, 1040), (2_003, 4096), (1_001, 5120), (701, 8192), (1_003, 8208),
                                    (703, 16384), (401, 16400), (333, 32768)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_forward_of_many_turns(rows, d, residual):
    g = gen(rows + d)
    x = (2 * randn(g, rows, d) * torch.exp(randn(g, rows, 1))).bfloat16()     # rows of different size: none passes for another
    r = randn(g, rows, d).bfloat16() if residual else None
    w = (1 + 0.2 * randn(g, d)).bfloat16()
    h = nan_like((rows, d), torch.bfloat16) if residual else None
    q, s = nan_like((rows, d), torch.float8_e4m3fn), nan_like((cdiv(d, 128), rows), torch.float32)
    y, y2, rstd = nan_like((rows, d), torch.bfloat16), nan_like((rows, d), torch.bfloat16), nan_like((rows,), torch.float32)
    up.rms_norm_fwd_fp8(x, w, q, s, rstd, residual=r, h=h, y=y)
    hd, rd, yd = norm_ref(x, r, w, 1e-5)
    assert h is None or torch.equal(h.double(), hd)
    within(rstd, rd, rd * ROW)
    within(y, yd, yd.abs() * (BF + ROW) + BF_TINY)
    check_q(q, s.t(), yd, 1, ROW)
    up.rms_norm_fwd(x, w, y2, residual=r, h=h)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("rows,cols", [(3_001, 4096), (40_001, 272), (90_001, 128)])
@pytest.mark.parametrize("block", [1, 128])
def test_quantiser_of_many_turns(rows, cols, block):
    g = gen(rows)
    x = (randn(g, rows, cols) * torch.exp(randn(g, rows, 1))).bfloat16()
    q = nan_like((rows, cols), torch.float8_e4m3fn)
    s = nan_like((cdiv(cols, 128), rows) if block == 1 else (cdiv(rows, 128), cdiv(cols, 128)), torch.float32)
    up.fp8_quantize(x, q, s, block_rows=block)
    want_q, want_s = oracle(x.float().cpu(), block)
    same_scales(s.t() if block == 1 else s, want_s)
    same_codes(q, want_q)
