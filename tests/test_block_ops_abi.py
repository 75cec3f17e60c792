"""Operators around the two blocks: what their entry points refuse, checked without a GPU (every check
runs on the host before any launch)."""
import ctypes
import math

import pytest
import torch

import long_context_attention_upipe_gb300 as up

FAKE, ODD = 0x100000, 0x100008  # never dereferenced: the checks fail first


def fake(i):
    """Distinct addresses, 1 TiB apart."""
    return FAKE + (i << 40)


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


@pytest.fixture(autouse=True)
def nothing_launched():
    n = up.launch_count()
    yield
    assert up.launch_count() == n


def norm_fwd(**kw):
    a = dict(rows=4, d=256, eps=1e-5, x=fake(0), res=None, w=fake(1), h=None, y=fake(2), q=None, scales=None, rstd=None)
    a.update(kw)
    return up.lib().upipe_attn_rms_norm_fwd(a["rows"], a["d"], a["eps"], a["x"], a["res"], a["w"], a["h"], a["y"], a["q"],
                                            a["scales"], a["rstd"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(d=0), 1), (dict(d=100), 2), (dict(d=32776), 2),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(x=None), 1), (dict(w=None), 1),
    (dict(y=None), 1), (dict(q=fake(3)), 1), (dict(scales=fake(3)), 1), (dict(res=fake(4)), 1), (dict(h=fake(4)), 1),
    (dict(d=264, q=fake(3), scales=fake(4)), 2), (dict(x=ODD), 3), (dict(rstd=ODD), 3),
    (dict(q=ODD, scales=fake(4)), 3),
    (dict(y=fake(0) + 512), 1),                       # y starts inside x
    (dict(res=fake(4), h=fake(2)), 1),                # h is y
    (dict(res=fake(4), h=fake(4) - 512), 1),          # h ends inside the residual
    (dict(q=fake(0), scales=fake(5)), 1),             # q over x
    (dict(y=fake(1)), 1), (dict(y=fake(1) - 1024), 1),  # y is w, y ends inside w
    (dict(rstd=fake(0)), 1), (dict(rstd=fake(2) + 16), 1), (dict(rstd=fake(1)), 1),
    (dict(q=fake(3), scales=fake(2)), 1), (dict(q=fake(3), scales=fake(0) + 16), 1), (dict(q=fake(1), scales=fake(4)), 1),
    (dict(q=fake(3), scales=fake(4), rstd=fake(4) + 16), 1),
    (dict(rows=0, x=None, w=None, y=None), 0),
])
def test_rms_norm_fwd_refusals(kw, code):
    assert norm_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(d=12), 2), (dict(dy=None), 1), (dict(rstd=None), 1), (dict(dw=None), 1), (dict(ws=None), 1),
    (dict(dres=ODD), 3), (dict(bytes=16), 4), (dict(dx=fake(0) + 256), 1), (dict(dx=fake(1) + 256), 1),
    (dict(dw=fake(2)), 1), (dict(dw=fake(4)), 1), (dict(dw=fake(0) + 16), 1), (dict(ws=fake(5)), 1), (dict(ws=fake(1)), 1),
    (dict(dx=fake(2)), 1), (dict(dx=fake(3)), 1), (dict(dres=fake(7), ws=fake(7) + 2032), 1),
    (dict(rows=0, dw=fake(2)), 1)])
def test_rms_norm_bwd_refusals(kw, code):
    a = dict(rows=4, d=256, dy=fake(0), h=fake(1), w=fake(2), rstd=fake(3), dres=None, dx=fake(4), dw=fake(5), ws=fake(6),
             bytes=1 << 40)
    a.update(kw)
    assert up.lib().upipe_attn_rms_norm_bwd(a["rows"], a["d"], a["dy"], a["h"], a["w"], a["rstd"], a["dres"], a["dx"],
                                            a["dw"], a["ws"], a["bytes"], None) == code


def test_rms_norm_workspace():
    assert up.rms_norm_workspace_bytes(1, 64) >= 64 * 4
    a, b = (up.rms_norm_workspace_bytes(n, 4096) for n in (1 << 20, 1 << 24))
    assert a == b                                     # a share per resident group of threads, not per row
    for d in (8, 4096, 5120, 8192, 8208, 10240, 16384, 32768):         # a share per group, at most a row's threads each
        assert up.rms_norm_workspace_bytes(1, d) <= 16 * 4 * d
    with pytest.raises(up.UpipeError):
        up.rms_norm_workspace_bytes(4, 20)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(cols=24), 2), (dict(block=64), 1), (dict(x=None), 1), (dict(q=ODD), 3),
    (dict(q=fake(0) + 1024), 1), (dict(scales=fake(0)), 1), (dict(scales=fake(1) + 16), 1), (dict(block=128, scales=fake(1)), 1),
    (dict(rows=0, x=None, q=None, scales=None), 0)])
def test_fp8_quantize_refusals(kw, code):
    a = dict(rows=4, cols=256, block=1, x=fake(0), q=fake(1), scales=fake(2))
    a.update(kw)
    assert up.lib().upipe_attn_fp8_quantize(a["rows"], a["cols"], a["block"], a["x"], a["q"], a["scales"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(M=1 << 31), 1), (dict(K=24, lda=32, ldb=32), 2), (dict(N=12, ldc=16), 2),
    (dict(lda=128), 1), (dict(ldb=264), 2), (dict(ldc=100), 1), (dict(ldc=516), 2), (dict(lds=63), 1), (dict(ct=2), 1), (dict(A=None), 1),
    (dict(sb=None), 1), (dict(A=ODD), 3), (dict(C=ODD), 3), (dict(sa=ODD), 3),
    (dict(C=fake(0)), 1), (dict(C=fake(2) + 4096), 1),  # C over A, inside B
    (dict(C=fake(1)), 1), (dict(C=fake(3)), 1),         # over the scales
    (dict(M=1 << 30, N=1 << 30, ldc=1 << 30, lds=1 << 30), 2),
    (dict(M=0, A=None, sa=None, C=None), 0)])
def test_gemm_fp8_refusals(kw, code):
    a = dict(M=64, N=512, K=256, A=fake(0), lda=256, sa=fake(1), lds=64, B=fake(2), ldb=256, sb=fake(3), C=fake(4), ldc=512,
             ct=1)
    a.update(kw)
    assert up.lib().upipe_attn_gemm_fp8_nt(a["M"], a["N"], a["K"], a["A"], a["lda"], a["sa"], a["lds"], a["B"], a["ldb"],
                                           a["sb"], a["C"], a["ldc"], a["ct"], None) == code


def rope_side(**kw):
    a = dict(in_=fake(0), out=fake(1), in_head_stride=64 * 128, in_token_stride=128, out_head_stride=64 * 128,
             out_token_stride=128, n_heads=4)
    a.update(kw)
    return up.RopeTensor(*(a[f] for f, _ in up.RopeTensor._fields_))


def rope(side, desc=None, tokens=64, pos=fake(9), k=None):
    desc = desc or up.make_rope_desc(128, [1.0 / (j + 1) for j in range(64)])
    return up.lib().upipe_attn_rope(ctypes.byref(desc), tokens, pos, ctypes.byref(side), ctypes.byref(k) if k else None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(in_=None), 1), (dict(out=None), 1), (dict(n_heads=-1), 1), (dict(in_=ODD), 3), (dict(in_token_stride=132), 2),
    (dict(in_head_stride=-128), 1), (dict(out_token_stride=0), 1), (dict(out_head_stride=128), 1),
    (dict(out_token_stride=64), 1),                                  # rows of the output overlap
    (dict(out=fake(0), out_head_stride=128, out_token_stride=512), 1),  # in place, other strides
    (dict(out=fake(0) + 256), 1), (dict(n_heads=65536, in_head_stride=0, out_head_stride=8192), 2)])
def test_rope_refuses_layouts(kw, code):
    assert rope(rope_side(**kw)) == code
    good = rope_side(in_=fake(2), out=fake(3))
    if kw.get("n_heads", 1) < 65536:
        assert rope(good, k=rope_side(**kw)) == code


def test_rope_tells_parts_of_one_tensor_from_tensors_that_meet():
    """Only refusals are called here: what is accepted would launch."""
    tok = 12 * 128                                                     # token-major: 8 + 2 + 2 heads of 128
    side = lambda base, out, heads, hs=128, ts=tok, oh=128, ot=tok: up.RopeTensor(base, out, hs, ts, oh, ot, heads)
    a, b = fake(0), fake(5)
    kb = 8 * 128 * 2                                                   # bytes to the first key head
    bad = [
        (side(a, b, 8), side(a + kb, b, 2)),                           # the same output twice
        (side(a, b, 8), side(a + kb, b + kb - 256, 2)),                # outputs that share a head
        (side(a, a + 256, 2), None),                                   # moved by one head, over its neighbour
        (side(a, a, 8), side(a + kb - 256, b, 2)),                     # q in place over a head that k reads
        (side(a + kb, b, 2), side(a, a, 9)),                           # k in place over heads that q reads
        (side(a, b, 8), side(a + kb, b + kb, 2, oh=128, ot=tok * 2)),  # outputs of different strides, ranges that overlap
        (side(a, b, 8, oh=64 * 128, ot=128), side(a + kb, b + 2 * 7 * 64 * 128, 2, oh=64 * 128, ot=128)),
    ]
    for q, k in bad:
        assert rope(q, k=k) == 1
    one = up.RopeTensor(a, ODD, 3, 5, 3, 5, 1)                         # one head, one token: strides do not count
    assert rope(one, tokens=1) == 3


def test_rope_refuses_descriptors():
    good = [0.5] * 64
    for change, code in (({"head_dim": 120}, 1), ({"head_dim": 136}, 2), ({"head_dim": 272}, 2), ({"rotary_dim": 0}, 1),
                         ({"rotary_dim": 24}, 2), ({"n_axes": 0}, 1), ({"n_axes": 5}, 1), ({"adjacent": 2}, 1), ({"inverse": -1}, 1)):
        d = up.make_rope_desc(128, good)
        for f, v in change.items():
            setattr(d, f, v)
        assert rope(rope_side(), d) == code, change
    d = up.make_rope_desc(128, good, [0] * 63 + [2])
    d.n_axes = 2
    assert rope(rope_side(), d) == 1                                  # a pair reads a row of positions that is not there
    assert rope(rope_side(), up.make_rope_desc(128, [math.inf] + good[1:])) == 1
    assert rope(rope_side(), pos=None) == 1
    assert rope(rope_side(), pos=ODD) == 3
    assert rope(rope_side(), pos=fake(1) + 64) == 1                   # positions inside the output
    assert rope(rope_side(), pos=fake(4) - 16, k=rope_side(in_=fake(3), out=fake(4))) == 1
    assert rope(rope_side(), tokens=-1) == 1
    assert rope(rope_side(in_=None, out=None), tokens=0, pos=None) == 0
    for bad in (([0.1] * 129, None), (good, [0] * 63), (good, [4] * 64), (good, [-1] * 64)):
        with pytest.raises(up.UpipeError):
            up.make_rope_desc(128, *bad)


def clip(entries, max_norm=1.0, norm=fake(30), ws=fake(31), ws_bytes=1 << 40):
    arr = (up.GradTensor * max(1, len(entries)))(*(up.GradTensor(*e) for e in entries))
    return up.lib().upipe_attn_grad_clip(arr, len(entries), max_norm, norm, ws, ws_bytes, None)


def test_grad_clip_refusals():
    one = (fake(0), None, 100, 0, 0)
    assert clip([one], max_norm=0.0) == 1
    assert clip([one], max_norm=-1.0) == 1
    assert clip([one], max_norm=math.nan) == 1
    assert clip([one], norm=None) == 1
    assert clip([one], ws=None) == 1
    assert clip([one], ws=ODD) == 3
    assert clip([one], ws_bytes=8) == 4
    assert clip([(None, None, 1, 0, 0)]) == 1
    assert clip([(fake(0), None, -1, 0, 0)]) == 1
    assert clip([(fake(0), None, 4, 2, 0)]) == 1
    assert clip([(fake(0), fake(1), 4, 0, 2)]) == 1
    assert clip([(ODD, None, 4, 0, 0)]) == 3
    assert clip([(fake(0), ODD, 4, 0, 0)]) == 3
    assert clip([one, one]) == 1                                      # the same tensor twice
    assert clip([one, (fake(0) + 384, None, 100, 0, 0)]) == 1          # two that overlap
    assert clip([one, (fake(1), fake(0) + 16, 4, 0, 0)]) == 1          # an output inside another gradient
    assert clip([(fake(0), fake(0), 4, 0, 1)]) == 1                    # in place into another type
    assert clip([one], norm=fake(0) + 16) == 1                        # the norm, the workspace over a tensor
    assert clip([one], ws=fake(0) + 384) == 1
    assert clip([(fake(0), fake(31) + 64, 100, 0, 0)]) == 1
    assert clip([one], norm=fake(31)) == 1
    n = ctypes.c_size_t(0)
    assert up.lib().upipe_attn_grad_clip_workspace_size(-1, ctypes.byref(n)) == 1
    assert up.lib().upipe_attn_grad_clip_workspace_size(4, None) == 1


def test_binding_refuses_tensors_that_are_not_on_the_gpu():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(2, 4)
    f = torch.zeros(256)
    desc = up.make_rope_desc(64, [0.5] * 32)
    for call in (lambda: up.rms_norm_fwd(x, x[0], x.clone()), lambda: up.rms_norm_fwd_fp8(x, x[0], q, s),
                 lambda: up.rms_norm_fwd_fp8(x, x[0], None, None), lambda: up.rms_norm_fwd(x[0], x[0], x[0]),
                 lambda: up.rms_norm_bwd(x, x, x[0], f[:4], x, f, q), lambda: up.fp8_quantize(x, q, s),
                 lambda: up.fp8_quantize(x, q, s, block_rows=2), lambda: up.gemm_fp8_nt(q, s, q, s[:1, :2], x[:, :4]),
                 lambda: up.rope(desc, x.view(4, 4, 64), None, torch.zeros(1, 4, dtype=torch.int32), x.view(4, 4, 64), None),
                 lambda: up.rope(desc, x, None, torch.zeros(1, 4, dtype=torch.int32), x, None),
                 lambda: up.GradClip([x]), lambda: up.GradClip([x.double()]), lambda: up.GradClip([x], [])):
        with pytest.raises(ValueError):
            call()
