"""Cases of the operators around the attention layer and the feed-forward step of a transformer block:
the root-mean-square norm with the residual's addition (to bf16, to e4m3 with a scale for each block of
128, and backward), the 8-bit block quantiser, the 8-bit block-scaled matrix product, rotary positions
with several axes, and the global gradient norm with clipping.

`run` computes each operator in plain torch, or, where `own` is true, calls the library's entry points.
`exact` restates each operator in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128          # elements (of K, or of a weight's rows) that share a scale
E4M3_MAX = 448.0     # largest finite e4m3 value
TINY = 2.0 ** -100   # a block whose largest magnitude is below this has scale 1 and quantises to zeros
EPS = 1e-5           # of the norm
CLIP_EPS = 1e-6      # of the clip's divisor


def listed():
    return [
        # one decoded token passes a 4096-wide block: residual addition and norm before the projections
        dict(name="norm_fwd_1x4096", op="norm_fwd", rows=1, d=4096, residual=True, out="bf16"),
        # a 32K-token sequence, norm straight into the 8-bit operand of the QKV or gate/up product
        dict(name="norm_fwd_e4m3_32768x4096", op="norm_fwd", rows=32768, d=4096, residual=True, out="e4m3"),
        # backward in training at the 5120-wide model's hidden size, a ragged shard of a packed sequence; the gradient
        # of the residual stream is added on the way
        dict(name="norm_bwd_16381x5120", op="norm_bwd", rows=16381, d=5120, residual=True),
        # the gate/up weights are quantised once for each training step
        dict(name="quant_weight_28672x4096", op="quant", rows=28672, d=4096, block=128),
        # activations of a ragged batch, last column block partly filled (d = 8 * 128 + 16)
        dict(name="quant_rows_1001x1040", op="quant", rows=1001, d=1040, block=1),
        # decode: 16 sequences' tokens through the QKV projection of the 8B-shaped layer
        dict(name="gemm_16x6144x4096", op="gemm", m=16, n=6144, k=4096),
        # a ragged prefill batch through the output projection of a 5120-wide layer
        dict(name="gemm_1000x5120x8192", op="gemm", m=1000, n=5120, k=8192),
        # one 8192-row tile of the sequence-tiled feed-forward step: gate/up product
        dict(name="gemm_8192x28672x4096", op="gemm", m=8192, n=28672, k=4096),
        # one decoded token: text positions, far into a long sequence
        dict(name="rope_1_text", op="rope", tokens=1, hq=32, hkv=8, dh=128, rotary=128, axes=1, pairs="split", inverse=False),
        # backward over 32K tokens of video (time, height, width): the attention core's dQ and dK, head by head, turned
        # back into the gradient of the projection's output
        dict(name="rope_32768_video_bwd", op="rope", tokens=32768, hq=32, hkv=8, dh=128, rotary=128, axes=3, pairs="split", inverse=True),
        # the weight gradients of one 8B-shaped layer, clipped into the bf16 copies that are reduced
        dict(name="clip_1_layer_8b", op="clip", layers=1, hidden=4096, heads=48, ffn=14336, extra=0, out="bf16"),
        # many small tensors of a narrow stack, one of an odd length, clipped in 32 bits
        dict(name="clip_8_layers_512", op="clip", layers=8, hidden=512, heads=12, ffn=1408, extra=1000003, out="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _step(x, step):
    return max(step, x // step * step)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_fwd", "norm_bwd", "quant", "gemm", "gemm", "rope", "rope", "clip"])
    if op in ("norm_fwd", "norm_bwd"):
        out = rng.choice(["bf16", "e4m3"])
        d = _step(_log(rng, 64, 8192), 16 if out == "e4m3" else 8)
        rows = _log(rng, 1, min(65536, 32768 * 4096 // d))
        case = dict(op=op, rows=rows, d=d, residual=rng.random() < 0.6)
        return dict(case, out=out) if op == "norm_fwd" else case
    if op == "quant":
        d = _step(_log(rng, 64, 8192), 16)
        return dict(op=op, rows=_log(rng, 1, min(32768, 28672 * 4096 // d)), d=d, block=rng.choice([1, 128]))
    if op == "gemm":
        n, k = _step(_log(rng, 64, 28672), 8), _step(_log(rng, 64, 14336), 16)
        return dict(op=op, m=_log(rng, 1, min(8192, 8192 * 28672 * 4096 // (n * k))), n=n, k=k)
    if op == "rope":
        dh = rng.choice([64, 80, 128])
        hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 32768), hq=hkv * rng.choice([1, 2, 4]), hkv=hkv, dh=dh,
                    rotary=rng.choice([dh, _step(dh // 2, 16)]), axes=rng.choice([1, 2, 3]),
                    pairs=rng.choice(["split", "adjacent"]), inverse=rng.random() < 0.5)
    hidden = _step(_log(rng, 64, 4096), 64)
    return dict(op=op, layers=rng.randint(1, 8) if hidden < 1024 else 1, hidden=hidden, heads=_step(_log(rng, 4, 48), 2),
                ffn=_step(_log(rng, 64, 14336), 64), extra=rng.choice([0, 1, 1000003]), out=rng.choice(["bf16", "fp32"]))


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, d):
    """Hidden states: channels of different strength, one in a hundred an outlier channel."""
    strength = torch.exp(0.5 * _randn(g, d))
    strength = torch.where(torch.rand(d, generator=g, device="cuda") < 0.01, 20 * strength, strength)
    return (_randn(g, rows, d) * strength).bfloat16()


def _blocks(x, br, bc):
    """x [rows, cols] zero-padded and cut into blocks: [row blocks, br, column blocks, bc]."""
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % bc, 0, -r % br))
    return x.view(x.shape[0] // br, br, x.shape[1] // bc, bc)


def _quant(x, br):
    """Codes and scales of fp32 x, a scale for each block of br rows and 128 columns."""
    b = _blocks(x, br, BLOCK)
    amax = b.abs().amax(dim=(1, 3))
    s = torch.where(amax < TINY, torch.ones_like(amax), amax / E4M3_MAX)
    q = (b / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    q = q.reshape(b.shape[0] * br, -1)[: x.shape[0], : x.shape[1]]
    return q.to(torch.float8_e4m3fn), s


def _clip_sizes(c):
    h, dh = c["hidden"], 128
    layer = [c["heads"] * dh * h, h * c["heads"] * dh * 2 // 3, 2 * c["ffn"] * h, h * c["ffn"], h, h]
    return layer * c["layers"] + ([c["extra"]] if c["extra"] else [])


def _rope_plan(c):
    """Angular step of each rotary pair, the positions' axis that it reads, and the pairs of a row."""
    half = c["rotary"] // 2
    inv_freq = [500000.0 ** (-j / half) for j in range(half)]
    axis = [j * c["axes"] // half for j in range(half)]
    return inv_freq, axis


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c, keep={})
    if c["op"] in ("norm_fwd", "norm_bwd"):
        rows, d = c["rows"], c["d"]
        s["x"] = _activations(g, rows, d)
        s["w"] = (1 + 0.1 * _randn(g, d)).bfloat16()
        if c["op"] == "norm_fwd":
            s["res"] = _activations(g, rows, d) if c["residual"] else None
            s["h"] = torch.empty_like(s["x"]) if c["residual"] else None
            s["rstd"] = torch.empty(rows, device="cuda")
            if c["out"] == "bf16":
                s["y"] = torch.empty_like(s["x"])
            else:
                s["q"] = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda")
                s["scales"] = torch.empty(-(-d // BLOCK), rows, device="cuda")
        else:  # what the forward pass left: h (as x) and 1 / rms
            s["dy"] = _randn(g, rows, d).bfloat16()
            s["dres"] = _randn(g, rows, d).bfloat16() if c["residual"] else None
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty(d, device="cuda")
    elif c["op"] == "quant":
        rows, d = c["rows"], c["d"]
        s["x"] = _activations(g, rows, d) if c["block"] == 1 else (0.02 * _randn(g, rows, d)).bfloat16()
        s["q"] = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda")
        nb = -(-d // BLOCK)
        s["scales"] = torch.empty(*((nb, rows) if c["block"] == 1 else (-(-rows // BLOCK), nb)), device="cuda")
    elif c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        s["a"], sa = _quant(_activations(g, m, k).float(), 1)
        s["sa"] = sa.t().contiguous()
        s["b"], s["sb"] = _quant(0.02 * _randn(g, n, k), BLOCK)
        s["c"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "rope":
        t, hq, hkv, dh = c["tokens"], c["hq"], c["hkv"], c["dh"]
        s["qkv"] = _randn(g, t, hq + 2 * hkv, dh).bfloat16()  # as the projection writes it, token by token
        s["q"] = _randn(g, hq, t, dh).bfloat16()  # as the attention core reads and writes them, head by head
        s["k"] = _randn(g, hkv, t, dh).bfloat16()
        first = int(torch.randint(0, 5_000_000, (1,), generator=g, device="cuda"))
        idx = torch.arange(t, device="cuda")
        if c["axes"] == 1:
            pos = (first + idx)[None]
        else:  # frames of 16 x 24 patches
            pos = torch.stack([first + idx // 384, first + idx // 24 % 16, first + idx % 24])[: c["axes"]]
        s["pos"] = pos.int().contiguous()
    else:
        s["grads"] = [_randn(g, n) * 1e-3 for n in _clip_sizes(c)]
        kind = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        s["outs"] = [torch.empty_like(t, dtype=kind) for t in s["grads"]]
        s["max_norm"] = 1.0 if seed % 4 else 1e4  # most steps are clipped, some are not
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def _rms(x, res):
    h = x.float()
    if res is not None:
        h = (h + res.float()).bfloat16().float()  # the residual stream is stored in bf16
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    return h, rstd


def _norm_fwd(s):
    h, rstd = _rms(s["x"], s["res"])
    y = h * rstd[:, None] * s["w"].float()
    out = dict(rstd=rstd)
    if s["res"] is not None:
        out["h"] = h.bfloat16()
    if s["case"]["out"] == "bf16":
        out["y"] = y.bfloat16()
    else:
        q, scales = _quant(y, 1)
        out["q"], out["scales"] = q, scales.t().contiguous()
    return out


def _norm_bwd(s):
    h, rstd, dy = s["x"].float(), s["rstd"][:, None], s["dy"].float()
    t = dy * s["w"].float()
    dx = rstd * (t - h * (rstd * rstd * (t * h).mean(1, keepdim=True)))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.bfloat16(), dw=(dy * h * rstd).sum(0))


def _quantise(s):
    q, scales = _quant(s["x"].float(), s["case"]["block"])
    return dict(q=q, scales=scales.t().contiguous() if s["case"]["block"] == 1 else scales)


def _gemm(s):
    n, k = s["b"].shape
    a = s["a"].float() * s["sa"].t().repeat_interleave(BLOCK, 1)[:, :k]
    b = s["b"].float() * s["sb"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return (a @ b.t()).bfloat16()


def _rotate(x, cos, sin, c):
    """x [tokens, heads, dh] in fp32; cos, sin [tokens, 1, rotary / 2]."""
    r, half = c["rotary"], c["rotary"] // 2
    if c["pairs"] == "split":
        a, b = x[..., :half], x[..., half:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _rope(s):
    c = s["case"]
    inv_freq, axis = _rope_plan(c)
    f = torch.tensor(inv_freq, dtype=torch.float64, device="cuda")
    angle = s["pos"].double()[torch.tensor(axis, device="cuda")].t() * f  # [tokens, pairs]: far positions need 64 bits
    if c["inverse"]:
        angle = -angle
    x = torch.cat([s["q"], s["k"]]).transpose(0, 1) if c["inverse"] else s["qkv"][:, : c["hq"] + c["hkv"]]
    y = _rotate(x.float(), angle.cos().float()[:, None], angle.sin().float()[:, None], c).bfloat16()
    if c["inverse"]:
        return y.contiguous()
    y = y.transpose(0, 1).contiguous()
    return dict(q=y[: c["hq"]], k=y[c["hq"]:])


def _clip(s):
    total = torch.stack([(t * t).sum(dtype=torch.float64) for t in s["grads"]]).sum()
    norm = total.sqrt().float()
    coef = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    return dict(norm=norm.reshape(1), out=[(t * coef).to(o.dtype) for t, o in zip(s["grads"], s["outs"])])


def _own(s):
    import long_context_attention_upipe_gb300 as up

    c, keep = s["case"], s["keep"]
    if c["op"] == "norm_fwd":
        if c["out"] == "bf16":
            up.rms_norm_fwd(s["x"], s["w"], s["y"], s["rstd"], residual=s["res"], h=s["h"], eps=EPS)
        else:
            up.rms_norm_fwd_fp8(s["x"], s["w"], s["q"], s["scales"], s["rstd"], residual=s["res"], h=s["h"], eps=EPS)
        return {k: s[k] for k in ("rstd", "h", "y", "q", "scales") if s.get(k) is not None}
    if c["op"] == "norm_bwd":
        if "ws" not in keep:  # a program allocates its workspace once
            keep["ws"] = torch.empty(up.rms_norm_workspace_bytes(c["rows"], c["d"]), dtype=torch.uint8, device="cuda")
        up.rms_norm_bwd(s["dy"], s["x"], s["w"], s["rstd"], s["dx"], s["dw"], keep["ws"], dres=s["dres"])
        return dict(dx=s["dx"], dw=s["dw"])
    if c["op"] == "quant":
        up.fp8_quantize(s["x"], s["q"], s["scales"], block_rows=c["block"])
        return dict(q=s["q"], scales=s["scales"])
    if c["op"] == "gemm":
        up.gemm_fp8_nt(s["a"], s["sa"], s["b"], s["sb"], s["c"])
        return s["c"]
    if c["op"] == "rope":
        if "desc" not in keep:  # the model's rotary description
            inv_freq, axis = _rope_plan(c)
            keep["desc"] = up.make_rope_desc(c["dh"], inv_freq, axis, adjacent=c["pairs"] == "adjacent")
        heads = s["qkv"].transpose(0, 1)
        hq, hk = heads[: c["hq"]], heads[c["hq"]: c["hq"] + c["hkv"]]
        if c["inverse"]:
            up.rope(keep["desc"], s["q"], s["k"], s["pos"], hq, hk, inverse=True)
            return s["qkv"][:, : c["hq"] + c["hkv"]]
        up.rope(keep["desc"], hq, hk, s["pos"], s["q"], s["k"])
        return dict(q=s["q"], k=s["k"])
    if "clip" not in keep:  # the list of the model's gradients, with its workspace
        keep["clip"] = up.GradClip(s["grads"], s["outs"])
    norm = keep["clip"](s["max_norm"])
    return dict(norm=norm, out=s["outs"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "norm_fwd":
        return _norm_fwd(state)
    if op == "norm_bwd":
        return _norm_bwd(state)
    if op == "quant":
        return _quantise(state)
    if op == "gemm":
        return _gemm(state)
    if op == "rope":
        return _rope(state)
    return _clip(state)


def work(case):
    """Each input read once, each output written once."""
    c = case
    if c["op"] == "norm_fwd":
        n = c["rows"] * c["d"]
        out = 2 * n if c["out"] == "bf16" else n + 4 * c["rows"] * -(-c["d"] // BLOCK)
        return dict(bytes=2 * n + (4 * n if c["residual"] else 0) + out + 2 * c["d"] + 4 * c["rows"], flops=5 * n)
    if c["op"] == "norm_bwd":
        n = c["rows"] * c["d"]
        return dict(bytes=6 * n + (2 * n if c["residual"] else 0) + 6 * c["d"] + 4 * c["rows"], flops=10 * n)
    if c["op"] == "quant":
        n, nb = c["rows"] * c["d"], -(-c["d"] // BLOCK)
        return dict(bytes=3 * n + 4 * nb * -(-c["rows"] // c["block"]), flops=3 * n)
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        nk = -(-k // BLOCK)
        return dict(bytes=m * k + n * k + 2 * m * n + 4 * nk * (m + -(-n // BLOCK)), flops=2 * m * n * k)
    if c["op"] == "rope":
        n = c["tokens"] * (c["hq"] + c["hkv"]) * c["dh"]
        return dict(bytes=4 * n + 4 * c["axes"] * c["tokens"], flops=3 * n * c["rotary"] // c["dh"])
    n = sum(_clip_sizes(c))
    return dict(bytes=n * (4 + (2 if c["out"] == "bf16" else 4)) + 4, flops=3 * n)


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------

def _exact_quant(x, br):
    """Block maxima / 448 and the values divided by them, before the rounding to e4m3."""
    rows, d = x.shape
    nr, nc = -(-rows // br), -(-d // BLOCK)
    scale = torch.empty(nr, nc, dtype=torch.float64, device="cuda")
    for j in range(nc):
        top = x[:, j * BLOCK: (j + 1) * BLOCK].abs().max(1).values
        top = torch.cat([top, top.new_zeros(nr * br - rows)]).view(nr, br).max(1).values
        scale[:, j] = torch.where(top < TINY, torch.ones_like(top), top / E4M3_MAX)
    value = torch.empty_like(x)
    per_row = scale[torch.arange(rows, device="cuda") // br]
    for j in range(nc):
        value[:, j * BLOCK: (j + 1) * BLOCK] = x[:, j * BLOCK: (j + 1) * BLOCK] / per_row[:, j: j + 1]
    return value, scale


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm_fwd":
        h = s["x"].double()
        if c["residual"]:
            h = (h + s["res"].double()).to(torch.bfloat16).double()  # both are bf16: the sum in 64 bits is exact
        ms = torch.linalg.vector_norm(h, dim=1) ** 2 / c["d"]
        rstd = 1.0 / torch.sqrt(ms + EPS)
        y = torch.einsum("rd,r,d->rd", h, rstd, s["w"].double())
        out = dict(rstd=rstd)
        if c["residual"]:
            out["h"] = h
        if c["out"] == "bf16":
            out["y"] = y
        else:
            out["q"], scale = _exact_quant(y, 1)
            out["scales"] = scale.t().contiguous()
        return out
    if c["op"] == "norm_bwd":  # through the product rule on y = h * rstd * w, rstd = (mean h^2 + eps)^(-1/2)
        h, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        rstd = (torch.linalg.vector_norm(h, dim=1) ** 2 / c["d"] + EPS) ** -0.5
        drstd = torch.einsum("rd,rd,d->r", dy, h, w)
        dx = torch.einsum("rd,d,r->rd", dy, w, rstd) - torch.einsum("r,r,rd->rd", drstd, rstd ** 3 / c["d"], h)
        dw = torch.einsum("rd,rd,r->d", dy, h, rstd)
        return dict(dx=dx + s["dres"].double() if c["residual"] else dx, dw=dw)
    if c["op"] == "quant":
        q, scale = _exact_quant(s["x"].double(), c["block"])
        return dict(q=q, scales=scale.t().contiguous() if c["block"] == 1 else scale)
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        out = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        for k0 in range(0, k, BLOCK):  # block by block: the scales leave the sum over a block
            part = s["a"][:, k0: k0 + BLOCK].double() @ s["b"][:, k0: k0 + BLOCK].double().t()
            part *= s["sa"][k0 // BLOCK].double()[:, None]
            part *= s["sb"][:, k0 // BLOCK].double()[torch.arange(n, device="cuda") // BLOCK]
            out += part
        return out
    if c["op"] == "rope":
        inv_freq, axis = _rope_plan(c)
        x = s["qkv"].double()[:, : c["hq"] + c["hkv"]]
        if c["inverse"]:
            x = torch.cat([s["q"], s["k"]]).double().permute(1, 0, 2)
        y = x.clone()
        half = c["rotary"] // 2
        for j in range(half):  # each pair as a complex number times e^(i angle)
            angle = s["pos"][axis[j]].double() * inv_freq[j] * (-1.0 if c["inverse"] else 1.0)
            i0, i1 = (j, j + half) if c["pairs"] == "split" else (2 * j, 2 * j + 1)
            z = torch.complex(x[..., i0], x[..., i1]) * torch.polar(torch.ones_like(angle), angle)[:, None]
            y[..., i0], y[..., i1] = z.real, z.imag
        if c["inverse"]:
            return y.contiguous()
        y = y.permute(1, 0, 2)
        return dict(q=y[: c["hq"]].contiguous(), k=y[c["hq"]:].contiguous())
    norm = math.sqrt(math.fsum(float(t.double().square().sum()) for t in s["grads"]))
    coef = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
    return dict(norm=torch.tensor([norm], dtype=torch.float64), out=[t.double() * coef for t in s["grads"]])
