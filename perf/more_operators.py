"""Cases of the paged cache of keys and values and of the attention that reads it: writing new tokens' keys and
values into pages (bf16, or e4m3 with a scale for each token and head), reading them back, and the attention of the
newest tokens of many sequences over their cached keys.

`run` computes each operator in plain torch, or, where `own` is true, calls the library's entry points.
`exact` restates each operator in 64 bits.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0     # largest finite e4m3 value
TINY = 2.0 ** -100   # a row whose largest magnitude is below this has scale 1 and quantises to zeros


def listed():
    return [
        # a decode step of 16 sequences writes one token each (8 key heads of the 8B-shaped layer)
        dict(name="write_16_e4m3", op="write", seqs=16, longest=8192, new=1, hq=32, hkv=8, dh=128, page=64, kind="e4m3"),
        # a 32K-token prompt goes into a bf16 cache
        dict(name="write_32768_bf16", op="write", seqs=1, longest=32768, new=0, hq=32, hkv=8, dh=128, page=64, kind="bf16"),
        # 15 prompts of a packed batch go into an 8-bit cache
        dict(name="write_15_prompts_e4m3", op="write", seqs=15, longest=16384, new=0, hq=32, hkv=8, dh=128, page=128, kind="e4m3"),
        # short sequences of a small model leave a bf16 cache (handed to another worker)
        dict(name="read_5_short_bf16", op="read", seqs=5, longest=1001, new=0, hq=4, hkv=2, dh=64, page=16, kind="bf16"),
        # the 1M-token share's one key head, back to bf16 for the attention core
        dict(name="read_1048576_e4m3", op="read", seqs=1, longest=1048576, new=0, hq=4, hkv=1, dh=128, page=128, kind="e4m3"),
        # one user, a page begun: latency
        dict(name="decode_1x4097_bf16", op="decode", seqs=1, longest=4097, new=1, hq=32, hkv=8, dh=128, page=64, kind="bf16"),
        # the 1M-token share: one sequence, one key head, split over its length
        dict(name="decode_1x1048576_bf16", op="decode", seqs=1, longest=1048576, new=1, hq=4, hkv=1, dh=128, page=128, kind="bf16"),
        # the 5M-token share of the 32B-shaped layer, 8 query heads on one key head, 8-bit cache
        dict(name="decode_1x5242880_e4m3", op="decode", seqs=1, longest=5242880, new=1, hq=8, hkv=1, dh=128, page=128, kind="e4m3"),
        # serving: 64 sequences of very different lengths, 8-bit cache
        dict(name="decode_64x16384_e4m3", op="decode", seqs=64, longest=16384, new=1, hq=32, hkv=8, dh=128, page=64, kind="e4m3"),
        # the 5120-wide model's 40 query heads over 8 key heads, bf16 cache
        dict(name="decode_48x8192_bf16", op="decode", seqs=48, longest=8192, new=1, hq=40, hkv=8, dh=128, page=32, kind="bf16"),
        # many short sequences of a small model, one slot in eight empty
        dict(name="decode_256x500_bf16", op="decode", seqs=256, longest=500, new=1, hq=4, hkv=2, dh=64, page=16, kind="bf16"),
        # four drafted tokens of each sequence at once
        dict(name="decode_16x32768_4_e4m3", op="decode", seqs=16, longest=32768, new=4, hq=32, hkv=8, dh=128, page=64, kind="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "write", "read", "decode", "decode", "decode", "decode"])
    dh, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    case = dict(op=op, hq=hkv * rng.choice([1, 2, 4, 5, 8]), hkv=hkv, dh=dh, page=rng.choice([16, 32, 48, 64, 128]),
                kind=rng.choice(["bf16", "e4m3"]))
    seqs = _log(rng, 1, 256)
    if op == "decode":  # keys of all sequences, padded to the longest
        most = 2_000_000 // hkv
        return dict(case, seqs=seqs, longest=_log(rng, 1, max(2, most // seqs)), new=rng.choice([1, 1, 1, 2, 3, 4, 8]))
    if op == "write" and rng.random() < 0.4:
        return dict(case, seqs=seqs, longest=_log(rng, 1, 8192), new=rng.choice([1, 1, 2, 4]))
    return dict(case, seqs=seqs, longest=_log(rng, 1, max(2, 500_000 // (hkv * seqs))), new=0)


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _lens(c):
    """Keys of each sequence: the longest, and shorter ones down to a hundredth of it; with one in eight slots of a
    large batch empty.  They are part of the case."""
    rng = random.Random(c["seqs"] * 1000003 + c["longest"])
    lens = [c["longest"]]
    while len(lens) < c["seqs"]:
        empty = c["op"] == "decode" and c["seqs"] >= 128 and rng.random() < 0.125
        lens.append(0 if empty else max(1, _log(rng, max(1, c["longest"] // 100), c["longest"])))
    return lens


def _places(c):
    """(sequence, position) of every token that is written or read: the newest `new` of each sequence, or all."""
    out = []
    for b, n in enumerate(_lens(c)):
        out += [(b, p) for p in range(max(0, n - c["new"]) if c["new"] else 0, n)]
    return out


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _quant(x):
    """Codes and scales of fp32 rows, a scale for each row."""
    amax = x.abs().amax(-1)
    s = torch.where(amax < TINY, torch.ones_like(amax), amax * (1.0 / E4M3_MAX))
    q = (x / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn), s


def _pool(g, pages, c, strength):
    """A cache's rows as earlier calls left them: codes and scales, or bf16 and None."""
    x = _randn(g, pages, c["hkv"], c["page"], c["dh"]) * strength
    return _quant(x) if c["kind"] == "e4m3" else (x.bfloat16(), None)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c, keep={})
    lens = _lens(c)
    held = [-(-n // c["page"]) for n in lens]
    pages = sum(held) + 3
    # channels of keys differ in strength; the queries' are such that scores spread over a few units
    strength = torch.exp(0.5 * _randn(g, c["dh"]))
    s["k_cache"], s["k_scale"] = _pool(g, pages, c, strength)
    s["v_cache"], s["v_scale"] = _pool(g, pages, c, torch.ones_like(strength))
    # pages are given out as they come free: any order; the table's unused entries are -1
    order = torch.randperm(pages, generator=g, device="cuda").int()
    used = torch.arange(max(held), device="cuda")[None] < torch.tensor(held, device="cuda")[:, None]
    table = torch.full((c["seqs"], max(held)), -1, dtype=torch.int32, device="cuda")
    table[used] = order[: sum(held)]
    s["table"] = table
    if c["op"] == "decode":
        t = c["seqs"] * c["new"]
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = (2 * _randn(g, c["hq"], t, c["dh"]) / strength).bfloat16()  # as the rotation writes it, head by head
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(c["hq"], t, device="cuda")
        return s
    if c["new"]:
        place = torch.tensor(_places(c), dtype=torch.int32, device="cuda")
        s["seq"], s["pos"] = place[:, 0].contiguous(), place[:, 1].contiguous()
    else:
        n = torch.tensor(lens, device="cuda")
        s["seq"] = torch.arange(c["seqs"], device="cuda").repeat_interleave(n).int()
        first = (n.cumsum(0) - n).repeat_interleave(n)
        s["pos"] = (torch.arange(sum(lens), device="cuda") - first).int()
    t = s["seq"].numel()
    s["k"] = (_randn(g, c["hkv"], t, c["dh"]) * strength).bfloat16()  # as the rotation writes it, head by head
    if c["op"] == "write":  # the values are a part of the projection's output, token by token
        s["kv"] = _randn(g, t, 2 * c["hkv"], c["dh"]).bfloat16()
        s["v"] = s["kv"][:, c["hkv"]:].transpose(0, 1)
    else:
        s["v"] = torch.empty_like(s["k"])
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def _rows(s):
    """Page and row in it of every token, as columns."""
    c = s["case"]
    seq, pos = s["seq"].long(), s["pos"].long()
    return s["table"][seq, pos // c["page"]].long()[:, None], (pos % c["page"])[:, None]


def _write(s):
    c = s["case"]
    page, row = _rows(s)
    head = torch.arange(c["hkv"], device="cuda")[None]
    for name in ("k", "v"):
        x = s[name].transpose(0, 1)  # [tokens, heads, dh]
        cache = s[name + "_cache"]
        if c["kind"] == "e4m3":
            x, s[name + "_scale"][page, head, row] = _quant(x.float())
            x, cache = x.view(torch.uint8), cache.view(torch.uint8)
        cache[page, head, row] = x
    return _cache(s)


def _picked(x, *index):
    """x[index]; indexing is not defined for every 8-bit float type, so it goes by the bytes."""
    return x.view(torch.uint8)[index].view(x.dtype) if x.element_size() == 1 else x[index]


def _cache(s):
    return {k: s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale") if s[k] is not None}


def _read(s):
    page, row = _rows(s)
    head = torch.arange(s["case"]["hkv"], device="cuda")[None]
    out = {}
    for name in ("k", "v"):
        x = _picked(s[name + "_cache"], page, head, row)
        if s[name + "_scale"] is not None:
            x = (x.float() * s[name + "_scale"][page, head, row][..., None]).bfloat16()
        out[name] = x.transpose(0, 1).contiguous()
    return out


def _gather(s, name):
    """Cached rows of all sequences in fp32, [sequences, heads, positions of the whole table, dh]."""
    at = s["table"].clamp(min=0).long()
    x = _picked(s[name + "_cache"], at).float()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][at][..., None]
    b, p, h, n, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, p * n, d)


def _decode(s):
    c = s["case"]
    t, g = c["new"], c["hq"] // c["hkv"]
    # rows of a key head: its query heads, each with the new tokens
    q = s["q"].float().view(c["hkv"], g, c["seqs"], t, c["dh"]).permute(2, 0, 1, 3, 4).reshape(c["seqs"], c["hkv"], g * t, c["dh"])
    k = _gather(s, "k")
    score = q @ k.transpose(2, 3) * (1 / math.sqrt(c["dh"]))
    seen = s["lens"].long()[:, None] - t + 1 + torch.arange(t, device="cuda")  # [sequences, new]
    hidden = torch.arange(k.shape[2], device="cuda") >= seen[:, None, None, :, None]  # [sequences, 1, 1, new, positions]
    score = score.view(c["seqs"], c["hkv"], g, t, -1).masked_fill(hidden, -math.inf).view(score.shape)
    del k
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ _gather(s, "v")) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).squeeze(-1)

    def back(x):  # [sequences, key heads, g * new, ...] -> [query heads, sequences * new, ...]
        x = x.view(c["seqs"], c["hkv"], g, t, *x.shape[3:]).transpose(0, 1).transpose(1, 2)
        return x.reshape(c["hq"], c["seqs"] * t, *x.shape[4:])
    return dict(o=back(o).bfloat16(), lse=back(lse))


def _own(s):
    import long_context_attention_upipe_gb300 as up

    c, keep = s["case"], s["keep"]
    if "cache" not in keep:  # a program sets its cache up once
        keep["cache"] = up.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    cache = keep["cache"]
    if c["op"] == "write":
        up.kv_write(cache, s["k"], s["v"], s["seq"], s["pos"], s["table"])
        return _cache(s)
    if c["op"] == "read":
        up.kv_read(cache, s["seq"], s["pos"], s["table"], s["k"], s["v"])
        return dict(k=s["k"], v=s["v"])
    if "ws" not in keep:
        keep["ws"] = torch.empty(up.decode_workspace_bytes(cache, c["seqs"], c["hq"], c["new"]), dtype=torch.uint8, device="cuda")
    up.decode(cache, s["q"], s["table"], s["lens"], s["o"], keep["ws"], lse=s["lse"])
    return dict(o=s["o"], lse=s["lse"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "write":
        return _write(state)
    if op == "read":
        return _read(state)
    return _decode(state)


def work(case):
    """Each input read once, each output written once."""
    c = case
    lens = _lens(c)
    row = 2 * c["dh"] if c["kind"] == "bf16" else c["dh"] + 4  # bytes of a cached row
    if c["op"] == "decode":
        new = c["seqs"] * c["new"] * c["hq"]
        seen = sum(max(0, n - c["new"] + 1 + t) for n in lens for t in range(c["new"]))
        return dict(bytes=2 * sum(lens) * c["hkv"] * row + new * (4 * c["dh"] + 4) + 4 * c["seqs"], flops=4 * seen * c["hq"] * c["dh"])
    t = sum(min(n, c["new"]) if c["new"] else n for n in lens)
    rows = 2 * t * c["hkv"]
    return dict(bytes=rows * (2 * c["dh"] + row) + 8 * t, flops=(3 if c["kind"] == "e4m3" else 0) * rows * c["dh"])


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------

def _exact_rows(s, name, b, n):
    """The first n cached rows of sequence b in 64 bits, [heads, n, dh]."""
    c = s["case"]
    pages = s["table"][b, : -(-n // c["page"])].long()
    x = _picked(s[name + "_cache"], pages).double().movedim(1, 0).flatten(1, 2)
    if c["kind"] == "e4m3":
        x = torch.einsum("hnd,hn->hnd", x, s[name + "_scale"][pages].double().movedim(1, 0).flatten(1, 2))
    return x[:, :n]


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "decode":
        t, g = c["new"], c["hq"] // c["hkv"]
        o = torch.zeros(c["hq"], c["seqs"] * t, c["dh"], dtype=torch.float64, device="cuda")
        lse = torch.full((c["hq"], c["seqs"] * t), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lens(c)):
            if n == 0:
                continue
            k, v = _exact_rows(s, "k", b, n), _exact_rows(s, "v", b, n)
            for j in range(max(0, t - n), t):
                see = n - t + 1 + j
                q = s["q"][:, b * t + j].double().view(c["hkv"], g, c["dh"])
                score = torch.einsum("hgd,hnd->hgn", q, k[:, :see]) / c["dh"] ** 0.5
                norm = torch.logsumexp(score, -1)
                weight = torch.exp(score - norm[..., None])
                lse[:, b * t + j] = norm.reshape(-1)
                o[:, b * t + j] = torch.einsum("hgn,hnd->hgd", weight, v[:, :see]).reshape(c["hq"], c["dh"])
        return dict(o=o, lse=lse)
    table = s["table"].tolist()
    if c["op"] == "write":
        out = {k: x.double() for k, x in _cache(s).items()}
        for name in ("k", "v"):
            i = 0
            for b, n in enumerate(_lens(c)):  # page by page: a run of tokens fills a run of rows
                p = max(0, n - c["new"]) if c["new"] else 0
                while p < n:
                    page, row = table[b][p // c["page"]], p % c["page"]
                    m = min(c["page"] - row, n - p)
                    x = s[name][:, i: i + m].double()
                    if c["kind"] == "e4m3":
                        top = torch.linalg.vector_norm(x, ord=math.inf, dim=-1)
                        scale = torch.where(top < TINY, torch.ones_like(top), top / E4M3_MAX)
                        out[name + "_scale"][page, :, row: row + m] = scale
                        x = torch.einsum("hnd,hn->hnd", x, 1.0 / scale)
                    out[name + "_cache"][page, :, row: row + m] = x
                    i, p = i + m, p + m
        return out
    return {name: torch.cat([_exact_rows(s, name, b, n) for b, n in enumerate(_lens(c))], 1) for name in ("k", "v")}
