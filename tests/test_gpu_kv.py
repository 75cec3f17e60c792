"""Paged cache of keys and values and the attention that reads it, against plain 64-bit arithmetic.

Tolerances count roundings; u = 2^-24 is fp32's relative half step, 2^-8 bf16's, 2^-11 fp16's.

Decode, for a query row with scores s_j = scale q . k_j and weights w_j = exp(s_j - lse):
  - q . k: D products of at most 8 x 8 significant bits, exact in fp32, and D additions that may truncate (2 u each): off by
    2 D u sum_i |q_i k_ij|.  A score takes at most four more fp32 roundings (the scale of a row, the softmax scale, log2 e, and
    the constants' own): in units of the exponent ds = |scale| (2 D + 8) u max_j sum_i |q_i k_ij|, and the difference to the running
    maximum is rounded once more, u times the largest |score| in units of log2: + 4 u max_j |s_j| in all.
  - a weight: exp2 within 2^-21 and the error of its exponent: relative ew = e^(2 ds) - 1 + 2^-20 (numerator and denominator alike).
    Rescaling to a new maximum multiplies by a number with the same relative error once; at most 64 times along a chain that
    changes its maximum (a power of two per change at the least, from scores that spread over less than 2^6 powers here).
  - the weight is rounded before it meets v: two bf16 numbers (2^-16) or one fp16 number (2^-11, with an e4m3 cache; below the
    smallest normal fp16 an absolute 2^-32 of the largest).
  - the sum over n keys: n products of which 16 at a time join a chain, 2 u each; at most n / 16 + 64 links + 32 of trees.
so o is within |o| 2^-8 + W (2 ew + r + (n / 16 + 96) 2 u) of its value with W = sum_j w_j |v_j|, r = 2^-16 or 2^-10, and lse
within ds + ew + (n / 16 + 96) 2 u + 4 u |lse|.
"""
import math

import pytest
import torch

import long_context_attention_upipe_gb300 as up

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
NAN = float("nan")


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


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def quant(x):
    """Codes and scales of rows by the library's quantiser of blocks of 128 columns (rows of 64 are padded with zeros)."""
    d = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, 128 - d)).reshape(-1, 128).contiguous()
    q, s = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(1, x.shape[0], device="cuda")
    if x.shape[0]:
        up.fp8_quantize(x, q, s)
    return bits(q)[:, :d], s[0]


LAYOUTS = ["heads", "tokens", "interleaved", "both", "layer"]


def pool(layout, pages, hkv, size, dh, dtype):
    """k, v [pages, hkv, size, dh] as parts of the memory that the layout names."""
    new = lambda *s: torch.zeros(*s, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device="cuda")  # noqa: E731
    if layout == "heads":
        k, v = new(pages, hkv, size, dh), new(pages, hkv, size, dh)
    elif layout == "tokens":
        k, v = (new(pages, size, hkv, dh).transpose(1, 2) for _ in range(2))
    elif layout == "interleaved":
        x = new(pages, 2, hkv, size, dh)
        k, v = x[:, 0], x[:, 1]
    elif layout == "both":
        x = new(pages, size, 2 * hkv, dh).transpose(1, 2)
        k, v = x[:, :hkv], x[:, hkv:]
    else:
        x = new(pages, 3, 2, hkv, size, dh)
        k, v = x[:, 1, 0], x[:, 1, 1]
    return (k.view(dtype), v.view(dtype)) if dtype == torch.float8_e4m3fn else (k, v)


def scales(layout, pages, hkv, size):
    if layout in ("tokens", "both"):
        return tuple(torch.zeros(pages, size, hkv, device="cuda").transpose(1, 2) for _ in range(2))
    return torch.zeros(pages, hkv, size, device="cuda"), torch.zeros(pages, hkv, size, device="cuda")


def make_cache(kind, layout="heads", pages=8, hkv=2, size=16, dh=128, fill=None):
    """A cache whose every place holds `fill` (a generator: random rows; "nan"; None: zeros)."""
    dtype = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    k, v = pool(layout, pages, hkv, size, dh, dtype)
    ks, vs = scales(layout, pages, hkv, size) if kind == "e4m3" else (None, None)
    for x, s in ((k, ks), (v, vs)):
        if fill == "nan":
            (bits(x) if kind == "e4m3" else x).copy_(torch.full((), 0x7f if kind == "e4m3" else NAN, device="cuda"))
            if s is not None:
                s.fill_(NAN)
        elif fill is not None:
            rows = randn(fill, pages, hkv, size, dh).bfloat16()
            if kind == "e4m3":
                q, sc = quant(rows)
                bits(x).copy_(q.view(rows.shape))
                s.copy_(sc.view(s.shape))
            else:
                x.copy_(rows)
    return up.KVCache(k, v, ks, vs)


def tensors(c):
    return [t for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]


def table_of(g, lens, size, pages, max_pages=None, unused=None):
    """Random pages for every sequence; the entries behind a sequence's last page are garbage."""
    held = [-(-max(0, n) // size) for n in lens]
    m = max(held + [1]) if max_pages is None else max_pages
    junk = torch.randint(-2 ** 31, 2 ** 31 - 1, (len(lens), m), generator=g, device="cuda").int()
    order = torch.randperm(pages, generator=g, device="cuda").int()
    i = 0
    for b, n in enumerate(held):
        junk[b, :n] = order[i: i + n]
        i += n
    assert i <= pages
    return junk


# ------------------------------------------------------------------------------------------------
# write and read
# ------------------------------------------------------------------------------------------------

def heads(g, layout, hkv, tokens, dh, scale=1.0):
    """bf16 [hkv, tokens, dh]: head by head, or a part of a projection's output."""
    if layout == "head":
        return (scale * randn(g, hkv, tokens, dh)).bfloat16()
    x = (scale * randn(g, tokens, 3 * hkv, dh)).bfloat16()
    return x[:, hkv: 2 * hkv].transpose(0, 1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("tokens,hkv,size,dh", [(1, 1, 16, 64), (7, 2, 16, 128), (70, 3, 48, 64), (333, 8, 32, 128)])
def test_write_and_read(kind, layout, tokens, hkv, size, dh):
    g = gen(tokens * 131 + hkv * 7 + dh)
    lens = [tokens // 3, 0, tokens - tokens // 3]
    pages = sum(-(-n // size) for n in lens) + 2
    c = make_cache(kind, layout, pages, hkv, size, dh, g)
    table = table_of(g, lens, size, pages)
    where = [(b, p) for b, n in enumerate(lens) for p in range(n)]
    where += [(-1, 0), (-5, 3), (0, -1), (3, 0), (2, 10 ** 6), (2 ** 31 - 1, 0)]     # padding, and places that do not exist
    where = torch.tensor(where, dtype=torch.int32, device="cuda")
    where = where[torch.randperm(len(where), generator=g, device="cuda")]
    seq, pos = where[:, 0].contiguous(), where[:, 1].contiguous()
    n = len(where)
    k, v = heads(g, "head", hkv, n, dh, 3.0), heads(g, "token", hkv, n, dh)
    want = [t.clone() for t in tensors(c)]
    good = [i for i, (b, p) in enumerate(where.tolist()) if 0 <= b < 3 and 0 <= p < lens[b]]
    for j, x in enumerate((k, v)):
        rows = x[:, good]
        page = torch.tensor([int(table[b, p // size]) for b, p in where[good].tolist()], device="cuda").long()
        row = pos[good].long() % size
        if kind == "e4m3":
            q, s = quant(rows)
            bits(want[j])[page, :, row] = q.view(hkv, -1, dh).transpose(0, 1)
            want[2 + j][page, :, row] = s.view(hkv, -1).t()
        else:
            want[j][page, :, row] = rows.transpose(0, 1)
    up.kv_write(c, k, v, seq, pos, table)
    for got, w in zip(tensors(c), want):
        assert torch.equal(bits(got), bits(w))
    # read: as they were in the cache, times their scales; padding stays, what does not exist is NaN
    out = torch.full((n, 2 * hkv, dh), 77.0, dtype=torch.bfloat16, device="cuda")
    ko, vo = out[:, :hkv].transpose(0, 1), out[:, hkv:].transpose(0, 1)
    up.kv_read(c, seq, pos, table, ko, vo)
    for j, (x, o) in enumerate(((k, ko), (v, vo))):
        rows = x[:, good]
        if kind == "e4m3":
            q, s = quant(rows)
            rows = (q.view(torch.float8_e4m3fn).float() * s[:, None]).bfloat16().view(hkv, -1, dh)
        assert torch.equal(o[:, good], rows)
        for i, (b, p) in enumerate(where.tolist()):
            if b < 0:
                assert bool((o[:, i] == 77).all())
            elif i not in good:
                assert bool(o[:, i].isnan().all())


@pytest.mark.parametrize("dh", [64, 128])
def test_write_keeps_nan_infinity_and_zero_in_their_rows(dh):
    g = gen(dh)
    c = make_cache("e4m3", pages=2, hkv=2, size=16, dh=dh)
    k, v = heads(g, "head", 2, 6, dh), heads(g, "head", 2, 6, dh)
    k[0, 1, 5], k[1, 2, 0], k[0, 3, 63] = NAN, float("inf"), -float("inf")
    v[1, 4] = 0
    v[0, 5] = 1e-38                     # below 2^-100: zeros with scale 1
    seq, pos = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.arange(6, device="cuda").int()
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    up.kv_write(c, k, v, seq, pos, table)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    up.kv_read(c, seq, pos, table, ko, vo)
    bad = torch.zeros(2, 6, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 2] = bad[0, 3] = True
    assert torch.equal(ko.isnan().all(-1), bad) and torch.equal(ko.isnan().any(-1), bad)
    assert bool((vo[1, 4] == 0).all()) and bool((vo[0, 5] == 0).all()) and float(c.v_scale[1, 0, 5]) == 1.0
    assert bool(vo.isfinite().all())


def test_write_codes_of_every_pair_of_significands():
    """Rows whose largest magnitude and elements take every bf16 significand: the codes are those of the exact quotient."""
    top = torch.arange(128, 256, device="cuda").float()
    x = torch.arange(128, 256, device="cuda").float()
    for shift in (0, 1, 2, 5, 8, 12, 16):
        for size in (2.0 ** -7, 2.0 ** 40, 2.0 ** 70, 2.0 ** -90):
            rows = torch.minimum(x[None] / 2 ** shift, top[:, None]).repeat(1, 1)
            rows[:, 0] = top
            rows = (rows * size * torch.where(torch.arange(128, device="cuda") % 2 == 1, -1, 1)).bfloat16()
            c = make_cache("e4m3", pages=8, hkv=1, size=16, dh=128)
            pos, table = torch.arange(128, device="cuda").int(), torch.arange(8, device="cuda").int()[None].contiguous()
            up.kv_write(c, rows[None], rows[None], torch.zeros_like(pos), pos, table)
            s = rows.float().abs().amax(1) * torch.tensor(1 / 448, dtype=torch.float32, device="cuda")
            want = (rows.double() / s.double()[:, None]).float().to(torch.float8_e4m3fn)
            assert torch.equal(bits(c.k).view(128, 128), bits(want)) and torch.equal(bits(c.v), bits(c.k))
            assert torch.equal(c.k_scale.view(-1), s) and torch.equal(c.v_scale, c.k_scale)


def test_no_tokens():
    c = make_cache("bf16")
    e, i = torch.empty(2, 0, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    n = up.launch_count()
    up.kv_write(c, e, e, i, i, torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    up.kv_read(c, i, i, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), e, e.clone())
    assert up.launch_count() == n


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_pages_past_32_bit_offsets(kind):
    """A cache of more than 2^32 elements for keys and values each; the pages at its end."""
    hkv, size, dh = 8, 64, 128
    pages = 2 ** 32 // (hkv * size * dh) + 3
    dtype = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    x = torch.empty(2, pages, hkv, size, dh, dtype=torch.uint8 if kind == "e4m3" else dtype, device="cuda").view(dtype)
    s = [torch.empty(pages, hkv, size, device="cuda") for _ in range(2)] if kind == "e4m3" else [None, None]
    c = up.KVCache(x[0], x[1], *s)
    g = gen(5)
    n = 100
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    k, v, pos = heads(g, "head", hkv, n, dh), heads(g, "head", hkv, n, dh), torch.arange(n, device="cuda").int()
    up.kv_write(c, k, v, torch.zeros_like(pos), pos, table)
    q = randn(g, 16, 1, dh).bfloat16()
    check_decode(c, q, table, [n])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    up.kv_read(c, torch.zeros_like(pos), pos, table, ko, vo)
    if kind == "bf16":
        assert torch.equal(ko, k) and torch.equal(vo, v)
    else:
        tol = k.double().abs() * (2.0 ** -4 + 2.0 ** -7) + k.abs().amax(-1, keepdim=True).double() / 448 * 2.0 ** -9
        assert bool(((ko.double() - k.double()).abs() <= tol).all())


# ------------------------------------------------------------------------------------------------
# decode
# ------------------------------------------------------------------------------------------------

def cached(c, name, table, b, n):
    """The first n rows of sequence b in 64 bits [hkv, n, dh]."""
    x, s = getattr(c, name), getattr(c, name + "_scale")
    pages = table[b, : -(-n // c.page_size)].long()
    rows = bits(x)[pages].view(x.dtype).double()
    if s is not None:
        rows = rows * s[pages].double()[..., None]
    return rows.transpose(0, 1).flatten(1, 2)[:, :n]


def run_decode(c, q, table, lens, scale=0.0, q_len=1, o=None, lse=True, ws=None):
    o = torch.full_like(q, 55.0) if o is None else o
    e = torch.full(q.shape[:2], 55.0, device="cuda") if lse else None
    if ws is None:  # nothing is expected of what lies in it
        ws = torch.full((up.decode_workspace_bytes(c, table.shape[0], q.shape[0], q_len),), 0xff, dtype=torch.uint8, device="cuda")
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda") if isinstance(lens, list) else lens
    up.decode(c, q, table, lens, o, ws, lse=e, scale=scale)
    return o, e


def check_decode(c, q, table, lens, scale=0.0, q_len=1, **kw):
    o, lse = run_decode(c, q, table, lens, scale, q_len, **kw)
    hq, dh = q.shape[0], q.shape[2]
    grp = hq // c.n_kv_heads
    sc = scale or dh ** -0.5
    assert bool(o.isfinite().all())
    for b, n in enumerate(lens):
        n = max(0, n)
        if n:
            k, v = cached(c, "k", table, b, n), cached(c, "v", table, b, n)
        for t in range(q_len):
            i, see = b * q_len + t, n - q_len + 1 + t
            if see <= 0:
                assert bool((o[:, i] == 0).all()) and bool((lse[:, i] == -math.inf).all())
                continue
            x = q[:, i].double().view(c.n_kv_heads, grp, dh)
            s = x @ k[:, :see].transpose(1, 2) * sc
            want = torch.logsumexp(s, -1, keepdim=True)
            w = torch.exp(s - want)
            ref, size = w @ v[:, :see], w @ v[:, :see].abs()
            mass = (x.abs() @ k[:, :see].abs().transpose(1, 2)).amax(-1, keepdim=True)
            ds = abs(sc) * (2 * dh + 8) * U * mass + 4 * U * s.abs().amax(-1, keepdim=True)
            ew = torch.expm1(2 * ds) + 65 * 2.0 ** -20
            chain = (see / 16 + 96) * 2 * U
            r = 2.0 ** -10 if c.k_scale is not None else 2.0 ** -16
            tol = ref.abs() * BF + size * (2 * ew + r + chain) + 2.0 ** -130
            err = (o[:, i].double().view(ref.shape) - ref).abs()
            assert bool((err <= tol).all()), f"sequence {b} token {t}: {float((err - tol).max())} over"
            err = (lse[:, i].double().view(want.shape[:2]) - want[..., 0]).abs()
            assert bool((err <= (ds + ew + chain)[..., 0] + 4 * U * want[..., 0].abs()).all()), f"lse of sequence {b} token {t}"
    return o, lse


def setup(kind, lens, hq, hkv, dh, size, q_len=1, layout="heads", seed=0, spread=2.0, extra=3):
    """A cache whose unused places and pages are NaN, its table, and queries."""
    g = gen(seed * 977 + len(lens) * 31 + hq + dh)
    pages = sum(-(-max(0, n) // size) for n in lens) + extra
    c = make_cache(kind, layout, pages, hkv, size, dh, "nan")
    table = table_of(g, lens, size, pages)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        pos = torch.arange(n, device="cuda").int()
        k, v = heads(g, "head", hkv, n, dh), heads(g, "head", hkv, n, dh)
        up.kv_write(c, k, v + 0.5, torch.full_like(pos, b), pos, table)
    return c, table, (spread * randn(g, hq, len(lens) * q_len, dh)).bfloat16()


KINDS = ["bf16", "e4m3"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (8, 1), (6, 2), (10, 2), (32, 2), (34, 2)])
def test_decode_lengths(kind, dh, hq, hkv):
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 127, 128, 129, 500, -3, 0]
    c, table, q = setup(kind, lens, hq, hkv, dh, 32)
    check_decode(c, q, table, lens)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_len", [2, 3, 4, 8, 16])
@pytest.mark.parametrize("hq,hkv,dh", [(4, 4, 64), (8, 2, 128), (10, 2, 64)])
def test_decode_several_tokens(kind, q_len, hq, hkv, dh):
    lens = [0, 1, q_len - 1, q_len, q_len + 1, 16, 17, 20, 129, 300]
    c, table, q = setup(kind, lens, hq, hkv, dh, 16, q_len)
    check_decode(c, q, table, lens, q_len=q_len)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("size", [16, 48, 128])
def test_decode_layouts_and_pages(kind, layout, size):
    lens = [200, 3, size, size + 1, 2 * size - 1]
    c, table, q = setup(kind, lens, 8, 2, 128, size, layout=layout)
    o, lse = check_decode(c, q, table, lens)
    # a slice of a wider table, queries and outputs as parts of token-major tensors
    wide = torch.full((len(lens), table.shape[1] + 7), -7, dtype=torch.int32, device="cuda")
    wide[:, 3: 3 + table.shape[1]] = table
    both = torch.zeros(len(lens), 24, 128, dtype=torch.bfloat16, device="cuda")
    both[:, 4:12] = q.transpose(0, 1)
    o2, lse2 = run_decode(c, both[:, 4:12].transpose(0, 1), wide[:, 3: 3 + table.shape[1]], lens, o=both[:, 12:20].transpose(0, 1))
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    assert bool((both[:, :4] == 0).all()) and bool((both[:, 20:] == 0).all()) and torch.equal(both[:, 4:12].transpose(0, 1), q)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,hq,hkv,dh,size", [
    ([70001], 4, 1, 128, 128), ([20011], 8, 8, 64, 64), ([5003, 12, 0, 9001, 777], 40, 8, 128, 32)])
def test_decode_long(kind, lens, hq, hkv, dh, size):
    c, table, q = setup(kind, lens, hq, hkv, dh, size)
    check_decode(c, q, table, lens)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_many_sequences(kind):
    lens = [(i * 37) % 90 if i % 5 else 0 for i in range(3001)]
    c, table, q = setup_many(kind, lens, 4, 2, 64, 16)
    check_decode(c, q, table, lens)


def setup_many(kind, lens, hq, hkv, dh, size):
    """As setup, with all sequences written in one call."""
    g = gen(len(lens))
    pages = sum(-(-n // size) for n in lens) + 1
    c = make_cache(kind, "heads", pages, hkv, size, dh, "nan")
    table = table_of(g, lens, size, pages)
    seq = torch.tensor([b for b, n in enumerate(lens) for _ in range(n)], dtype=torch.int32, device="cuda")
    pos = torch.tensor([p for n in lens for p in range(n)], dtype=torch.int32, device="cuda")
    up.kv_write(c, heads(g, "head", hkv, len(pos), dh), heads(g, "token", hkv, len(pos), dh), seq, pos, table)
    return c, table, (2 * randn(g, hq, len(lens), dh)).bfloat16()


@pytest.mark.parametrize("kind", KINDS)
def test_decode_many_rows(kind):
    lens = [3, 40, 100]
    c, table, q = setup(kind, lens, 256, 2, 64, 16, 16)
    check_decode(c, q, table, lens, q_len=16)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_decode_flat_and_peaked_scores(kind, spread):
    lens = [700, 33]
    c, table, q = setup(kind, lens, 8, 2, 128, 64, spread=spread)
    check_decode(c, q, table, lens)
    check_decode(c, q, table, lens, scale=-0.03)


def test_decode_scales_of_any_size():
    """Rows whose largest magnitudes differ by many powers of two, in an 8-bit cache."""
    g = gen(11)
    n, hkv, dh = 300, 2, 128
    c = make_cache("e4m3", pages=20, hkv=hkv, size=16, dh=dh)
    table, pos = table_of(g, [n], 16, 20), torch.arange(n, device="cuda").int()
    size = torch.exp2(torch.randint(-60, 40, (hkv, n, 1), generator=g, device="cuda").float())
    for v in (randn(g, hkv, n, dh) * size, randn(g, hkv, n, dh) * 2.0 ** 60, randn(g, hkv, n, dh) * 2.0 ** -60):
        up.kv_write(c, randn(g, hkv, n, dh).bfloat16(), v.bfloat16(), torch.zeros_like(pos), pos, table)
        check_decode(c, randn(g, 8, 1, dh).bfloat16(), table, [n])
    up.kv_write(c, (randn(g, hkv, n, dh) * 2.0 ** -40).bfloat16(), randn(g, hkv, n, dh).bfloat16(), torch.zeros_like(pos), pos, table)
    check_decode(c, (randn(g, 8, 1, dh) * 2.0 ** 40).bfloat16(), table, [n])
    check_decode(c, (randn(g, 8, 1, dh) * 2.0 ** -100).bfloat16(), table, [n])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("what", [NAN, float("inf"), -float("inf")])
def test_decode_keeps_what_is_masked_out(kind, what):
    """The newest token's key and value are not finite: the queries before it do not see them."""
    q_len, lens = 4, [100, 4, 37]
    c, table, q = setup(kind, lens, 8, 2, 128, 16, q_len)
    clean, clean_lse = check_decode(c, q, table, lens, q_len=q_len)
    last = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    k, v = heads(gen(3), "head", 2, 3, 128), heads(gen(4), "head", 2, 3, 128)
    k[0, :, 7], v[:, :, 100] = what, what
    up.kv_write(c, k, v, torch.arange(3, device="cuda").int(), last, table)
    o, lse = run_decode(c, q, table, lens, q_len=q_len)
    seen = torch.arange(12, device="cuda") % q_len == q_len - 1
    assert torch.equal(o[:, ~seen].isfinite(), torch.ones_like(o[:, ~seen], dtype=torch.bool))
    # as if the last token were not there: the same values but for the order of sums
    err = (o[:, ~seen].double() - clean[:, ~seen].double()).abs()
    assert bool((err <= clean[:, ~seen].double().abs() * 2 * BF + 2.0 ** -9).all())
    assert bool(((lse - clean_lse)[:, ~seen].abs() <= 2.0 ** -16).all())
    assert not bool(o[4:, seen, 100].isfinite().any()) and (kind == "e4m3" or bool(o[4:, seen, :100].isfinite().all()))


@pytest.mark.parametrize("what", [NAN, float("inf"), -float("inf")])
def test_decode_infinite_values_and_keys_that_are_seen(what):
    lens = [90, 90]
    c, table, q = setup("bf16", lens, 4, 1, 64, 16)
    clean, _ = run_decode(c, q, table, lens)
    page, row = int(table[0, 2]), 5
    c.v[page, 0, row, 9] = what
    o, lse = run_decode(c, q, table, lens)
    assert torch.equal(o[:, 0, 9].isnan(), torch.full_like(o[:, 0, 9], what != what, dtype=torch.bool))
    assert what != what or bool((o[:, 0, 9] == what).all())
    rest = torch.arange(64, device="cuda") != 9
    err = (o[:, 0, rest].double() - clean[:, 0, rest].double()).abs()
    assert bool((err <= clean[:, 0, rest].double().abs() * 2 * BF + 2.0 ** -9).all())
    assert torch.equal(o[:, 1], clean[:, 1]) and bool(lse.isfinite().all())
    c.v[page, 0, row, 9] = 0
    c.k[page, 0, row, 9] = what         # every score of the row is then NaN or +-infinity
    o, lse = run_decode(c, q, table, lens)
    s = q[:, 0, 9].double() * what
    nan = ~(s == -math.inf)              # a key at -infinity has no weight; +infinity and NaN leave nothing defined
    assert bool(o[nan, 0].isnan().all()) and bool(o[~nan, 0].isfinite().all()) and torch.equal(o[:, 1], clean[:, 1])


@pytest.mark.parametrize("kind", KINDS)
def test_decode_nan_queries_stay_in_their_rows(kind):
    lens = [50, 60]
    c, table, q = setup(kind, lens, 8, 2, 128, 16, 2)
    clean, lse = run_decode(c, q, table, lens, q_len=2)
    q[5, 2, 0] = NAN
    o, lse2 = run_decode(c, q, table, lens, q_len=2)
    assert bool(o[5, 2].isnan().all()) and bool(lse2[5, 2].isnan())
    o[5, 2], lse2[5, 2] = clean[5, 2], lse[5, 2]
    assert torch.equal(o, clean) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [-1, 1 << 20, -2 ** 31])
def test_decode_of_missing_pages_is_nan(kind, page):
    lens = [100, 100, 100]
    c, table, q = setup(kind, lens, 8, 2, 64, 16, 4)
    clean, _ = run_decode(c, q, table, lens, q_len=4)
    broken = table.clone()
    broken[1, 2] = page                  # in the middle of sequence 1
    broken[2, 6] = page                  # positions 96 to 99 of sequence 2: its first query sees 97 keys
    o, lse = run_decode(c, q, broken, lens, q_len=4)
    assert torch.equal(o[:, :4], clean[:, :4])
    assert bool(o[:, 4:].isnan().all()) and bool(lse[:, 4:].isnan().all())
    # lengths past the table
    o, lse = run_decode(c, q, table, [100, 2 ** 31 - 1, 113], q_len=4)
    assert torch.equal(o[:, :4], clean[:, :4]) and bool(o[:, 4:].isnan().all()) and bool(lse[:, 4:].isnan().all())
    # a table without columns: only empty sequences have no need of it
    o, lse = run_decode(c, q, table[:, :0], [0, 5, -1], q_len=4)
    assert bool((o[:, :4] == 0).all()) and bool((o[:, 8:] == 0).all()) and bool(o[:, 7].isnan().all())


@pytest.mark.parametrize("kind", KINDS)
def test_decode_is_repeatable_and_needs_no_lse(kind):
    lens = [4000, 17, 900]
    c, table, q = setup(kind, lens, 32, 8, 128, 64)
    o, lse = run_decode(c, q, table, lens)
    for _ in range(3):
        o2, lse2 = run_decode(c, q, table, lens)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o2, _ = run_decode(c, q, table, lens, lse=False)
    assert torch.equal(o, o2)


def test_decode_in_graphs_that_share_a_workspace():
    lens = [300, 0, 77]
    c, table, q = setup("e4m3", [2000, 2000, 2000], 8, 2, 128, 64)
    c2, table2, q2 = setup("bf16", [500, 500], 16, 2, 64, 16)
    ln, ln2 = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor([500, 1], dtype=torch.int32, device="cuda")
    ws = torch.full((max(up.decode_workspace_bytes(c, 3, 8), up.decode_workspace_bytes(c2, 2, 16)),), 0xff, dtype=torch.uint8, device="cuda")
    o, o2 = torch.empty_like(q), torch.empty_like(q2)
    lse, lse2 = torch.empty(8, 3, device="cuda"), torch.empty(16, 2, device="cuda")
    torch.cuda.synchronize()
    graphs = []
    for args in ((c, q, table, ln, o, lse), (c2, q2, table2, ln2, o2, lse2)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            up.decode(args[0], args[1], args[2], args[3], args[4], ws, lse=args[5])
        graphs.append(gr)
    for lens in ([300, 0, 77], [2000, 1999, 1], [0, 0, 0], [1, 1600, 16]):
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        for gr in graphs + graphs:
            gr.replay()
        torch.cuda.synchronize()
        want, wl = check_decode(c, q, table, lens)
        assert torch.equal(o, want) and torch.equal(lse, wl)
        want, wl = check_decode(c2, q2, table2, [500, 1])
        assert torch.equal(o2, want) and torch.equal(lse2, wl)


def test_decode_on_two_streams_at_once():
    lens = [3000, 500]
    sets = [setup(kind, lens, 8, 2, 128, 64) for kind in KINDS]
    want = [run_decode(s[0], s[2], s[1], lens) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = [(torch.empty_like(s[2]), torch.empty(8, 2, device="cuda"),
            torch.empty(up.decode_workspace_bytes(s[0], 2, 8), dtype=torch.uint8, device="cuda")) for s in sets]
    torch.cuda.synchronize()
    for _ in range(50):
        for s, st, (o, lse, ws) in zip(sets, streams, out):
            up.decode(s[0], s[2], s[1], ln, o, ws, lse=lse, stream=st)
    torch.cuda.synchronize()
    for (o, lse, _), (wo, wl) in zip(out, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


# ------------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
def test_generation_step_by_step(kind):
    """A prompt and then tokens one by one: rotation, write, decode; against the attention core over the whole sequence, and
    the rows read back against what was written."""
    S, n0, hq, hkv, dh, size = 200, 173, 8, 2, 128, 16
    g = gen(21)
    qkv = randn(g, S, hq + 2 * hkv, dh).bfloat16()
    rot = up.make_rope_desc(dh, [10000.0 ** (-j / 64) for j in range(64)])
    pages = -(-S // size)
    c = make_cache(kind, "interleaved", pages, hkv, size, dh, "nan")
    table = torch.randperm(pages, generator=g, device="cuda").int()[None].contiguous()
    q, k = torch.empty(hq, S, dh, dtype=torch.bfloat16, device="cuda"), torch.empty(hkv, S, dh, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(hq, S, device="cuda")
    ws = torch.empty(up.decode_workspace_bytes(c, 1, hq), dtype=torch.uint8, device="cuda")
    at = 0
    for n in [n0] + [1] * (S - n0):
        x = qkv[at: at + n].transpose(0, 1)
        pos = torch.arange(at, at + n, device="cuda").int()
        qs, ks = q[:, at: at + n], k[:, at: at + n]
        up.rope(rot, x[:hq], x[hq: hq + hkv], pos[None], qs, ks)
        up.kv_write(c, ks, x[hq + hkv:], torch.zeros_like(pos), pos, table)
        at += n
        if n == 1:
            ot, lt = torch.empty(hq, 1, dh, dtype=torch.bfloat16, device="cuda"), torch.empty(hq, 1, device="cuda")
            up.decode(c, qs, table, torch.tensor([at], dtype=torch.int32, device="cuda"), ot, ws, lse=lt)
            o[:, at - 1: at], lse[:, at - 1: at] = ot, lt
    kr, vr = torch.empty_like(k), torch.empty_like(k)
    pos = torch.arange(S, device="cuda").int()
    up.kv_read(c, torch.zeros_like(pos), pos, table, kr, vr)
    if kind == "bf16":
        assert torch.equal(kr, k) and torch.equal(vr, qkv[:, hq + hkv:].transpose(0, 1))
    # the attention core over the rows that the cache holds
    desc = up.make_desc(S, hq * dh, hq, hkv, dh)
    tab = torch.empty(up.tile_table_bytes(desc), dtype=torch.uint8, device="cuda")
    up.build_tile_table(desc, None, tab)
    oc, lc = torch.empty_like(q), torch.empty_like(lse)
    up.core_fwd(desc, q, kr, vr, None, tab, oc, lc)
    new = slice(n0, S)
    # off by 2^-8 of sum w |v| (the core rounds its weights to bf16) and 2^-8 |o| for either's output, 2^-12 for the rest; with e4m3
    # the core reads code * scale rounded to bf16, which moves a score by 2^-8 scale sum |q k| at most, and v by 2^-8 of itself
    ds = 0.0
    if kind == "e4m3":
        ds = float((q[:, new].double().abs().view(hkv, -1, dh) @ kr.double().abs().transpose(1, 2)).max()) * dh ** -0.5 * BF
    tol = float(vr.double().abs().max()) * (4 * BF + math.expm1(2 * ds) + 2.0 ** -12)
    assert float((o[:, new].double() - oc[:, new].double()).abs().max()) <= tol
    assert float((lse[:, new] - lc[:, new]).abs().max()) <= ds + 2.0 ** -12 * (1 + float(lse[:, new].abs().max()))


# ------------------------------------------------------------------------------------------------
# every way through the decode kernels: tables with room for far more keys than there are (the division of work goes by the
# device's lengths, the choice of kernels by the table's room), batches around 32 and 64 sequences, very many sequences
# ------------------------------------------------------------------------------------------------

def widened(table, columns, g):
    """The table with `columns` more entries of garbage in every row."""
    junk = torch.randint(-2 ** 31, 2 ** 31 - 1, (table.shape[0], columns), generator=g, device="cuda").int()
    return torch.cat([table, junk], 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dh,hq,hkv,q_len", [(64, 4, 2, 1), (128, 8, 1, 1), (128, 24, 3, 1), (128, 6, 3, 4), (64, 40, 2, 1), (64, 16, 4, 3)])
@pytest.mark.parametrize("columns", [100, 100000])
def test_decode_in_wide_tables(kind, dh, hq, hkv, q_len, columns):
    lens = [0, 1, 15, 16, 17, 40, 0, 127, 128, 129, 700, 2, 333]
    c, table, q = setup(kind, lens, hq, hkv, dh, 16, q_len)
    check_decode(c, q, widened(table, columns, gen(1)), lens, q_len=q_len)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [31, 32, 33, 63, 64, 65, 97, 256, 257])
def test_decode_batches(kind, n):
    g = torch.Generator()
    g.manual_seed(n)
    lens = [int(x) if x < 150 else 0 for x in torch.randint(0, 200, (n,), generator=g)]
    c, table, q = setup_many(kind, lens, 8, 2, 64, 16)
    check_decode(c, q, table, lens)
    check_decode(c, q, widened(table, 3000, gen(2)), lens)


def test_decode_65536_sequences():
    """Each of one key: o is its value, lse its score; every other sequence empty."""
    n, pages = 65536, 37
    c = make_cache("bf16", pages=pages, hkv=1, size=16, dh=64, fill=gen(9))
    b = torch.arange(n, device="cuda")
    table = (b % pages).int()[:, None].contiguous()
    lens = (b % 2).int()
    q = randn(gen(10), 2, n, 64).bfloat16()
    o, lse = run_decode(c, q, table, lens)
    assert bool((o[:, ::2] == 0).all()) and bool((lse[:, ::2] == -math.inf).all())
    rows = (b % pages)[1::2]
    assert torch.equal(o[:, 1::2], c.v[rows, 0, 0][None].expand(2, -1, -1))
    s = (q[:, 1::2].double() * c.k[rows, 0, 0].double()).sum(-1) / 8
    mass = (q[:, 1::2].double() * c.k[rows, 0, 0].double()).abs().sum(-1) / 8
    # (2 D + 8) roundings of the products' sum, 4 of the score in units of log2 and back, the logarithm's of l = 1
    assert bool(((lse[:, 1::2].double() - s).abs() <= mass * (2 * 64 + 8) * U + s.abs() * 8 * U + 2.0 ** -20).all())
    with pytest.raises(up.UpipeError):
        run_decode(c, torch.zeros(2, n + 1, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(n + 1, 1, dtype=torch.int32, device="cuda"),
                   [0] * (n + 1), ws=torch.empty(1 << 24, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("kind", KINDS)
def test_decode_whose_waits_run_out_gives_nan_or_the_right_values(kind):
    lens = [3000, 40, 900]
    c, table, q = setup(kind, lens, 8, 2, 128, 64)
    want, wl = run_decode(c, q, table, lens)
    try:
        up.set_wait_limit_ns(1)
        for _ in range(20):
            o, lse = run_decode(c, q, table, lens)
            torch.cuda.synchronize()
            lost = o.isnan().any(-1)
            assert torch.equal(o.isnan().all(-1), lost) and torch.equal(lse.isnan(), lost)
            assert torch.equal(o[~lost], want[~lost]) and torch.equal(lse[~lost], wl[~lost])
    finally:
        up.set_wait_limit_ns(0)
    o, lse = run_decode(c, q, table, lens)
    assert torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind", KINDS)
def test_write_and_decode_captured_and_replayed(kind):
    """A decode step as a graph: new tokens, positions, lengths and table are the device's."""
    hq, hkv, dh, n = 8, 2, 128, 5
    g = gen(33)
    lens = [30, 0, 63, 100, 16]
    c, table, q = setup(kind, [n + 8 for n in lens], hq, hkv, dh, 16)
    k, v = heads(g, "head", hkv, n, dh), heads(g, "token", hkv, n, dh)
    seq, pos = torch.arange(n, device="cuda").int(), torch.zeros(n, dtype=torch.int32, device="cuda")
    ln = torch.zeros(n, dtype=torch.int32, device="cuda")
    ws = torch.full((up.decode_workspace_bytes(c, n, hq),), 0xff, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(hq, n, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        up.kv_write(c, k, v, seq, pos, table)
        up.decode(c, q, table, ln, o, ws, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        up.kv_write(c, k, v, seq, pos, table)
        up.decode(c, q, table, ln, o, ws, lse=lse)
    for step in range(4):
        now = [x + step + 1 if b != 1 or step > 1 else 0 for b, x in enumerate(lens)]
        k.copy_(heads(g, "head", hkv, n, dh))
        v.copy_(heads(g, "token", hkv, n, dh))
        pos.copy_(torch.tensor([x - 1 for x in now], dtype=torch.int32))
        seq.copy_(torch.tensor([b if x > 0 else -1 for b, x in enumerate(now)], dtype=torch.int32))
        ln.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for b, x in enumerate(now):
            if x:
                rows = cached(c, "k", table, b, x)[:, -1]
                assert kind == "e4m3" or torch.equal(rows, k[:, b].double())
        want, wl = check_decode(c, q, table, now)
        assert torch.equal(o, want) and torch.equal(lse, wl)


def test_entry_points_on_a_stream_of_their_own():
    c, table, q = setup("e4m3", [200, 300], 8, 2, 128, 64)
    want, wl = run_decode(c, q, table, [200, 300])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pos, seq = torch.arange(200, device="cuda").int(), torch.zeros(200, dtype=torch.int32, device="cuda")
    k, v = torch.empty(2, 200, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 200, 128, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(8, 2, device="cuda")
    ws = torch.empty(up.decode_workspace_bytes(c, 2, 8), dtype=torch.uint8, device="cuda")
    ln = torch.tensor([200, 300], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    up.kv_read(c, seq, pos, table, k, v, stream=st)
    up.kv_write(c, k, v, seq, pos, table, stream=st)       # what was read is written back: the same codes, scales within a rounding
    up.kv_read(c, seq, pos, table, k, v, stream=st)
    up.decode(c, q, table, ln, o, ws, lse=lse, stream=st)
    st.synchronize()
    assert torch.equal(o[:, 1], want[:, 1]) and torch.equal(lse[:, 1], wl[:, 1])
    ref = cached(c, "k", table, 0, 200)
    assert bool(((k.double() - ref).abs() <= ref.abs() * BF + 2.0 ** -133).all())


def test_binding_refuses_on_the_gpu():
    c, table, q = setup("bf16", [20, 30], 8, 2, 128, 16)
    o, ws = torch.empty_like(q), torch.empty(up.decode_workspace_bytes(c, 2, 8), dtype=torch.uint8, device="cuda")
    ln = torch.tensor([20, 30], dtype=torch.int32, device="cuda")
    k = torch.zeros(2, 3, 128, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    n = up.launch_count()
    for call in (lambda: up.decode(c, q.float(), table, ln, o, ws), lambda: up.decode(c, q, table.long(), ln, o, ws),
                 lambda: up.decode(c, q, table, ln.long(), o, ws), lambda: up.decode(c, q, table, ln[:1], o, ws),
                 lambda: up.decode(c, q[:, :1], table, ln, o[:, :1], ws), lambda: up.decode(c, q, table, ln, o[:4], ws),
                 lambda: up.decode(c, q[..., :64], table, ln, o[..., :64], ws), lambda: up.decode(c, q, table[0], ln, o, ws),
                 lambda: up.decode(c, q, table.t(), ln, o, ws), lambda: up.decode(c, q, table, ln.cpu(), o, ws),
                 lambda: up.decode(c, q, table, ln, o, ws.int()), lambda: up.decode(c, q, table, ln, o, ws, lse=torch.empty(2, 8, device="cuda")),
                 lambda: up.decode(c, q[0], table, ln, o[0], ws), lambda: up.decode(c, q.transpose(1, 2), table, ln, o, ws),
                 lambda: up.kv_write(c, k[:1], k, i, i, table), lambda: up.kv_write(c, k, k.float(), i, i, table),
                 lambda: up.kv_write(c, k, k, i[:2], i, table), lambda: up.kv_write(c, k, k, i.long(), i, table),
                 lambda: up.kv_write(c, k, k, i, i, table.cpu()), lambda: up.kv_write(c, k, k, i[None], i, table),
                 lambda: up.kv_read(c, i, i, table, k, k.cpu()), lambda: up.KVCache(c.k, c.v.transpose(1, 2)),
                 lambda: up.KVCache(c.k, c.v, torch.zeros(1, device="cuda"), None), lambda: up.KVCache(c.k.transpose(2, 3), c.v.transpose(2, 3))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: up.decode(c, q, table, ln, q, ws), lambda: up.decode(c, q, table, ln, o, ws[:16]), lambda: up.kv_read(c, i, i, table, k, k),
                 lambda: up.decode(c, q, table, ln, o, ws, scale=math.nan), lambda: up.kv_write(c, c.k[0, :, :3], k, i, i, table)):
        with pytest.raises(up.UpipeError):
            call()
    assert up.launch_count() == n


@pytest.mark.parametrize("kind", KINDS)
def test_decode_of_the_longest_sequence(kind):
    """2^31 - 1 keys: one page of 2^20 tokens under every entry of the table.

    A lane's part of l is a chain of some 2 x 2^27 / (152 x 8) additions, each within 2^-24 of the sum so far, O's sums chains of half
    as many that may truncate (2^-23); W / |o| is small here, so the tolerance is in units of W."""
    size, dh, n = 1 << 20, 64, 2 ** 31 - 1
    g = gen(77)
    c = make_cache(kind, pages=1, hkv=1, size=size, dh=dh, fill=g)
    table = torch.zeros(1, 2048, dtype=torch.int32, device="cuda")
    q = randn(g, 2, 1, dh).bfloat16()
    o, lse = run_decode(c, q, table, [n])
    k, v = cached(c, "k", table, 0, size)[0], cached(c, "v", table, 0, size)[0]
    s = q[:, 0].double() @ k.t() / 8
    top = s.amax(1, keepdim=True)
    w = torch.exp(s - top)
    total = 2048 * w.sum(1) - w[:, -1]
    want = (2048 * (w @ v) - w[:, -1:] * v[-1:]) / total[:, None]
    size_ = (2048 * (w @ v.abs())) / total[:, None]
    chain = 2 * 2 ** 27 / (152 * 8) * 2.0 ** -24
    assert bool(((o[:, 0].double() - want).abs() <= want.abs() * BF + size_ * 2 * chain).all())
    assert bool(((lse[:, 0].double() - top[:, 0] - torch.log(total)).abs() <= chain + 2.0 ** -16).all())
    # one key more than the table holds, and the table's last key
    o, lse = run_decode(c, q, table[:, :2047], [2047 * size + 1])
    assert bool(o.isnan().all()) and bool(lse.isnan().all())
