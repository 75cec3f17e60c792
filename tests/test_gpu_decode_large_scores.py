"""Decode where scores are far larger than a model's, but finite: one key has all of a row's weight, and the row's o is its value.

The scores of the other keys are 60 or more below (e^-60 of the weight, 2^-20 in all for lse), so o is off by its own rounding and the
weight's alone (r = 2^-16 or 2^-10, and exp2's: numerator and denominator have the same), whatever the size of the scores, and by what the
others bring, whose values may be 2^40 larger: at most twice their weights' sum of |v| (a weight is off by less than a factor of two
where the gap is not in the thousands); lse by the roundings of a score, 2 D + 8 of sum_i |q_i k_i| and four of its own."""
import math

import pytest
import torch

import long_context_attention_upipe_gb300 as up
from test_gpu_kv import BF, U, cached, gen, make_cache, randn, run_decode, table_of, widened

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


FORMS = {  # lengths, query heads, key heads, head_dim, page, q_len, columns that the table has beside: each way through the kernels
    "cta": ([1, 17, 200], 4, 1, 128, 16, 1, 0), "cluster": ([2000], 4, 1, 128, 64, 1, 0),
    "whole": ([(i * 37) % 300 for i in range(200)], 2, 1, 64, 16, 1, 0), "line": ([5003, 12, 0, 777], 8, 2, 128, 32, 1, 0),
    "warps": ([6000, 40], 8, 2, 128, 16, 1, 100000), "rows": ([3001, 100], 8, 2, 64, 32, 4, 0), "blocks": ([600, 100], 40, 2, 128, 32, 2, 0),
    "wide32": ([3000, 0, 129], 24, 1, 128, 16, 1, 100000), "wide64": ([3000, 0, 129], 20, 1, 64, 16, 2, 100000),
}


def one_key_each(kind, form, power, spread=0):
    """Queries that are 2^power times a key of their sequence (a different one for each row), and which."""
    lens, hq, hkv, dh, size, q_len, more = FORMS[form]
    g = gen(len(lens) * 7 + dh + power)
    pages = sum(-(-n // size) for n in lens) + 1
    c = make_cache(kind, "heads", pages, hkv, size, dh, None)
    table = table_of(g, lens, size, pages)
    seq = torch.tensor([b for b, n in enumerate(lens) for _ in range(n)], dtype=torch.int32, device="cuda")
    pos = torch.tensor([p for n in lens for p in range(n)], dtype=torch.int32, device="cuda")
    tall = torch.exp2(torch.randint(-spread, spread + 1, (hkv, len(pos), 1), generator=g, device="cuda").float())
    up.kv_write(c, randn(g, hkv, len(pos), dh).bfloat16(), (tall * randn(g, hkv, len(pos), dh)).bfloat16(), seq, pos, table)
    q, which = torch.zeros(hq, len(lens) * q_len, dh, dtype=torch.float64, device="cuda"), torch.zeros(hq, len(lens) * q_len, dtype=torch.long)
    for b, n in enumerate(lens):
        k = cached(c, "k", table, b, n) if n else None
        for t in range(q_len):
            see = n - q_len + 1 + t
            for h in range(hq):
                if see > 0:
                    j = (h * 131 + t * 17 + see - 1) % see
                    which[h, b * q_len + t] = j
                    q[h, b * q_len + t] = k[h // (hq // hkv), j] * 2.0 ** power
    return c, widened(table, more, gen(1)) if more else table, q.bfloat16(), which


def check(kind, form, power, spread=0):
    lens, hq, hkv, dh, size, q_len, _ = FORMS[form]
    c, table, q, which = one_key_each(kind, form, power, spread)
    o, lse = run_decode(c, q, table, lens, q_len=q_len)
    sc, r = dh ** -0.5, 2.0 ** -10 if kind == "e4m3" else 2.0 ** -16
    for b, n in enumerate(lens):
        if not n:
            continue
        k, v = cached(c, "k", table, b, n), cached(c, "v", table, b, n)
        for t in range(q_len):
            i, see = b * q_len + t, n - q_len + 1 + t
            if see <= 0:
                assert bool((o[:, i] == 0).all()) and bool((lse[:, i] == -math.inf).all())
                continue
            x = q[:, i].double().view(hkv, hq // hkv, dh)
            s = x @ k[:, :see].transpose(1, 2) * sc
            j = which[:, i].to(s.device).view(hkv, -1, 1)
            top = s.gather(2, j)
            rest = s.scatter(2, j, -math.inf).amax(-1, keepdim=True)
            assert bool((top - rest > 60).all())
            others = torch.exp(s.scatter(2, j, -math.inf) - top) @ v[:, :see].abs()
            ref = v.gather(1, j.expand(-1, -1, dh))
            err = (o[:, i].double().view(ref.shape) - ref).abs()
            assert bool((err <= ref.abs() * (BF + r + 2.0 ** -18) + 2 * others + 2.0 ** -130).all()), f"sequence {b} token {t}: {float(err.max())}"
            mass = (x.abs()[..., None, :] @ k.gather(1, j.expand(-1, -1, dh)).abs()[..., None])[..., 0] * sc
            err = (lse[:, i].double().view(top.shape) - top).abs()
            assert bool((err <= mass * (2 * dh + 8) * U + 8 * U * top.abs() + 2.0 ** -20).all()), f"lse of sequence {b} token {t}"


@pytest.mark.parametrize("form", [f for f in FORMS if f[:4] != "wide"])
@pytest.mark.parametrize("power", [5, 10, 14, 18, 22])
def test_value_scales_beside_large_scores(power, form):
    """An e4m3 value's scale is part of its weight's exponent, and no bit of it is lost to the score."""
    check("e4m3", form, power)
    check("e4m3", form, power, 20)


@pytest.mark.parametrize("kind,form", [(k, f) for k in ("bf16", "e4m3") for f in FORMS if k == "bf16" or f[:4] != "wide"])
@pytest.mark.parametrize("power", [8, 24, 30, 60, 100])
def test_finite_scores_of_any_size(power, kind, form):
    check(kind, form, power)


@pytest.mark.parametrize("kind,form", [(k, f) for k in ("bf16", "e4m3") for f in FORMS if k == "bf16" or f[:4] != "wide"])
@pytest.mark.parametrize("power", [8, 14, 20, 40, 100])
def test_equal_keys_weigh_alike(power, kind, form):
    """Every key is there twice, in the other half of the sequence: o is the mean of two values, to its own rounding and the weights'."""
    lens, hq, hkv, dh, size, q_len, more = FORMS[form]
    lens = [n // 2 * 2 for n in lens]
    g = gen(len(lens) * 5 + dh + power)
    pages = sum(-(-n // size) for n in lens) + 1
    c = make_cache(kind, "heads", pages, hkv, size, dh, None)
    table = table_of(g, lens, size, pages)
    q = torch.zeros(hq, len(lens), dh, dtype=torch.bfloat16, device="cuda")
    which = torch.zeros(hq, len(lens), dtype=torch.long, device="cuda")
    for b, n in enumerate(lens):
        if n:
            k, v = randn(g, hkv, n // 2, dh).bfloat16(), randn(g, hkv, n, dh).bfloat16()
            pos = torch.arange(n, device="cuda").int()
            up.kv_write(c, torch.cat([k, k], 1), v, torch.full_like(pos, b), pos, table)
            for h in range(hq):
                which[h, b] = j = (h * 131 + 17) % (n // 2)
                q[h, b] = (cached(c, "k", table, b, n)[h // (hq // hkv), j] * 2.0 ** power).bfloat16()
    if more:
        table = widened(table, more, gen(1))
    o, _ = run_decode(c, q, table, lens)
    r = 2.0 ** -10 if kind == "e4m3" else 2.0 ** -16
    for b, n in enumerate(lens):
        if not n:
            continue
        x = q[:, b].double().view(hkv, -1, dh)
        s = (x @ cached(c, "k", table, b, n).transpose(1, 2))[..., : n // 2] * dh ** -0.5
        j = which[:, b].view(hkv, -1, 1)
        assert bool((s.gather(2, j) - s.scatter(2, j, -math.inf).amax(-1, keepdim=True) > 60).all())
        v = cached(c, "v", table, b, n)
        one, two = (v.gather(1, (j + i).expand(-1, -1, dh)) for i in (0, n // 2))
        ref, mass = (one + two) / 2, (one.abs() + two.abs()) / 2
        err = (o[:, b].double().view(ref.shape) - ref).abs()
        assert bool((err <= ref.abs() * BF + mass * (r + 2.0 ** -18) + 2.0 ** -20).all()), f"sequence {b}: {float(err.max())}"


@pytest.mark.parametrize("kind,form", [("bf16", "cta"), ("e4m3", "line"), ("bf16", "line"), ("bf16", "wide32"), ("bf16", "wide64")])
@pytest.mark.parametrize("power", [14, 24, 60])
def test_values_that_are_not_finite_beside_large_scores(power, kind, form):
    """A key without weight has an infinite value: the elements beside it are those of the key that has all of it."""
    lens, hq, hkv, dh, size, q_len, _ = FORMS[form]
    c, table, q, which = one_key_each(kind, form, power)
    clean, lse = run_decode(c, q, table, lens, q_len=q_len)
    page = int(table[0, 1]) if lens[0] > size else int(table[2, 1])
    b = 0 if lens[0] > size else 2
    (c.v.view(torch.uint8) if kind == "e4m3" else c.v)[page, :, 3, 9] = 0x7f if kind == "e4m3" else math.inf
    o, lse2 = run_decode(c, q, table, lens, q_len=q_len)
    rest = torch.arange(dh, device="cuda") != 9
    mine = slice(b * q_len, b * q_len + q_len)
    assert bool(((o - clean)[:, mine, rest].abs() <= clean[:, mine, rest].abs() * 2.0 ** -7 + 2.0 ** -130).all())
    assert bool(((lse2 - lse)[:, mine].abs() <= lse[:, mine].abs() * (2 * dh + 16) * 16 * U).all())
