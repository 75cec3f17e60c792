"""Decode over an e4m3 cache with queries whose elements differ by many powers of two: the loss of a score is counted against sum_i
|q_i k_i|, as for any other query, not against the largest element of q times the largest of k.  The tolerances are those of the
other decode tests."""
import pytest
import torch

import long_context_attention_upipe_gb300 as up
from test_gpu_kv import check_decode, gen, heads, make_cache, randn, run_decode, setup, table_of, widened

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


def one_large_channel(lens, hq, hkv, dh, size, q_len, power, rows, tiny=0.0, seed=0):
    """Queries of which `rows` (of 5) have an element 2^power times the others'; the keys there are `tiny` of a code's unit, or zero."""
    c, table, q = setup("e4m3", lens, hq, hkv, dh, size, q_len, seed=seed, spread=1.0)
    ch = 37
    codes = c.k.view(torch.uint8)
    codes[..., ch] = 1 if tiny else 0                       # 2^-9 of the scale, or nothing
    q = q.float()
    pick = torch.arange(hq, device="cuda")[:, None] * 7 + torch.arange(q.shape[1], device="cuda")[None] * 3
    big = (pick % 5 < rows)
    q[..., ch] = torch.where(big, torch.full_like(q[..., ch], 1.5), q[..., ch])
    if tiny:                                                # every score is moved alike, by some units
        q = torch.where(big[..., None], q * 2.0 ** -4, q)
        q[..., ch] = torch.where(big, torch.full_like(q[..., ch], 1.0), q[..., ch])
        small = q * 2.0 ** -power
        small[..., ch] = q[..., ch]
        return c, table, torch.where(big[..., None], small, q).bfloat16()
    q[..., ch] = torch.where(big, q[..., ch] * 2.0 ** power, q[..., ch])
    return c, table, q.bfloat16()


POWERS = [8, 14, 17, 22, 26, 31, 34, 40, 60, 100]
FORMS = [  # lengths, query heads, key heads, head_dim, page, q_len, columns that the table has beside: each way through the kernels
    ([1, 17, 200], 4, 1, 128, 16, 1, 0),             # a CTA to each item
    ([2000], 4, 1, 128, 64, 1, 0),                   # a cluster to the item
    ([(i * 37) % 300 for i in range(200)], 2, 1, 64, 16, 1, 0),   # parts of whole items
    ([5003, 12, 0, 777], 8, 2, 128, 32, 1, 0),       # the line and joins
    ([6000, 40], 8, 2, 128, 16, 1, 100000),          # 16 warps
    ([3001, 100], 8, 2, 64, 32, 4, 0),               # 16 rows
    ([600, 100], 40, 2, 128, 32, 2, 0),              # several blocks of rows
]


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("power", POWERS)
def test_large_channel_that_meets_zeros(power, form):
    lens, hq, hkv, dh, size, q_len, more = FORMS[form]
    c, table, q = one_large_channel(lens, hq, hkv, dh, size, q_len, power, 2)
    if more:
        table = widened(table, more, gen(1))
    check_decode(c, q, table, lens, q_len=q_len)


@pytest.mark.parametrize("power", [3, 10, 14, 18, 22])
def test_large_channel_that_meets_tiny_codes(power):
    lens = [700, 33]
    c, table, q = one_large_channel(lens, 8, 2, 128, 64, 1, power, 5, tiny=1.0)
    check_decode(c, q, table, lens)


@pytest.mark.parametrize("power", [22, 50])
def test_scores_that_come_from_the_small_elements_alone(power):
    """The case by hand: scores of a few units, all of them from elements far below the largest."""
    g = gen(3)
    n, hkv, dh = 300, 1, 128
    c = make_cache("e4m3", pages=20, hkv=hkv, size=16, dh=dh)
    table, pos = table_of(g, [n], 16, 20), torch.arange(n, device="cuda").int()
    k = randn(g, hkv, n, dh)
    k[..., 0] = 0
    up.kv_write(c, k.bfloat16(), randn(g, hkv, n, dh).bfloat16(), torch.zeros_like(pos), pos, table)
    q = 4 * randn(g, 8, 1, dh)
    q[..., 0] = 2.0 ** power
    o, lse = check_decode(c, q.bfloat16(), table, [n])
    other = q.clone()
    other[..., 0] = 0                       # the same scores
    o2, lse2 = check_decode(c, other.bfloat16(), table, [n])
    assert bool(((lse - lse2).abs() <= 2.0 ** -12).all())


@pytest.mark.parametrize("what", ["v", "k", "missing", "long", "nan"])
def test_far_apart_elements_beside_other_trouble(what):
    """Rows of such queries where values or keys are not finite, a page is missing, the length passes the table, or q is NaN."""
    lens, q_len = [1000, 90], 2
    c, table, q = one_large_channel(lens, 8, 2, 128, 16, q_len, 60, 2)
    clean, lse = check_decode(c, q, table, lens, q_len=q_len)
    codes, page = (c.v if what == "v" else c.k).view(torch.uint8), int(table[0, 20])
    if what in "vk":
        codes[page, :, 3, 9] = 0x7f
        o, e = run_decode(c, q, table, lens, q_len=q_len)
        if what == "v":
            rest = torch.arange(128, device="cuda") != 9
            assert bool(o[:, :2, 9].isnan().all()) and bool(e.isfinite().all())
            assert bool(((o - clean)[:, :2, rest].abs() <= clean[:, :2, rest].abs() * 2.0 ** -7 + 2.0 ** -9).all())
        else:
            assert bool(o[:, :2].isnan().all()) and bool(e[:, :2].isnan().all())
    elif what == "nan":
        q[3, 1, 5] = float("nan")
        o, e = run_decode(c, q, table, lens, q_len=q_len)
        assert bool(o[3, 1].isnan().all()) and bool(e[3, 1].isnan())
        o[3, 1], e[3, 1] = clean[3, 1], lse[3, 1]
        assert torch.equal(o, clean) and torch.equal(e, lse)
        return
    else:
        t, n = table.clone(), list(lens)
        if what == "missing":
            t[0, 20] = -1
        else:
            n[0] = t.shape[1] * 16 + 1
        o, e = run_decode(c, q, t, n, q_len=q_len)
        assert bool(o[:, :2].isnan().all()) and bool(e[:, :2].isnan().all())
    assert torch.equal(o[:, 2:], clean[:, 2:]) and torch.equal(e[:, 2:], lse[:, 2:])


def test_tokens_before_the_first_of_far_apart_queries():
    lens = [2, 0, 20]
    c, table, q = one_large_channel(lens, 4, 1, 64, 16, 4, 70, 5)
    check_decode(c, q, table, lens, q_len=4)


@pytest.mark.parametrize("power", [-126, -111, -60, 60])
def test_queries_of_any_size_as_a_whole(power):
    """Largest elements at both ends of bf16's range, subnormal ones among the others; keys of the opposite size."""
    g = gen(4)
    n, hkv, dh = 200, 2, 64
    c = make_cache("e4m3", pages=14, hkv=hkv, size=16, dh=dh)
    table, pos = table_of(g, [n], 16, 14), torch.arange(n, device="cuda").int()
    against = max(-90, min(110, -power))
    up.kv_write(c, (randn(g, hkv, n, dh) * 2.0 ** against).bfloat16(), randn(g, hkv, n, dh).bfloat16(), torch.zeros_like(pos), pos, table)
    check_decode(c, (randn(g, 8, 1, dh).double() * 2.0 ** power).bfloat16(), table, [n])


@pytest.mark.parametrize("power", [-140, -126, -118, -112, -60, 60, 100, 108])
@pytest.mark.parametrize("hq,q_len", [(8, 1), (8, 4)])
def test_scales_that_no_write_makes(power, hq, q_len):
    """Scales of keys down to subnormal numbers and up to 2^108, of a cache that was filled some other way; queries of the opposite size."""
    g = gen(6)
    n, hkv, dh = 200, 2, 128
    c = make_cache("e4m3", pages=14, hkv=hkv, size=16, dh=dh, fill=g)
    table = table_of(g, [n], 16, 14)
    c.k_scale.copy_((0.5 + torch.rand(c.k_scale.shape, generator=g, device="cuda")).double() * 2.0 ** power)
    q = randn(g, hq, q_len, dh).double() * 2.0 ** (min(122, -power) - 7)
    check_decode(c, q.bfloat16(), table, [n], q_len=q_len)


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("power", [-40, -90, -133])
def test_dead_channels(power, form):
    """Some elements of most queries are next to nothing, beside ordinary ones: no score shows it."""
    lens, hq, hkv, dh, size, q_len, more = FORMS[form]
    c, table, q = setup("e4m3", lens, hq, hkv, dh, size, q_len)
    dead = (torch.arange(dh, device="cuda") % 5 == 2) & (torch.arange(hq, device="cuda")[:, None, None] % 4 != 1)
    q = torch.where(dead, (q.double() * 2.0 ** power).bfloat16(), q)
    if more:
        table = widened(table, more, gen(1))
    check_decode(c, q, table, lens, q_len=q_len)


@pytest.mark.parametrize("what", ["v", "missing"])
def test_dead_channels_beside_other_trouble(what):
    """A row that needs nothing made anew for its small elements may need it for a value that is not finite."""
    lens = [1000, 90]
    c, table, q = setup("e4m3", lens, 8, 2, 128, 16)
    q[..., 5] = 1e-30
    clean, lse = check_decode(c, q, table, lens)
    if what == "v":
        c.v.view(torch.uint8)[int(table[0, 20]), :, 3, 9] = 0x7f
        rest = torch.arange(128, device="cuda") != 9
        o, e = run_decode(c, q, table, lens)
        assert bool(o[:, 0, 9].isnan().all()) and bool(e.isfinite().all())
        assert bool(((o - clean)[:, 0, rest].abs() <= clean[:, 0, rest].abs() * 2.0 ** -7 + 2.0 ** -9).all())
    else:
        table = table.clone()
        table[0, 20] = -1
        o, e = run_decode(c, q, table, lens)
        assert bool(o[:, 0].isnan().all()) and bool(e[:, 0].isnan().all())
    assert torch.equal(o[:, 1], clean[:, 1]) and torch.equal(e[:, 1], lse[:, 1])


@pytest.mark.parametrize("keys", [1.0, 2.0 ** 8, 2.0 ** 14, 2.0 ** 30])
def test_small_elements_that_matter_by_the_size_of_the_keys(keys):
    """Elements 2^-34 of a row's largest, which meets zeros: the score grows with the keys, and its loss would."""
    g = gen(9)
    n, hkv, dh = 300, 1, 128
    c = make_cache("e4m3", pages=20, hkv=hkv, size=16, dh=dh)
    table, pos = table_of(g, [n], 16, 20), torch.arange(n, device="cuda").int()
    k = keys * randn(g, hkv, n, dh)
    k[..., 0] = 0
    up.kv_write(c, k.bfloat16(), randn(g, hkv, n, dh).bfloat16(), torch.zeros_like(pos), pos, table)
    q = 4 * randn(g, 8, 1, dh) / keys
    q[..., 0] = 2.0 ** 36 / keys
    check_decode(c, q.bfloat16(), table, [n])
