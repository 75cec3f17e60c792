"""Decode of the longest sequence: with more than 16 query rows to a key head 2^31 - 1 keys, whose last tile of 128 ends where 32-bit positions do,
against plain 64-bit arithmetic; with an e4m3 cache, queries whose small elements have to be looked after."""
import math

import pytest
import torch

from test_gpu_kv import BF, NAN, U, cached, gen, make_cache, randn, run_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


@pytest.mark.parametrize("short", [1, 2, 127])
@pytest.mark.parametrize("dh,hq,q_len", [(128, 24, 1), (128, 12, 2), (128, 40, 1), (64, 20, 2)])
def test_masks_of_the_longest_sequence(dh, hq, q_len, short):
    """2^31 - short keys: page 0 under every entry of the table but the last, which names page 1.  The newest key takes nearly all of the
    weight of the query that sees it, and the rows behind the end are NaN.

    Of 2^31 keys a CTA has 1 / SMs, 16 to a link of O's chains, two products each that may truncate (2 u of the sum so far, which grows
    from nothing: half of it on average): the tolerance is in units of W.  A thread's sum of l has one key of 128, rounded to nearest."""
    size, n = 1 << 16, 2 ** 31 - short
    runs = 2 ** 31 // size - 1
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g = gen(dh + hq)
    c = make_cache("bf16", pages=2, hkv=1, size=size, dh=dh, fill=g)
    table = torch.zeros(1, runs + 1, dtype=torch.int32, device="cuda")
    table[0, runs] = 1
    c.v.add_(1.0)
    c.k[1, 0, size - short:] = NAN
    c.v[1, 0, size - short:] = NAN
    q = randn(g, hq, q_len, dh)
    q[..., 0] = 4.0
    q = q.bfloat16()
    c.k[:, 0, :, 0] = 0.0
    newest = size - short - 1
    c.k[1, 0, newest, 0] = 16 * dh ** 0.5       # a score of 64 +- 6: e^-36 of the weight is left to 2^31 others
    c.v[1, 0, newest] = 100.0
    o, lse = run_decode(c, q, table, [n], q_len=q_len)
    k0, v0 = cached(c, "k", table, 0, size)[0], cached(c, "v", table, 0, size)[0]
    k1, v1 = c.k[1, 0, : size - short].double(), c.v[1, 0, : size - short].double()
    links = 2 ** 31 / sms / 16 * 2
    for t in range(q_len):
        see = size - short - (q_len - 1 - t)
        x = q[:, t].double() * dh ** -0.5
        s0, s1 = x @ k0.t(), x @ k1[:see].t()
        want = torch.logsumexp(torch.cat([s0 + math.log(runs), s1], 1), 1)
        w0, w1 = torch.exp(s0 - want[:, None]) * runs, torch.exp(s1 - want[:, None])
        ref, mass = w0 @ v0 + w1 @ v1[:see], w0 @ v0.abs() + w1 @ v1[:see].abs()
        assert bool(((o[:, t].double() - ref).abs() <= ref.abs() * BF + mass * (2.0 ** -10 + links * U)).all())
        assert bool(((lse[:, t].double() - want).abs() <= 2.0 ** -10 + links / 16 * U).all())
        assert bool((ref > 99).all()) if t == q_len - 1 else bool((ref < 20).all())


def test_dead_channels_of_the_longest_sequence():
    """A query with an element next to nothing: the scales of all keys up to 2^31 - 1 are looked at, and the result is that without the element."""
    size, dh = 1 << 20, 64
    g = gen(78)
    c = make_cache("e4m3", pages=1, hkv=1, size=size, dh=dh, fill=g)
    table = torch.zeros(1, 2048, dtype=torch.int32, device="cuda")
    q = randn(g, 2, 1, dh).bfloat16()
    q[..., 9] = 0
    want, wl = run_decode(c, q, table, [2 ** 31 - 1])
    q[..., 9] = 1e-30
    o, lse = run_decode(c, q, table, [2 ** 31 - 1])
    assert bool(o.isfinite().all())
    # below fp16's smallest number, so the products are the same
    assert torch.equal(o, want) and torch.equal(lse, wl)
