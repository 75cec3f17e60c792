"""Decode with more than 16 query rows to a key head (32 with rows of 64 elements) and tables with room for many keys: blocks of 32 and
64 rows over tiles of 128 keys, against plain 64-bit arithmetic.  The tolerances are those of the other decode tests: the same roundings,
in chains of 16 keys of a CTA's part, with the weights as two bf16 numbers."""
import math

import pytest
import torch

import long_context_attention_upipe_gb300 as up
from test_gpu_kv import BF, LAYOUTS, NAN, cached, check_decode, gen, heads, make_cache, randn, run_decode, setup, setup_many, table_of, widened

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


def roomy(c, table):
    """The table with entries of garbage for as many keys as the larger tiles are taken for: 24 tiles of 128 to an SM."""
    keys = 24 * 128 * torch.cuda.get_device_properties(0).multi_processor_count
    return widened(table, -(-keys // (c.page_size * c.n_kv_heads * table.shape[0])), gen(1))


@pytest.mark.parametrize("dh,hq,hkv,q_len", [
    (128, 17, 1, 1), (128, 16, 2, 3), (128, 4, 1, 8), (128, 33, 1, 1), (128, 24, 3, 8), (128, 13, 1, 5), (128, 32, 2, 16), (128, 128, 1, 1),
    (64, 33, 1, 1), (64, 16, 2, 5), (64, 24, 3, 8), (64, 13, 1, 5), (64, 32, 2, 16)])
@pytest.mark.parametrize("size", [16, 48, 64, 256])
def test_lengths(dh, hq, hkv, q_len, size):
    lens = [0, 1, 15, 16, 17, 40, 127, 128, 0, 129, 255, 256, 257, 700, -3]
    c, table, q = setup("bf16", lens, hq, hkv, dh, size, q_len)
    check_decode(c, q, roomy(c, table), lens, q_len=q_len)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("size", [16, 32, 128])
@pytest.mark.parametrize("dh,hq", [(128, 48), (64, 80)])
def test_layouts_and_strides(layout, size, dh, hq):
    lens = [200, 3, size, 0, size + 1, 2 * size - 1]
    c, table, q = setup("bf16", lens, hq, 2, dh, size, layout=layout)
    table = roomy(c, table)
    o, lse = check_decode(c, q, table, lens)
    both = torch.zeros(len(lens), 2 * hq + 5, dh, dtype=torch.bfloat16, device="cuda")
    both[:, 3: 3 + hq] = q.transpose(0, 1)
    o2, lse2 = run_decode(c, both[:, 3: 3 + hq].transpose(0, 1), table, lens, o=both[:, 4 + hq: 4 + 2 * hq].transpose(0, 1))
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    assert bool((both[:, :3] == 0).all()) and bool((both[:, 3 + hq] == 0).all()) and bool((both[:, 4 + 2 * hq:] == 0).all())


@pytest.mark.parametrize("lens,hq,hkv,dh,size,q_len", [
    ([500000], 32, 1, 128, 128, 1), ([70001], 64, 8, 128, 64, 3), ([5003, 12, 0, 30001, 777], 40, 8, 128, 32, 4),
    ([300001], 40, 1, 64, 64, 1), ([60000, 7, 61000], 64, 4, 64, 16, 4)])
def test_long(lens, hq, hkv, dh, size, q_len):
    c, table, q = setup("bf16", lens, hq, hkv, dh, size, q_len)
    check_decode(c, q, roomy(c, table), lens, q_len=q_len)


@pytest.mark.parametrize("n", [31, 33, 64, 97, 257, 3001])
def test_batches(n):
    g = torch.Generator()
    g.manual_seed(n)
    lens = [int(x) if x < 300 else 0 for x in torch.randint(0, 400, (n,), generator=g)]
    c, table, q = setup_many("bf16", lens, 48, 2, 128, 16)
    check_decode(c, q, roomy(c, table), lens)


def test_65536_sequences_of_one_key():
    n, pages, hq = 65536, 37, 18
    c = make_cache("bf16", pages=pages, hkv=1, size=16, dh=128, fill=gen(9))
    b = torch.arange(n, device="cuda")
    table = (b % pages).int()[:, None].contiguous()
    q = randn(gen(10), hq, n, 128).bfloat16()
    o, lse = run_decode(c, q, table, (b % 2).int())
    assert bool((o[:, ::2] == 0).all()) and bool((lse[:, ::2] == -math.inf).all())
    assert torch.equal(o[:, 1::2], c.v[(b % pages)[1::2], 0, 0][None].expand(hq, -1, -1))


@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_flat_and_peaked_scores(spread):
    lens = [3000, 33]
    c, table, q = setup("bf16", lens, 48, 2, 128, 64, spread=spread)
    check_decode(c, q, roomy(c, table), lens)
    check_decode(c, q, roomy(c, table), lens, scale=-0.03)


@pytest.mark.parametrize("step", [0.3, -0.3, 30.0])
def test_scores_that_rise_and_fall_along_the_keys(step):
    """Every tile's scores pass the reference of those before it; or lie far below it."""
    n, hkv, hq, dh, size = 1500, 1, 24, 128, 16
    g = gen(5)
    c = make_cache("bf16", pages=100, hkv=hkv, size=size, dh=dh, fill=None)
    table, pos = table_of(g, [n], size, 100), torch.arange(n, device="cuda").int()
    k = 0.1 * randn(g, hkv, n, dh)
    k[..., 0] = step * torch.arange(n, device="cuda") / 16
    up.kv_write(c, k.bfloat16(), randn(g, hkv, n, dh).bfloat16(), torch.zeros_like(pos), pos, table)
    q = randn(g, hq, 1, dh)
    q[..., 0] = torch.linspace(-2, 3, hq, device="cuda")[:, None]
    check_decode(c, q.bfloat16(), roomy(c, table), [n])


@pytest.mark.parametrize("what", [NAN, float("inf"), -float("inf")])
def test_keeps_what_is_masked_out(what):
    """The newest token's key and value are not finite: the queries before it do not see them."""
    q_len, lens, hq = 4, [1000, 4, 37], 16
    c, table, q = setup("bf16", lens, hq, 2, 128, 16, q_len)
    table = roomy(c, table)
    clean, clean_lse = check_decode(c, q, table, lens, q_len=q_len)
    last = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    k, v = heads(gen(3), "head", 2, 3, 128), heads(gen(4), "head", 2, 3, 128)
    k[0, :, 7], v[:, :, 100] = what, what
    up.kv_write(c, k, v, torch.arange(3, device="cuda").int(), last, table)
    o, lse = run_decode(c, q, table, lens, q_len=q_len)
    seen = torch.arange(12, device="cuda") % q_len == q_len - 1
    assert bool(o[:, ~seen].isfinite().all())
    err = (o[:, ~seen].double() - clean[:, ~seen].double()).abs()
    assert bool((err <= clean[:, ~seen].double().abs() * 2 * BF + 2.0 ** -9).all())
    assert bool(((lse - clean_lse)[:, ~seen].abs() <= 2.0 ** -16).all())
    assert not bool(o[8:, seen, 100].isfinite().any()) and bool(o[8:, seen, :100].isfinite().all())


def test_infinite_values_and_keys_that_are_seen():
    lens, hq = [900, 90], 20
    c, table, q = setup("bf16", lens, hq, 1, 128, 16)
    table = roomy(c, table)
    clean, _ = run_decode(c, q, table, lens)
    page, rest = int(table[0, 20]), torch.arange(128, device="cuda") != 9
    for what in (NAN, math.inf, -math.inf):
        c.v[page, 0, 5, 9] = what
        o, lse = run_decode(c, q, table, lens)
        assert bool(o[:, 0, 9].isnan().all()) if what != what else bool((o[:, 0, 9] == what).all())
        err = (o[:, 0, rest].double() - clean[:, 0, rest].double()).abs()
        assert bool((err <= clean[:, 0, rest].double().abs() * 2 * BF + 2.0 ** -9).all())
        assert torch.equal(o[:, 1], clean[:, 1]) and bool(lse.isfinite().all())
        c.v[page, 0, 5, 9] = 0
        old = c.k[page, 0, 5, 9].clone()
        c.k[page, 0, 5, 9] = what
        o, lse = run_decode(c, q, table, lens)
        nan = ~(q[:, 0, 9].double() * what == -math.inf)
        assert bool(o[nan, 0].isnan().all()) and bool(o[~nan, 0].isfinite().all()) and torch.equal(o[:, 1], clean[:, 1])
        c.k[page, 0, 5, 9] = old


def test_nan_queries_stay_in_their_rows():
    lens = [50, 600]
    c, table, q = setup("bf16", lens, 32, 2, 128, 16, 2)
    table = roomy(c, table)
    clean, lse = run_decode(c, q, table, lens, q_len=2)
    q[5, 2, 0] = NAN
    o, lse2 = run_decode(c, q, table, lens, q_len=2)
    assert bool(o[5, 2].isnan().all()) and bool(lse2[5, 2].isnan())
    o[5, 2], lse2[5, 2] = clean[5, 2], lse[5, 2]
    assert torch.equal(o, clean) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dh,hq", [(128, 12), (64, 20)])
@pytest.mark.parametrize("page", [-1, 1 << 20, -2 ** 31])
def test_missing_pages_are_nan(page, dh, hq):
    lens = [100, 100, 100]
    c, table, q = setup("bf16", lens, hq, 2, dh, 16, 4)
    table = roomy(c, table)
    clean, _ = run_decode(c, q, table, lens, q_len=4)
    broken = table.clone()
    broken[1, 2] = page
    broken[2, 6] = page                  # positions 96 to 99: the first query sees 97 keys
    o, lse = run_decode(c, q, broken, lens, q_len=4)
    assert torch.equal(o[:, :4], clean[:, :4])
    assert bool(o[:, 4:].isnan().all()) and bool(lse[:, 4:].isnan().all())
    o, lse = run_decode(c, q, broken, [100, 32, 96], q_len=4)  # without the missing pages
    assert torch.equal(o[:, :4], clean[:, :4]) and bool(o.isfinite().all()) and bool(lse.isfinite().all())


def test_lengths_past_the_table_are_nan():
    c, table, q = setup("bf16", [3000] * 3, 48, 2, 128, 16, 1)
    keys = 24 * 128 * torch.cuda.get_device_properties(0).multi_processor_count
    table = table[:, :188].repeat(1, -(-keys // (188 * 16 * 6))).contiguous()
    cap = table.shape[1] * 16
    want, _ = run_decode(c, q, table, [cap, 3000, 5])
    o, lse = run_decode(c, q, table, [cap + 1, 3000, 5])
    assert bool(o[:, 0].isnan().all()) and bool(lse[:, 0].isnan().all()) and torch.equal(o[:, 1:], want[:, 1:])


def test_repeatable_and_needs_no_lse():
    lens = [40000, 17, 900]
    c, table, q = setup("bf16", lens, 64, 2, 128, 64)
    table = roomy(c, table)
    o, lse = run_decode(c, q, table, lens)
    for _ in range(5):
        o2, lse2 = run_decode(c, q, table, lens)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(o, run_decode(c, q, table, lens, lse=False)[0])


def test_graphs_of_both_kernels_share_a_workspace():
    c, table, q = setup("bf16", [2000, 2000, 2000], 48, 2, 128, 64)
    big = roomy(c, table)
    ln = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.full((up.decode_workspace_bytes(c, 3, 48),), 0xff, dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(q), torch.empty(48, 3, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for t, (o, lse) in zip((big, table), outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            up.decode(c, q, t, ln, o, ws, lse=lse)
        graphs.append(gr)
    for lens in ([300, 0, 77], [2000, 1999, 1], [0, 0, 0], [1, 1600, 128], [129, 127, 2000]):
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        for gr in graphs + graphs:
            gr.replay()
        torch.cuda.synchronize()
        for t, (o, lse) in zip((big, table), outs):
            want, wl = check_decode(c, q, t, lens)
            assert torch.equal(o, want) and torch.equal(lse, wl)


def test_two_streams_at_once():
    lens = [30000, 500]
    sets = [setup("bf16", lens, hq, 2, 128, 64, seed=hq) for hq in (48, 128)]
    sets = [(c, roomy(c, t), q) for c, t, q in sets]
    want = [run_decode(c, q, t, lens) for c, t, q in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = [(torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"),
            torch.empty(up.decode_workspace_bytes(c, 2, q.shape[0]), dtype=torch.uint8, device="cuda")) for c, _, q in sets]
    torch.cuda.synchronize()
    for _ in range(50):
        for (c, t, q), st, (o, lse, ws) in zip(sets, streams, out):
            up.decode(c, q, t, ln, o, ws, lse=lse, stream=st)
    torch.cuda.synchronize()
    for (o, lse, _), (wo, wl) in zip(out, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_beside_the_attention_core():
    """Both hold tensor memory: on two streams at once, neither waits for the other for ever or changes its results."""
    lens, S, hq, hkv, dh = [30000, 500], 4096, 8, 2, 128
    c, table, q = setup("bf16", lens, 48, 2, dh, 64)
    table = roomy(c, table)
    want, wl = run_decode(c, q, table, lens)
    g = gen(8)
    qs, ks, vs = (randn(g, h, S, dh).bfloat16() for h in (hq, hkv, hkv))
    desc = up.make_desc(S, hq * dh, hq, hkv, dh)
    tab = torch.empty(up.tile_table_bytes(desc), dtype=torch.uint8, device="cuda")
    up.build_tile_table(desc, None, tab)
    oc, lc = torch.empty_like(qs), torch.empty(hq, S, device="cuda")
    up.core_fwd(desc, qs, ks, vs, None, tab, oc, lc)
    core = oc.clone()
    ln, o = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    ws = torch.empty(up.decode_workspace_bytes(c, 2, 48), dtype=torch.uint8, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        up.decode(c, q, table, ln, o, ws, stream=a)
        with torch.cuda.stream(b):
            up.core_fwd(desc, qs, ks, vs, None, tab, oc, lc)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(oc, core)


def test_waits_that_run_out_give_nan_or_the_right_values():
    lens = [30000, 40, 900]
    c, table, q = setup("bf16", lens, 48, 2, 128, 64)
    table = roomy(c, table)
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


def test_pages_past_32_bit_offsets():
    hkv, size, dh = 8, 64, 128
    pages = 2 ** 32 // (hkv * size * dh) + 3
    x = torch.empty(2, pages, hkv, size, dh, dtype=torch.bfloat16, device="cuda")
    c = up.KVCache(x[0], x[1])
    g, n = gen(5), 100
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    k, v, pos = heads(g, "head", hkv, n, dh), heads(g, "head", hkv, n, dh), torch.arange(n, device="cuda").int()
    up.kv_write(c, k, v, torch.zeros_like(pos), pos, table)
    check_decode(c, randn(g, 24 * hkv, 1, dh).bfloat16(), roomy(c, table), [n])


def test_long_line_of_aliased_pages():
    """One sequence of 2^26 keys whose table names the same 64 pages again and again: n equal runs weigh alike, so o and lse - log n are
    those of one run.  A chain of a CTA's part adds its keys 16 at a time; additions that truncate lose up to 2 u of the sum each."""
    runs, size, pages, hq, dh = 2 ** 26 // (64 * 128), 128, 64, 24, 128
    c = make_cache("bf16", pages=pages, hkv=1, size=size, dh=dh, fill=gen(2))
    one = torch.arange(pages, device="cuda").int()[None]
    q = randn(gen(3), hq, 1, dh).bfloat16()
    o, lse = run_decode(c, q, one.repeat(1, runs).contiguous(), [runs * pages * size])
    s = (q[:, 0].double() @ cached(c, "k", one, 0, pages * size)[0].T) * dh ** -0.5
    want = torch.logsumexp(s, -1)
    w = torch.exp(s - want[:, None])
    v = cached(c, "v", one, 0, pages * size)[0]
    u = 2.0 ** -24
    links = 2 ** 26 / torch.cuda.get_device_properties(0).multi_processor_count / 16 * 2  # two products to 16 keys; + margin of the split's ends
    tol = (w @ v).abs() * BF + (w @ v.abs()) * (2.0 ** -14 + (links + 2000) * 2 * u)
    assert bool(((o[:, 0].double() - w @ v).abs() <= tol).all())
    # a thread's sum of l has one key of 128: 2^26 / SMs / 128 additions that round
    assert bool(((lse[:, 0].double() - want - math.log(runs)).abs() <= 2.0 ** -14 + (links / 16 + 200) * u).all())
