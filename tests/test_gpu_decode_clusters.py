"""Decode of short sequences: few of them with one CTA, or a cluster of 2, 4 or 8, to a sequence and key head, more as parts of the line that
begin and end with items, by the keys that the table has room for; against plain 64-bit arithmetic (the tolerances of the other decode
tests)."""
import pytest
import torch

import long_context_attention_upipe_gb300 as up
from test_gpu_kv import BF, KINDS, LAYOUTS, NAN, check_decode, gen, heads, run_decode, setup, widened

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


ROOMS = [512, 528, 1024, 1040, 2048, 2064, 4096, 4112]  # keys: 512 for one CTA, 256 each for 4 and 8, 512 each for 8, the line beyond


def room(c, table, keys):
    assert table.shape[1] * c.page_size <= keys
    return widened(table, keys // c.page_size - table.shape[1], gen(1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("keys", ROOMS)
@pytest.mark.parametrize("dh,hq,hkv,q_len", [(128, 4, 1, 1), (64, 6, 2, 1), (128, 8, 1, 2), (64, 9, 1, 3), (128, 12, 1, 16)])
def test_rooms(kind, keys, dh, hq, hkv, q_len):
    lens = [0, 1, 130, keys if keys < 2048 else 33, -2]
    c, table, q = setup(kind, lens, hq, hkv, dh, 16, q_len)
    check_decode(c, q, room(c, table, keys), lens, q_len=q_len)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 127, 129, 500, 1023, 1025, 2000, 2048])
def test_one_sequence(kind, n):
    c, table, q = setup(kind, [n], 16, 4, 128, 16)
    check_decode(c, q, room(c, table, 2048), [n])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seqs", [6, 7, 12, 13, 16, 17, 32, 33, 64, 65, 100])
def test_batches(kind, seqs):
    g = torch.Generator()
    g.manual_seed(seqs)
    lens = [int(x) if x < 1000 else 0 for x in torch.randint(0, 1200, (seqs,), generator=g)]
    c, table, q = setup(kind, lens, 2, 1, 64, 48)
    check_decode(c, q, widened(table, max(0, 21 - table.shape[1]), gen(1)), lens)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_layouts_and_strides(kind, layout):
    lens = [900, 3]
    c, table, q = setup(kind, lens, 8, 2, 128, 32, layout=layout)
    table = room(c, table, 2048)
    o, lse = check_decode(c, q, table, lens)
    both = torch.zeros(len(lens), 24, 128, dtype=torch.bfloat16, device="cuda")
    both[:, 4:12] = q.transpose(0, 1)
    o2, lse2 = run_decode(c, both[:, 4:12].transpose(0, 1), table, lens, o=both[:, 12:20].transpose(0, 1))
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    assert bool((both[:, :4] == 0).all()) and bool((both[:, 20:] == 0).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("what", [NAN, float("inf"), -float("inf")])
def test_keeps_what_is_masked_out(kind, what):
    q_len, lens = 4, [1000, 4, 37]
    c, table, q = setup(kind, lens, 4, 2, 128, 16, q_len)
    table = room(c, table, 2048)
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
    assert not bool(o[2:, seen, 100].isfinite().any())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [-1, 1 << 20])
def test_missing_pages_and_lengths_past_the_table_are_nan(kind, page):
    lens = [1000, 1000]
    c, table, q = setup(kind, lens, 8, 2, 64, 16)
    table = room(c, table, 2048)
    clean, _ = run_decode(c, q, table, lens)
    broken = table.clone()
    broken[1, 20] = page
    o, lse = run_decode(c, q, broken, lens)
    assert torch.equal(o[:, 0], clean[:, 0]) and bool(o[:, 1].isnan().all()) and bool(lse[:, 1].isnan().all())
    o, lse = run_decode(c, q, table, [1000, 2049])
    assert torch.equal(o[:, 0], clean[:, 0]) and bool(o[:, 1].isnan().all()) and bool(lse[:, 1].isnan().all())


@pytest.mark.parametrize("kind", KINDS)
def test_graph_replayed_with_other_lengths(kind):
    c, table, q = setup(kind, [2000, 1500], 8, 2, 128, 16)
    table = room(c, table, 2048)
    ln, o, lse = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.empty(8, 2, device="cuda")
    ws = torch.full((up.decode_workspace_bytes(c, 2, 8),), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        up.decode(c, q, table, ln, o, ws, lse=lse)
        up.decode(c, q, table, ln, o, ws, lse=lse)
    for lens in ([2000, 1500], [0, 1], [1, 0], [17, 1025], [0, 0], [129, 1500]):
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want, wl = check_decode(c, q, table, lens)
        assert torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind", KINDS)
def test_waits_that_run_out_give_nan_or_the_right_values(kind):
    lens = [2000, 40, 900]
    c, table, q = setup(kind, lens, 8, 2, 128, 64)
    table = room(c, table, 2048)
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


def test_clusters_beside_other_work():
    """Many at once on two streams, with a library product between them."""
    sets = [setup(kind, [2000, 700], 8, 4, 128, 64, seed=i) for i, kind in enumerate(KINDS)]
    sets = [(c, room(c, t, 2048), q) for c, t, q in sets]
    want = [run_decode(c, q, t, [2000, 700]) for c, t, q in sets]
    ln = torch.tensor([2000, 700], dtype=torch.int32, device="cuda")
    out = [(torch.empty_like(q), torch.empty(8, 2, device="cuda"), torch.empty(up.decode_workspace_bytes(c, 2, 8), dtype=torch.uint8, device="cuda"))
           for c, _, q in sets]
    streams, x = [torch.cuda.Stream() for _ in sets], torch.randn(1024, 1024, device="cuda")
    torch.cuda.synchronize()
    for _ in range(50):
        for (c, t, q), st, (o, lse, ws) in zip(sets, streams, out):
            up.decode(c, q, t, ln, o, ws, lse=lse, stream=st)
            with torch.cuda.stream(st):
                x @ x
    torch.cuda.synchronize()
    for (o, lse, _), (wo, wl) in zip(out, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seqs,hkv", [(153, 1), (160, 2), (100, 3), (304, 2), (608, 1), (609, 1)])
@pytest.mark.parametrize("some", ["none", "one", "last", "few", "many"])
def test_more_items_than_ctas(kind, seqs, hkv, some):
    """Up to 512 keys each; most sequences empty or not."""
    keys = {"none": [], "one": [(77, 300)], "last": [(seqs - 1, 512)], "few": [(i, 1 + i * 5 % 512) for i in range(3, seqs, 29)],
            "many": [(i, i * 7 % 130) for i in range(seqs) if i % 6]}[some]
    lens = [-1] * seqs
    for i, n in keys:
        lens[i] = n
    c, table, q = setup(kind, lens, 4 * hkv, hkv, 64, 32)
    check_decode(c, q, widened(table, 16 - table.shape[1], gen(1)), lens)


@pytest.mark.parametrize("kind", KINDS)
def test_more_items_than_ctas_replayed_with_other_lengths(kind):
    seqs = 200
    c, table, q = setup(kind, [64] * seqs, 24, 1, 128, 64)
    ln, o, lse = torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.empty(24, seqs, device="cuda")
    ws = torch.full((up.decode_workspace_bytes(c, seqs, 24),), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        up.decode(c, q, table, ln, o, ws, lse=lse)
        up.decode(c, q, table, ln, o, ws, lse=lse)
    for step in range(4):
        lens = [(i * (step + 3)) % 65 for i in range(seqs)] if step else [0] * seqs
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want, wl = check_decode(c, q, table, lens)
        assert torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("columns", [1, 3, 40])
def test_lengths_past_the_table_and_no_table(columns):
    """65 keys and a table of fewer, for few and for many items and for the line: NaN; the others as they were."""
    for seqs in (3, 200, 700):
        c, table, q = setup("bf16", [16] * seqs, 8, 2, 64, 16)
        table = widened(table, columns - 1, gen(2))
        lens = [16 if i % 3 else columns * 16 + 1 for i in range(seqs)]
        o, lse = run_decode(c, q, table, lens)
        lost = torch.arange(seqs, device="cuda") % 3 == 0
        assert bool(o[:, lost].isnan().all()) and bool(lse[:, lost].isnan().all()) and bool(o[:, ~lost].isfinite().all())
        o, lse = run_decode(c, q, table[:, :0], [0 if i % 3 else 5 for i in range(seqs)])
        assert bool(o[:, lost].isnan().all()) and bool((o[:, ~lost] == 0).all()) and bool((lse[:, ~lost] == -float("inf")).all())


def test_many_empty_sequences_among_long_ones():
    lens = [0 if i % 8 else 1200 + i for i in range(150)]
    c, table, q = setup("bf16", lens, 40, 8, 128, 64, 2)
    check_decode(c, q, table, lens, q_len=2)
