"""Paged cache of keys and values and the attention that reads it: what the entry points refuse, checked without a
GPU (every check runs on the host before any launch)."""
import ctypes
import math

import pytest
import torch

import long_context_attention_upipe_gb300 as up

ODD = 8  # bytes off a 16-byte boundary


def fake(i):
    """Distinct addresses, 1 TiB apart; never dereferenced."""
    return 0x100000 + (i << 40)


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


@pytest.fixture(autouse=True)
def nothing_launched():
    n = up.launch_count()
    yield
    assert up.launch_count() == n


PAGES, HEADS, SIZE, DIM = 10, 4, 32, 128


def cache(e4m3=False, **kw):
    a = dict(k=fake(0), v=fake(1), k_scale=fake(2) if e4m3 else None, v_scale=fake(3) if e4m3 else None, n_pages=PAGES,
             page_stride=HEADS * SIZE * DIM, head_stride=SIZE * DIM, token_stride=DIM, scale_page_stride=HEADS * SIZE,
             scale_head_stride=SIZE, scale_token_stride=1, page_size=SIZE, n_kv_heads=HEADS, head_dim=DIM, dtype=int(e4m3))
    a.update(kw)
    return up.KVCacheDesc(*(a[f] for f, _ in up.KVCacheDesc._fields_))


def table(**kw):
    a = dict(pages=fake(4), stride=6, n_seqs=3, max_pages=5)
    a.update(kw)
    return up.PageTable(*(a[f] for f, _ in up.PageTable._fields_))


def copy(f, c=None, t=None, **kw):
    a = dict(tokens=7, seq=fake(5), pos=fake(6), k=fake(7), khs=7 * DIM, kts=DIM, v=fake(8), vhs=7 * DIM, vts=DIM)
    a.update(kw)
    return f(ctypes.byref(c or cache()), ctypes.byref(t or table()), a["tokens"], a["seq"], a["pos"], a["k"], a["khs"], a["kts"],
             a["v"], a["vhs"], a["vts"], None)


def decode(c=None, t=None, **kw):
    tokens = 3 * kw.get("q_len", 2)
    a = dict(lens=fake(5), hq=8, q_len=2, scale=0.0, q=fake(6), qhs=tokens * DIM, qts=DIM, o=fake(7), ohs=tokens * DIM, ots=DIM,
             lse=fake(8), ws=fake(9), bytes=1 << 39)
    a.update(kw)
    return up.lib().upipe_attn_decode(ctypes.byref(c or cache()), ctypes.byref(t or table()), a["lens"], a["hq"], a["q_len"], a["scale"],
                                      a["q"], a["qhs"], a["qts"], a["o"], a["ohs"], a["ots"], a["lse"], a["ws"], a["bytes"], None)


def size(c=None, n_seqs=3, hq=8, q_len=1):
    n = ctypes.c_size_t(0)
    return up.lib().upipe_attn_decode_workspace_size(ctypes.byref(c or cache()), n_seqs, hq, q_len, ctypes.byref(n)), n.value


# what any call refuses of a cache; the arguments that follow are valid, so nothing else is in the way
CACHES = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(n_pages=0), 1), (dict(n_pages=1 << 31), 1), (dict(page_size=0), 1),
    (dict(page_size=24), 2), (dict(page_size=1 << 21), 2), (dict(n_kv_heads=0), 1), (dict(n_kv_heads=1025, page_stride=1 << 30), 2),
    (dict(head_dim=96), 2), (dict(head_dim=0), 1), (dict(dtype=2), 1), (dict(dtype=1), 1), (dict(k_scale=fake(2)), 1),
    (dict(e4m3=True, v_scale=None), 1), (dict(k=fake(0) + ODD), 3), (dict(v=fake(1) + ODD), 3), (dict(e4m3=True, k_scale=fake(2) + ODD), 3),
    (dict(page_stride=-1), 1), (dict(page_stride=1 << 60), 1), (dict(token_stride=132, head_stride=1 << 16, page_stride=1 << 20), 2),
    (dict(token_stride=64), 1), (dict(head_stride=SIZE * DIM - 8), 1), (dict(page_stride=HEADS * SIZE * DIM - 8), 1),
    (dict(v=fake(0)), 1), (dict(v=fake(0) + 2 * DIM), 1), (dict(v=fake(0) + 2 * HEADS * SIZE * DIM), 1),
    (dict(page_stride=2 * HEADS * SIZE * DIM, v=fake(0) + HEADS * SIZE * DIM), 1),       # half a page's keys under the values
    (dict(e4m3=True, v_scale=fake(2)), 1), (dict(e4m3=True, scale_token_stride=0), 1), (dict(e4m3=True, k_scale=fake(0) + 4096), 1),
    (dict(e4m3=True, head_stride=SIZE * DIM + 8, page_stride=1 << 20), 2),
]


@pytest.mark.parametrize("kw,code", CACHES)
def test_cache_refusals(kw, code):
    c = cache(**kw)
    assert copy(up.lib().upipe_attn_kv_write, c) == code
    assert copy(up.lib().upipe_attn_kv_read, c) == code
    assert decode(c) == code
    assert size(c)[0] == code


def test_cache_layouts_that_are_taken():
    """Every check passes and the call ends at the missing index array (1) or, for the size, well."""
    inter = dict(page_stride=2 * HEADS * SIZE * DIM, v=fake(0) + 2 * HEADS * SIZE * DIM)              # [pages, 2, heads, ...]
    by_token = dict(page_stride=SIZE * HEADS * DIM, head_stride=DIM, token_stride=HEADS * DIM)        # [pages, tokens, heads, ...]
    both = dict(page_stride=SIZE * 2 * HEADS * DIM, head_stride=DIM, token_stride=2 * HEADS * DIM, v=fake(0) + 2 * HEADS * DIM)
    one = dict(n_pages=1, page_stride=-5, n_kv_heads=1, head_stride=3)                               # strides that do not count
    heads_out = dict(head_stride=PAGES * SIZE * DIM, page_stride=SIZE * DIM)
    for kw in (inter, by_token, both, one, heads_out):
        assert size(cache(**kw))[0] == 0
    assert size(cache(True, scale_page_stride=SIZE * HEADS, scale_head_stride=1, scale_token_stride=HEADS))[0] == 0


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), 1), (dict(max_pages=-1), 1), (dict(stride=4), 1), (dict(pages=None), 1), (dict(n_seqs=65537), 2),
    (dict(pages=fake(4) + 2), 3), (dict(stride=1 << 60), 1)])
def test_table_refusals(kw, code):
    for f in (up.lib().upipe_attn_kv_write, up.lib().upipe_attn_kv_read):
        assert copy(f, t=table(**kw)) == code
    assert decode(t=table(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 1), (dict(tokens=1 << 31), 1), (dict(seq=None), 1), (dict(pos=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(k=fake(7) + ODD), 3), (dict(seq=fake(5) + 2), 3), (dict(kts=132), 2), (dict(vhs=-8), 1), (dict(vts=1 << 60), 1),
    (dict(k=fake(0)), 1), (dict(v=fake(1) + 4096), 1),                       # over the cache
    (dict(tokens=0, seq=None, pos=None, k=None, v=None), 0)])
def test_copy_refusals(kw, code):
    assert copy(up.lib().upipe_attn_kv_write, **kw) == code
    assert copy(up.lib().upipe_attn_kv_read, **kw) == code


def test_write_refuses_indices_in_the_cache():
    f = up.lib().upipe_attn_kv_write
    assert copy(f, seq=fake(0) + 64) == 1 and copy(f, pos=fake(1)) == 1 and copy(f, t=table(pages=fake(1) + 4)) == 1
    assert copy(f, cache(True), seq=fake(2)) == 1


def test_read_refuses_outputs_that_meet():
    f = up.lib().upipe_attn_kv_read
    assert copy(f, v=fake(7)) == 1 and copy(f, v=fake(7) + 2 * DIM) == 1                    # k and v
    assert copy(f, kts=64) == 1 and copy(f, khs=0) == 1                                   # rows of one output
    assert copy(f, k=fake(5)) == 1 and copy(f, v=fake(6)) == 1 and copy(f, k=fake(4)) == 1  # over the indices, the table
    assert copy(f, cache(True), k=fake(2)) == 1                                           # over the scales


@pytest.mark.parametrize("kw,code", [
    (dict(hq=0), 1), (dict(hq=6), 1), (dict(hq=4 * 129), 2), (dict(q_len=0), 1), (dict(q_len=17), 2), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(lens=None), 1), (dict(q=None), 1), (dict(o=None), 1), (dict(ws=None), 1), (dict(bytes=0), 4),
    (dict(q=fake(6) + ODD), 3), (dict(lse=fake(8) + 4), 3), (dict(ws=fake(9) + ODD), 3), (dict(lens=fake(5) + 2), 3), (dict(qts=132), 2),
    (dict(ohs=-8), 1), (dict(ots=64), 1),
    (dict(o=fake(6)), 1), (dict(o=fake(6) + 2 * DIM), 1), (dict(o=fake(0)), 1), (dict(o=fake(4)), 1), (dict(o=fake(5)), 1),
    (dict(lse=fake(7)), 1), (dict(lse=fake(6) + 64), 1), (dict(lse=fake(5)), 1), (dict(lse=fake(1)), 1),
    (dict(ws=fake(8)), 1), (dict(ws=fake(7)), 1), (dict(ws=fake(4)), 1), (dict(ws=fake(0)), 1)])
def test_decode_refusals(kw, code):
    assert decode(**kw) == code


def test_decode_of_no_sequences_and_sizes():
    assert decode(t=table(n_seqs=0, pages=None), lens=None, q=None, o=None, lse=None, ws=None, bytes=0) == 0
    assert size(n_seqs=-1)[0] == 1 and size(n_seqs=65537)[0] == 2 and size(hq=6)[0] == 1 and size(q_len=17)[0] == 2
    assert up.lib().upipe_attn_decode_workspace_size(ctypes.byref(cache()), 1, 8, 1, None) == 1
    # nothing that grows with the cache's length or the number of sequences
    assert size(n_seqs=1)[1] == size(cache(n_pages=1 << 20), n_seqs=1)[1] <= 1 << 24


def test_binding_refuses():
    k = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: up.KVCache(k, k.clone()), lambda: up.KVCache(k[0], k[0]), lambda: up.KVCache(k.float(), k.float()),
                 lambda: up.KVCache(k, k, torch.zeros(2, 2, 16), None),
                 lambda: up.KVCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn))):
        with pytest.raises(ValueError):
            call()


def test_codes_of_bf16_rows_do_not_hang_on_the_quotients_last_bits():
    """For every bf16 magnitude over a scale that a bf16 magnitude gives: the quotient lowered and raised by 2^-42 of itself (the
    kernel's is within 2^-43) rounds to the same code, by way of fp32 as the definition has it."""
    top = torch.arange(128, 256, dtype=torch.float32)
    scale = top * torch.tensor(1.0 / 448.0, dtype=torch.float32)
    x = torch.arange(128, 256, dtype=torch.float64)
    for shift in range(24):                              # below that every code is zero
        q = (x / 2.0 ** shift)[None, :] / scale.double()[:, None]
        q = torch.where((x / 2.0 ** shift)[None, :] <= top.double()[:, None], q, torch.zeros_like(q))
        low, high = ((q * (1 + d)).float().to(torch.float8_e4m3fn).view(torch.uint8) for d in (-2.0 ** -42, 2.0 ** -42))
        assert torch.equal(low, high)
