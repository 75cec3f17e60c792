"""Decode whose waits run out, in every form of the kernels."""
import pytest
import torch

import long_context_attention_upipe_gb300 as up
from test_gpu_kv import run_decode, setup, setup_many, widened, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


@pytest.fixture(autouse=True)
def usual_limit():
    yield
    up.set_wait_limit_ns(0)


FORMS = {  # lengths, query heads, key heads, head_dim, page, q_len, columns that the table has beside: each way through the kernels
    "cta": ([1, 17, 500], 4, 1, 128, 16, 1, 0), "cluster": ([2000], 4, 1, 128, 64, 1, 0), "clusters": ([2000, 40, 0, 900], 8, 2, 128, 64, 1, 0),
    "whole": ([(i * 37) % 300 for i in range(200)], 2, 1, 64, 16, 1, 0), "line": ([30000, 12, 0, 777], 8, 2, 128, 32, 1, 0),
    "many": ([(i * 37) % 300 for i in range(700)], 2, 1, 64, 16, 1, 0),
    "warps": ([60000, 40], 8, 2, 128, 16, 1, 100000), "rows": ([30001, 100], 8, 2, 64, 32, 4, 0), "blocks": ([6000, 100], 40, 2, 128, 32, 2, 0),
    "wide32": ([30000, 0, 129], 24, 1, 128, 16, 1, 100000), "wide64": ([30000, 0, 129], 20, 1, 64, 16, 2, 100000),
    "wide64 of 128": ([30000, 40, 900], 48, 2, 128, 64, 1, 100000),
}
CASES = [(k, f) for k in ("bf16", "e4m3") for f in FORMS if k == "bf16" or f[:4] != "wide"]


def case(kind, form):
    lens, hq, hkv, dh, size, q_len, more = FORMS[form]
    c, table, q = setup_many(kind, lens, hq, hkv, dh, size) if len(lens) > 300 else setup(kind, lens, hq, hkv, dh, size, q_len)
    if more:
        table = widened(table, more, gen(1))
    return c, table, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), q_len


@pytest.mark.parametrize("kind,form", CASES)
def test_a_call_after_one_that_gave_up(kind, form):
    """What a call that gave up leaves in shared memory is nothing to the next one."""
    c, table, q, ln, q_len = case(kind, form)
    want, wl = run_decode(c, q, table, ln, q_len=q_len)
    ws = torch.full((up.decode_workspace_bytes(c, table.shape[0], q.shape[0], q_len),), 0xff, dtype=torch.uint8, device="cuda")
    lost, good = (torch.full_like(q, 55.0) for _ in range(2))
    for limit in (1, 2, 3, 5):
        lse = torch.empty(q.shape[:2], device="cuda")
        good.fill_(55.0)
        up.set_wait_limit_ns(limit)
        up.decode(c, q, table, ln, lost, ws)
        up.set_wait_limit_ns(0)
        up.decode(c, q, table, ln, good, ws, lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(good, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind,form", CASES)
def test_waits_run_out(kind, form):
    """Limits below 64 ns: a wait for the first tile of every queue runs out (1), or for a later one.  A row is all NaN, or what it is with the usual
    limit."""
    c, table, q, ln, q_len = case(kind, form)
    want, wl = run_decode(c, q, table, ln, q_len=q_len)
    seen = ~((want == 0).all(-1) & (wl == -float("inf")))
    for limit in (1, 2, 3, 4, 5, 6, 63):
        up.set_wait_limit_ns(limit)
        o, lse = run_decode(c, q, table, ln, q_len=q_len)
        up.set_wait_limit_ns(0)
        torch.cuda.synchronize()
        lost = o.isnan().any(-1)
        assert torch.equal(o.isnan().all(-1), lost) and torch.equal(lse.isnan(), lost) and not bool((lost & ~seen).any())
        assert torch.equal(o[~lost], want[~lost]) and torch.equal(lse[~lost], wl[~lost])
        if limit == 1:
            assert torch.equal(lost, seen)
    o, lse = run_decode(c, q, table, ln, q_len=q_len)
    assert torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind,form", [("bf16", "line"), ("bf16", "clusters"), ("bf16", "wide64")])
def test_calls_that_gave_up_in_a_graph(kind, form):
    """The limit is the one at the capture: every replay gives up, and the call behind it in the same workspace does not."""
    c, table, q, ln, q_len = case(kind, form)
    want, wl = run_decode(c, q, table, ln, q_len=q_len)
    ws = torch.full((up.decode_workspace_bytes(c, table.shape[0], q.shape[0], q_len),), 0xff, dtype=torch.uint8, device="cuda")
    lost, good, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        up.set_wait_limit_ns(1)
        up.decode(c, q, table, ln, lost, ws)
        up.set_wait_limit_ns(0)
        up.decode(c, q, table, ln, good, ws, lse=lse)
    for _ in range(5):
        lost.zero_()
        good.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(good, want) and torch.equal(lse, wl) and bool(lost.isnan().all(-1)[wl > -float("inf")].all())
