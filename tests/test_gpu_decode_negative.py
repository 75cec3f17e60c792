"""Decode with lengths at the lower end of 32 bits: every negative length is one of an empty sequence."""
import math

import pytest
import torch

from test_gpu_kv import KINDS, check_decode, gen, run_decode, setup, widened

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


LOWEST = -2 ** 31


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_len", [1, 2, 16])
@pytest.mark.parametrize("hq,columns", [(2, 0), (2, 3), (2, 4000), (8, 100000)])
def test_lowest_lengths(kind, q_len, hq, columns):
    lens = [LOWEST, 33, LOWEST + 1, LOWEST + 14, LOWEST + 15, -1, 0, 40]
    c, table, q = setup(kind, lens, hq, 1, 128, 16, q_len)
    table = widened(table, columns, gen(1))
    check_decode(c, q, table, lens, q_len=q_len)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seqs", [3, 200, 3000])
def test_lowest_lengths_without_a_table(kind, seqs):
    c, table, q = setup(kind, [16], 4, 1, 64, 16, 4)
    q = q.repeat(1, seqs, 1)
    table = table[:, :0].expand(seqs, 0).contiguous()
    o, lse = run_decode(c, q, table, [LOWEST + i % 16 for i in range(seqs)], q_len=4)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
