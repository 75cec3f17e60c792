"""Which places of the values beside the keys a paged cache takes, checked without a GPU: a cache is refused where a row of one tensor
shares bytes with a row of the other, and taken where none does, whatever the strides.  The answer is compared with that of a
set of all units that the rows cover."""
import ctypes
import itertools
import random

import pytest

import long_context_attention_upipe_gb300 as up

BASE = 1 << 44


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


def code(pages, heads, tokens, strides, v, e4m3=False, scales=None, vs=0):
    """Status of a cache of rows of one unit (64 elements); strides and the values' place in units, scales' in numbers."""
    unit = 64
    size = unit if e4m3 else 2 * unit
    ss = scales or (0, 0, 0)
    far = 1 << 46
    d = up.KVCacheDesc(BASE, BASE + v * size, far if e4m3 else None, far + 4 * vs if e4m3 else None, pages, strides[0] * unit,
                       strides[1] * unit, strides[2] * unit, *ss, tokens, heads, 64, int(e4m3))
    n = ctypes.c_size_t(0)
    return up.lib().upipe_attn_decode_workspace_size(ctypes.byref(d), 1, heads, 1, ctypes.byref(n))


def cover(pages, heads, tokens, strides, at=0):
    return [at + p * strides[0] + h * strides[1] + t * strides[2] for p, h, t in itertools.product(range(pages), range(heads), range(tokens))]


def nested(n, s):
    """Every level's stride, from the largest down, is at least what the levels below span: what the rule on one tensor asks."""
    order = sorted((x for x in zip(s, n) if x[1] > 1), reverse=True)
    return all(s >= 1 + sum((m - 1) * t for t, m in order[i + 1:]) for i, (s, _) in enumerate(order))


@pytest.mark.parametrize("name,pages,heads,strides,v", [
    ("values one page behind the keys, three units to a head", 4, 2, (8 * 16, 3 * 16, 1), 8 * 16),
    ("values a page and more behind", 4, 2, (4 * 16, 19, 1), 4 * 16),
    ("values at the second head's place", 1, 2, (0, 2 * 16 + 1, 2), 2 * 16 + 1),
    ("values at the second head's second token", 1, 2, (0, 2 * 16 + 1, 2), 2 * 16 + 3)])
def test_layouts_that_meet(name, pages, heads, strides, v):
    a = cover(pages, heads, 16, strides)
    assert len(set(a)) == len(a) and set(a) & set(cover(pages, heads, 16, strides, v))
    assert code(pages, heads, 16, strides, v) == 1, name
    assert code(pages, heads, 16, strides, -v) == 1, name
    assert code(pages, heads, 16, [x * 2 for x in strides], 2 * v, True, (1 << 20, 1 << 10, 1), 1 << 30) == 1, name
    # the scales' tensors by the same rule
    assert code(pages, heads, 16, (1 << 20, 1 << 10, 1), 1 << 30, True, strides, v) in (1, 3)
    assert code(pages, heads, 16, (1 << 20, 1 << 10, 1), 1 << 30, True, [4 * x for x in strides], 4 * v) == 1, name


@pytest.mark.parametrize("seed", range(6))
def test_random_layouts(seed):
    rng = random.Random(seed)
    met = apart = 0
    while met < 150 or apart < 150:
        n = (rng.choice([1, 2, 3, 5]), rng.choice([1, 2, 4]), 16)
        order = rng.sample(range(3), 3)
        s, span = [0, 0, 0], 1
        for i in order:
            s[i] = span + rng.choice([0, 0, 1, 2, 5, span, 2 * span])
            span += (n[i] - 1) * s[i]
        assert nested(n, s)
        a = cover(*n, s)
        v = rng.choice([rng.randint(-span - 2, span + 2), rng.choice(s) * rng.randint(-3, 3) + rng.randint(-1, 1)])
        meets = bool(set(a) & set(cover(*n, s, v)))
        met, apart = met + meets, apart + (not meets)
        assert code(*n, s, v) == (1 if meets else 0), (n, s, v)
        # rows of scales: 4 numbers (16 bytes) to a unit, since both tensors begin on 16 bytes
        assert code(*n, (1 << 20, 1 << 12, 1), 1 << 30, True, [4 * x for x in s], 4 * v) == (1 if meets else 0), (n, s, v)


def test_rows_that_overlap_in_part():
    """Half a unit off: rows share bytes although no two begin at one place."""
    for e4m3, size in ((False, 128), (True, 64)):
        d = [BASE, BASE + size // 2, 1 << 46 if e4m3 else None, 1 << 47 if e4m3 else None, 1, 0, 0, 128, 0, 0, 1, 16, 1, 64, int(e4m3)]
        n = ctypes.c_size_t(0)
        for v, want in ((size // 2, 1), (size, 0), (3 * size // 2, 1), (16 * 2 * size - size, 0), (16 * 2 * size - 3 * size // 2, 1), (-size // 2, 1),
                        (-size, 0)):
            d[1] = BASE + v
            assert up.lib().upipe_attn_decode_workspace_size(ctypes.byref(up.KVCacheDesc(*d)), 1, 1, 1, ctypes.byref(n)) == want, (e4m3, v)
