"""The decode kernel's division of work, on a model: the line of tiles, the warps' parts of it, the pieces of items that these
leave, their joins in a CTA and over CTAs.

The model follows the kernel's integer arithmetic step by step.  Checked for many batches: every tile of every item is computed
once, by warps in order; the pieces of an item that meet in a CTA are joined in order; what an item leaves in several CTAs
forms one chain from the CTA where it begins to the one that its first piece names as its last, and nothing else.
"""
import random

import pytest

TILE = 16


def tiles_of(n, cap):
    return (min(max(n, 0), cap) + TILE - 1) // TILE


def next_seq(lens, b):
    """The kernel's search: the next sequence with keys (its length may pass the table; an empty table is dealt with apart)."""
    b += 1
    while b < len(lens) and lens[b] <= 0:
        b += 1
    return b if b < len(lens) else None


def warp_parts(lens, hkv, cap, ctas, warps, end):
    """[cta][warp] -> (first unit, units, unit after) of the line, with the total and the number of parts."""
    units = [tiles_of(n, cap) + end if tiles_of(n, cap) else 0 for n in lens]
    total = sum(units) * hkv
    parts = max((total + warps - 1) // warps, 1) if total < ctas * warps else ctas
    out = []
    for x in range(ctas):
        t0, t1 = (total * x // parts, total * (x + 1) // parts) if x < parts else (0, 0)
        row = []
        for w in range(warps):
            first = t0 + (t1 - t0) * w // warps
            left = t0 + (t1 - t0) * (w + 1) // warps - first
            row.append((first, left, first + left))
        out.append(row)
    return units, total, parts, out


def walk(lens, hkv, cap, ctas, warps, end):
    """Runs every warp; returns the tiles in order, whole items, and each CTA's pieces."""
    units, total, parts, plan = warp_parts(lens, hkv, cap, ctas, warps, end)
    upto, s = [], 0
    for u in units:
        s += u
        upto.append(s)
    seen, whole, pieces = [], [], []
    for x in range(ctas):
        cta = []
        for w in range(warps):
            first, left, after = plan[x][w]
            head = tail = None
            if left > 0:
                b = next(i for i, u in enumerate(upto) if u > first // hkv)
                n = units[b]
                rest = first - (upto[b] - n) * hkv
                hk, t = rest // n, rest % n
                if t >= n - end:                       # within an item's end
                    left -= n - t
                    t, hk = 0, hk + 1
                    if hk == hkv:
                        hk, b = 0, next_seq(lens, b)
                        if b is None:
                            left = 0
                while left > 0:
                    begin, cn = t, tiles_of(lens[b], cap)
                    while True:
                        seen.append((b, hk, t))
                        left -= 1
                        t += 1
                        if not (left > 0 and t < cn):
                            break
                    item = b * hkv + hk
                    if t == cn and begin == 0:
                        whole.append(item)
                    elif t == cn:
                        assert head is None
                        head = (item, begin, t)
                    else:
                        assert tail is None and left == 0
                        last = (after + cn - t) * parts + total - 1
                        tail = (item, begin, t, last // total - 1)
                    if t == cn:
                        left -= end
                        if left > 0:
                            t, hk = 0, hk + 1
                            if hk == hkv:
                                hk, b = 0, next_seq(lens, b)
                                assert b is not None
            cta += [head, tail]
        pieces.append(cta)
    return seen, whole, pieces


def join(pieces):
    """Runs of a CTA's pieces, then chains over CTAs: {item: tile ranges in the order of the joins}."""
    done, metas = {}, []
    for cta in pieces:
        ends_item = leaves = None
        runs = []
        for p in (p for p in cta if p is not None):
            if runs and runs[-1][0][0] == p[0]:
                runs[-1].append(p)
            else:
                runs.append([p])
        for run in runs:
            begins, ends = run[0][1] == 0, len(run[-1]) == 3
            span = [(q[1], q[2]) for q in run]
            if begins and ends:
                assert run[0][0] not in done
                done[run[0][0]] = span
            elif ends:
                assert ends_item is None
                ends_item = (run[0][0], span)
            else:
                assert leaves is None
                leaves = (run[0][0], begins, run[-1][3], span)
        metas.append((ends_item, leaves))
    used = set()
    for x, (_, leaves) in enumerate(metas):
        if leaves is None or not leaves[1]:
            continue
        item, _, last, span = leaves
        for y in range(x + 1, last):
            assert metas[y][1][0] == item and not metas[y][1][1]
            span = span + metas[y][1][3]
            used.add((y, 1))
        assert metas[last][0][0] == item
        used |= {(x, 1), (last, 0)}
        assert item not in done
        done[item] = span + metas[last][0][1]
    assert used == {(x, i) for x, m in enumerate(metas) for i in range(2) if m[i] is not None}  # nothing is left over
    return done


def check(lens, hkv, cap, ctas, warps, end):
    seen, whole, pieces = walk(lens, hkv, cap, ctas, warps, end)
    want = [(b, h, t) for b, n in enumerate(lens) for h in range(hkv) for t in range(tiles_of(n, cap))]
    assert seen == want
    done = join(pieces)
    items = {b * hkv + h: tiles_of(n, cap) for b, n in enumerate(lens) for h in range(hkv) if tiles_of(n, cap)}
    assert set(whole) | set(done) == set(items) and not set(whole) & set(done) and len(whole) == len(set(whole))
    for item, span in done.items():
        at = 0
        for a, b in span:
            assert a == at and b > a
            at = b
        assert at == items[item]


@pytest.mark.parametrize("warps,end", [(8, 2), (8, 4), (16, 4)])
@pytest.mark.parametrize("seed", range(8))
def test_random_batches(seed, warps, end):
    rng = random.Random(seed)
    for _ in range(40):
        n = rng.choice([1, 1, 2, 5, 31, 32, 33, 64, 65, 130])
        top = rng.choice([1, 16, 17, 100, 700, 5000])
        lens = [rng.choice([0, -3, rng.randint(0, top), rng.randint(0, top)]) for _ in range(n)]
        cap = rng.choice([1 << 30, 1 << 30, 16 * rng.randint(1, 40)])
        check(lens, rng.choice([1, 2, 3, 8]), cap, rng.choice([1, 2, 7, 38, 152]), warps, end)


@pytest.mark.parametrize("lens,hkv", [([0], 1), ([0] * 40, 2), ([1], 1), ([1 << 18], 1), ([1 << 16, 1], 2), ([5] * 300, 1), ([16 * 152 * 8], 1),
                                      ([16 * 152 * 8 - 1], 1), ([16 * 152 * 8 + 1], 1)])
def test_edges(lens, hkv):
    for warps, end in ((8, 2), (16, 4)):
        check(lens, hkv, 1 << 30, 152, warps, end)


def test_parts_are_even():
    """No warp has more than a unit more than another, whatever the lengths."""
    rng = random.Random(3)
    lens = [int(10 ** rng.uniform(0, 4.5)) for _ in range(200)]
    _, _, parts, plan = warp_parts(lens, 8, 1 << 30, 152, 16, 4)
    counts = [left for row in plan[:parts] for _, left, _ in row]
    assert max(counts) - min(counts) <= 2
