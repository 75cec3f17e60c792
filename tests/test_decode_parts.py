"""The decode kernels' other divisions of work, on a model: parts of the line that begin and end with items (many short items, one
launch), clusters of CTAs with an item each, and the larger tiles' line, where a CTA is the unit and each of its roles walks the line for
itself.

The model follows the kernels' integer arithmetic.  Checked: every tile is computed once and in order; parts of whole items leave no
piece to another CTA; all roles of a CTA walk the same tiles; what an item leaves in several CTAs is one chain, from the CTA where it
begins to the one that is named as its last.
"""
import random

import pytest

from test_decode_line import join, next_seq


def tiles_of(n, cap, tile):
    return (min(max(n, 0), cap) + tile - 1) // tile


class Place:
    """Where a place on the line lies: sequence, head, tile (which may be within the item's end), and the item's length there."""

    def __init__(self, units, hkv, place):
        upto = before = 0
        for b, n in enumerate(units):
            upto += n
            if upto > place // hkv:
                break
            before += n
        else:
            raise AssertionError("no such place")
        rest = place - before * hkv
        self.b, self.n = b, n
        self.hk = min(rest // n, hkv - 1)
        self.tile = rest - self.hk * n


def parts_of(total, ctas, warps):
    return max((total + warps - 1) // warps, 1) if total < ctas * warps else ctas


def walk_warp(lens, units, hkv, cap, first, left, end, tile=16):
    """The tiles of a warp's part and its pieces [(item, begin, end of the tiles, whether it ends the item)]."""
    seen, pieces = [], []
    if left <= 0:
        return seen, pieces
    at = Place(units, hkv, first)
    b, hk, t = at.b, at.hk, at.tile
    if t >= at.n - end:
        left -= at.n - t
        t, hk = 0, hk + 1
        if hk == hkv:
            hk, b = 0, next_seq(lens, b)
            if b is None:
                left = 0
    while left > 0:
        n, begin = tiles_of(lens[b], cap, tile), t
        count = min(left, n - t)
        seen += [(b, hk, t + i) for i in range(count)]
        left, t = left - count, t + count
        pieces.append((b * hkv + hk, begin, t, t == n))
        if t == n:
            left -= end
            if left > 0:
                t, hk = 0, hk + 1
                if hk == hkv:
                    hk, b = 0, next_seq(lens, b)
                    assert b is not None
    return seen, pieces


def whole_items(lens, hkv, cap, ctas, warps, end):
    units = [tiles_of(n, cap, 16) + end if tiles_of(n, cap, 16) else 0 for n in lens]
    total = sum(units) * hkv
    parts = parts_of(total, ctas, warps)
    seen = []
    for x in range(min(parts, ctas)):
        bounds = []
        for place in (total * x // parts, total * (x + 1) // parts):
            if place >= total:
                bounds.append(total)
                continue
            at = Place(units, hkv, place)
            bounds.append(place - at.tile + at.n if at.tile else place)
        t0, t1 = bounds
        assert t0 <= t1
        open_item = None
        for w in range(warps):
            first = t0 + (t1 - t0) * w // warps
            tiles, pieces = walk_warp(lens, units, hkv, cap, first, t0 + (t1 - t0) * (w + 1) // warps - first, end)
            seen += tiles
            for i, (item, begin, t, ends) in enumerate(pieces):
                # a piece goes on where the one before stopped, in this CTA, or begins its item; no more than two are not whole
                assert open_item == ((item, begin) if begin else None)
                assert i in (0, len(pieces) - 1) or (begin == 0 and ends)
                open_item = None if ends else (item, t)
        assert open_item is None
    assert seen == [(b, h, t) for b, n in enumerate(lens) for h in range(hkv) for t in range(tiles_of(n, cap, 16))]


def batch(rng, most, top):
    n = rng.choice([1, 2, 5, 31, 32, 33, 64, 65, 130, 200, 300][:most])
    return [rng.choice([0, -3, rng.randint(0, top), rng.randint(0, top), rng.randint(0, top)]) for _ in range(n)]


@pytest.mark.parametrize("warps,end", [(8, 2), (8, 4)])
@pytest.mark.parametrize("seed", range(6))
def test_parts_of_whole_items(seed, warps, end):
    rng = random.Random(seed)
    for _ in range(25):
        lens = batch(rng, 11, rng.choice([1, 16, 17, 100, 512]))
        whole_items(lens, rng.choice([1, 2, 3, 4]), rng.choice([1 << 30, 16 * rng.randint(1, 32)]), rng.choice([1, 7, 38, 76, 152]), warps, end)


@pytest.mark.parametrize("lens", [[], [0] * 200, [512] * 200, [0] * 77 + [512] + [0] * 99, [1] * 608, [512] + [1] * 300, [1] * 300 + [512]])
def test_parts_of_whole_items_at_the_edges(lens):
    for warps, end in ((8, 2), (8, 4)):
        whole_items(lens, 1, 512, 152, warps, end)
        whole_items(lens, 3, 512, 152, warps, end)


@pytest.mark.parametrize("share", [1, 2, 4, 8])
def test_clusters(share):
    """Tiles n me / (share warps) ..: all of them once, in the order of the CTAs' and warps' pieces."""
    for warps in (8,):
        for n in list(range(0, 260)) + [511, 512, 513]:
            of, at = share * warps, 0
            for me in range(of):
                first, left = n * me // of, n * (me + 1) // of - n * me // of
                assert first == at
                at += left
            assert at == n


# ------------------------------------------------------------------------------------------------
# tiles of 128 keys
# ------------------------------------------------------------------------------------------------

TILE, END = 128, 4


class Line:
    """A role's walk along a CTA's part (struct Line and its functions)."""

    def __init__(self, lens, units, hkv, cap, first, left):
        self.lens, self.hkv, self.cap, self.left = lens, hkv, cap, left
        at = Place(units, hkv, first)
        self.b, self.hk, self.tile = at.b, at.hk, at.tile
        self.n = max(tiles_of(lens[self.b], cap, TILE), 1)
        if self.tile >= self.n:
            self.left -= at.n - self.tile - END
            self.next()

    def next(self):
        self.left -= END
        if self.left <= 0:
            return
        self.tile, self.hk = 0, self.hk + 1
        if self.hk < self.hkv:
            return
        self.hk, self.b = 0, next_seq(self.lens, self.b)
        assert self.b is not None
        self.n = max(tiles_of(self.lens[self.b], self.cap, TILE), 1)

    def step(self, tiles):
        self.left -= tiles
        self.tile += tiles
        if self.tile >= self.n:
            self.next()

    def rest(self):
        return min(self.left, self.n - self.tile)


def large_tiles(lens, hkv, cap, ctas):
    units = [tiles_of(n, cap, TILE) + END if tiles_of(n, cap, TILE) else 0 for n in lens]
    total = sum(units) * hkv
    parts = parts_of(total, ctas, 1)
    seen, whole, pieces = [], [], []
    for x in range(ctas):
        head = tail = None
        if x < parts and total > 0:
            first, after = total * x // parts, total * (x + 1) // parts
            copies, made = [], []                  # tiles as the warps that bring and multiply them walk them, and as the weights' do
            w = Line(lens, units, hkv, cap, first, after - first)
            last_of_items = 0
            while w.left > 0:
                last_of_items += w.rest() == 1
                copies.append((w.b, w.hk, w.tile))
                w.step(1)
            w = Line(lens, units, hkv, cap, first, after - first)
            items = 0
            while w.left > 0:
                begin, tiles, n, item = w.tile, w.rest(), w.n, w.b * hkv + w.hk
                made += [(w.b, w.hk, begin + i) for i in range(tiles)]
                items += 1
                if begin + tiles < n:
                    assert tail is None and w.left == tiles
                    tail = (item, begin, begin + tiles, ((after + n - begin - tiles) * parts + total - 1) // total - 1)
                elif begin:
                    assert head is None and items == 1
                    head = (item, begin, n)
                else:
                    whole.append(item)
                w.step(tiles)
            assert copies == made and last_of_items == items
            seen += made
        pieces.append([head, tail])
    assert seen == [(b, h, t) for b, n in enumerate(lens) for h in range(hkv) for t in range(tiles_of(n, cap, TILE))]
    done = join(pieces)
    items = {b * hkv + h: tiles_of(n, cap, TILE) for b, n in enumerate(lens) for h in range(hkv) if tiles_of(n, cap, TILE)}
    assert set(whole) | set(done) == set(items) and not set(whole) & set(done) and len(whole) == len(set(whole))
    for item, span in done.items():
        at = 0
        for a, b in span:
            assert a == at and b > a
            at = b
        assert at == items[item]


@pytest.mark.parametrize("seed", range(8))
def test_large_tiles(seed):
    rng = random.Random(seed)
    for _ in range(40):
        lens = batch(rng, 9, rng.choice([1, 127, 128, 129, 1000, 40000]))
        large_tiles(lens, rng.choice([1, 2, 3, 8]), rng.choice([1 << 30, 1 << 30, 16 * rng.randint(1, 300)]), rng.choice([1, 2, 7, 38, 76, 152]))


@pytest.mark.parametrize("lens,hkv", [([0], 1), ([0] * 40, 2), ([1], 1), ([2 ** 22], 1), ([2 ** 20, 1], 2), ([5] * 300, 1), ([128 * 152], 1),
                                      ([128 * 148], 1), ([128 * 148 + 1], 1)])
def test_large_tiles_at_the_edges(lens, hkv):
    large_tiles(lens, hkv, 1 << 30, 152)
