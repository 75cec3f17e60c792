"""The warp-specialised kernels of the 8-bit product and of the norm's backward pass, on a model.

Every role is an actor that waits on mbarriers (phases with parities, arrivals and bytes, as the hardware counts
them), loads land and MMAs run in their own time, and a random schedule interleaves everything.  What lies in a stage,
an accumulator or a scale slot is the turn that it belongs to, so a value that was built from anything else is known.
Any wait may run out: its actor gives up, and so does every other actor of its block that finds nothing to do.  Checked:
  - with no wait running out every schedule ends, and every output is right (no barrier phase is missed or mixed up);
  - with waits that run out in any role every schedule still ends, and no output that is not NaN is wrong;
  - at the end nothing is in flight towards shared memory or an accumulator that the block leaves behind.
`old` holds the rules that a role may break (arrive although it gave up; leave without waiting for its copies): the
model finds the wrong values and the copies that these let through.
"""
import random

import pytest


class Bar:
    """mbarrier: `count` arrivals and the bytes they announce complete a phase."""

    def __init__(self, count):
        self.count, self.left, self.tx, self.phase = count, count, 0, 0

    def _turn(self):
        if self.left == 0 and self.tx == 0:
            self.phase += 1
            self.left = self.count

    def arrive(self, tx=0):
        assert self.left > 0, "more arrivals than the phase takes"
        self.tx += tx
        self.left -= 1
        self._turn()

    def complete(self, n=1):
        self.tx -= n
        self._turn()

    def done(self, parity):
        return (self.phase & 1) != parity


class Ring:
    """Position in a ring and the parity of its waits."""

    def __init__(self, n, parity):
        self.n, self.at, self.parity = n, 0, parity

    def step(self):
        self.at += 1
        if self.at == self.n:
            self.at, self.parity = 0, self.parity ^ 1


class World:
    def __init__(self, rng, give_up, blocks, old=()):
        self.rng, self.give_up, self.old = rng, give_up, old
        self.abort = [False] * blocks      # the blocks' abort flags
        self.flight = []                   # loads on their way: functions that land them
        self.queue = []                    # MMAs and commits, in order
        self.pace = rng.choice([0.01, 0.1, 0.25])   # how fast loads and MMAs are beside the actors
        self.wrong, self.nan, self.right = 0, 0, 0

    def store(self, ok, value_right):
        if not ok:
            self.nan += 1
        elif value_right:
            self.right += 1
        else:
            self.wrong += 1

    def run(self, actors):
        """Steps random actors until all have ended; an actor yields (block, barrier, parity), or ("drain", barrier, parity),
        whose limit runs out only once nothing is on its way any more (a second against microseconds)."""
        todo = {i: (a, next(a, None)) for i, a in enumerate(actors)}
        todo = {i: x for i, x in todo.items() if x[1] is not None}
        idle = 0
        while todo:
            r = self.rng.random()
            if r < self.pace and self.flight:
                self.flight.pop(self.rng.randrange(len(self.flight)))()
                idle = 0
                continue
            if self.pace <= r < 2 * self.pace and self.queue:
                self.queue.pop(0)()
                idle = 0
                continue
            i = self.rng.choice(list(todo))
            actor, (block, bar, parity) = todo[i]
            if bar.done(parity):
                answer = True
            elif block == "threads":                # a barrier of threads: nobody gives up on it
                answer = None
            elif block == "drain":
                answer = False if not self.flight and not self.queue and idle > 200 else None
            elif self.abort[block] and self.rng.random() < 0.02:
                answer = False
            elif self.rng.random() < self.give_up or (idle > 400 and self.give_up):
                self.abort[block] = True
                answer = False
            else:
                answer = None
            if answer is None:
                idle += 1
                assert self.give_up or idle < 5000, "nobody can go on"
                continue
            idle = 0
            try:
                todo[i] = (actor, actor.send(answer))
            except StopIteration:
                del todo[i]


def last_turns(n, ring):
    return range(max(0, n - ring), n)


# ------------------------------------------------------------------------------------------------
# product: CTA pairs (many rows), or one CTA (few rows)
# ------------------------------------------------------------------------------------------------

def product(w, pair, tiles, nkb, stages, accs, group, slots, warps=2):
    """`pair`: two CTAs, the even one issues for both and its accumulators are handed back by both; scaling warps wait on
    the stages' ring.  Otherwise one CTA whose accumulators have barriers of their own.  All indices are turns: block of K
    `kb` of tile `t` is turn t * nkb + kb."""
    n_cta = 2 if pair else 1
    full = Bar(1)  # replaced below; in the pair only the even CTA's are used
    full = [Bar(1) for _ in range(stages)]
    empty = [[Bar(1) for _ in range(stages)] for _ in range(n_cta)]
    acc_full = [Bar(1) for _ in range(accs)]
    acc_empty = [Bar(n_cta * warps) for _ in range(accs)]
    sc_full = [[Bar(2) for _ in range(slots)] for _ in range(n_cta)]
    sc_empty = [[Bar(warps) for _ in range(slots)] for _ in range(n_cta)]
    stage = [[None] * stages for _ in range(n_cta)]
    acc = [[None] * accs for _ in range(n_cta)]
    scales = [[[None, None] for _ in range(slots)] for _ in range(n_cta)]

    def producer(c):
        ring, ok, n = Ring(stages, 1), True, 0
        for t in range(tiles):
            if not ok:
                break
            for kb in range(nkb):
                ok = (yield (c, empty[c][ring.at], ring.parity)) and ok
                if ok:
                    s, turn = ring.at, t * nkb + kb
                    if c == 0:
                        full[s].arrive(tx=n_cta)

                    def land(s=s, turn=turn):
                        stage[c][s] = turn
                        full[s].complete()
                    w.flight.append(land)
                    n += 1
                ring.step()
        if "leave" not in w.old:
            for i in last_turns(n, stages):
                if pair:
                    yield ("drain", empty[c][i % stages], i // stages & 1)
                else:
                    yield ("drain", full[i % stages], i // stages & 1)

    def issuer():
        ring, buf, ok, n = Ring(stages, 0), Ring(accs, 1), True, 0
        for t in range(tiles):
            if not ok:
                break
            for kb in range(nkb):
                ok = (yield (0, full[ring.at], ring.parity)) and ok
                ok = (yield (0, acc_empty[buf.at], buf.parity)) and ok
                if ok:
                    def mma(s=ring.at, b=buf.at, turn=t * nkb + kb):
                        for c in range(n_cta):
                            acc[c][b] = turn if all(stage[k][s] == turn for k in range(n_cta)) else "mixed"
                    w.queue.append(mma)
                    if not pair:
                        w.queue.append(acc_full[buf.at].arrive)
                    for c in range(n_cta):
                        w.queue.append(empty[c][ring.at].arrive)
                    n += 1
                ring.step()
                buf.step()
        if not pair and "leave" not in w.old:
            for i in last_turns(n, stages):
                yield ("drain", empty[0][i % stages], i // stages & 1)
            for i in last_turns(n, accs):
                yield ("drain", acc_full[i % accs], i // accs & 1)

    def fetcher(c, half):
        ring, ok = Ring(slots, 1), True
        for t in range(tiles):
            for kb in range(0, nkb, group):
                ok = (yield (c, sc_empty[c][ring.at], ring.parity)) and ok
                if ok:
                    scales[c][ring.at][half] = (t, kb // group)
                elif "arrive" not in w.old:
                    return
                sc_full[c][ring.at].arrive()
                ring.step()

    def scaler(c):
        slot, st, buf, ok = Ring(slots, 0), Ring(stages, 0), Ring(accs, 0), True
        for t in range(tiles):
            right = True
            for kb in range(nkb if ok or "arrive" in w.old else 0):
                last = kb % group == group - 1 or (pair and kb + 1 == nkb)
                if kb % group == 0:
                    ok = (yield (c, sc_full[c][slot.at], slot.parity)) and ok
                sc = list(scales[c][slot.at])
                if pair:
                    ok = (yield (c, empty[c][st.at], st.parity)) and ok
                    st.step()
                else:
                    ok = (yield (c, acc_full[buf.at], buf.parity)) and ok
                right = right and acc[c][buf.at] == t * nkb + kb and sc == [(t, kb // group)] * 2
                if ok or "arrive" in w.old:
                    if last:
                        sc_empty[c][slot.at].arrive()
                    acc_empty[buf.at].arrive()
                if last:
                    slot.step()
                buf.step()
            w.store(ok, right)

    actors = [issuer()]
    for c in range(n_cta):
        actors += [producer(c), fetcher(c, 0), fetcher(c, 1)] + [scaler(c) for _ in range(warps)]
    w.run(actors)
    # the loads and MMAs that are left run into memory that the CTAs gave back
    return n_cta * warps * tiles


# stages, accumulators, blocks of K of a group of scales, groups: as csrc/gemm_fp8.cu has them
PAIR = [(5, 2, 8, 2), (6, 2, 8, 2), (6, 3, 8, 2), (6, 4, 8, 2)]
FEW = [(5, 8, 4, 4), (4, 8, 4, 4), (3, 4, 4, 4), (4, 4, 4, 4)]
NKB = [1, 2, 3, 5, 7, 8, 9, 16, 17, 18, 33]


def drain(w):
    """Everything that is still on its way, and whether anything was."""
    return bool(w.flight or w.queue)


def constants():
    """The products' ring sizes, from their source."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_attention_upipe_gb300", "csrc",
                            "gemm_fp8.cu")).read()
    return {k: re.search(k + r" = ([^;]+);", src).group(1) for k in ("STAGES", "NBUF", "kScSlots", "ACCS")}, src


def test_the_model_has_the_kernels_rings():
    got, src = constants()
    assert got["STAGES"] == "TN == 16 ? 5 : TN == 64 ? 3 : 4" and got["NBUF"] == "TN <= 32 ? 8 : 4"
    assert "STAGES = NCH == 8 ? 5 : 6" in src and got["ACCS"] == "512 / BN" and "kScSlots = 2, kScGroup = 8" in src
    for nch in (4, 5, 6, 7, 8):
        assert (5 if nch == 8 else 6, 512 // (32 * nch), 8, 2) in PAIR


@pytest.mark.parametrize("rings", PAIR)
def test_pair_product_ends_and_is_right(rings):
    rng = random.Random(1)
    for _ in range(150):
        w = World(rng, 0.0, 2)
        n = product(w, True, rng.choice([1, 2, 3]), rng.choice(NKB), *rings)
        assert w.right == n and not w.nan and not drain(w)


@pytest.mark.parametrize("rings", FEW)
def test_few_rows_product_ends_and_is_right(rings):
    rng = random.Random(2)
    for _ in range(150):
        w = World(rng, 0.0, 1)
        n = product(w, False, 1, rng.choice(NKB), *rings)
        assert w.right == n and not w.nan and not drain(w)


def with_waits_that_run_out(pair, rings, old, runs, seed):
    """Stored outputs that are wrong, NaN, right, over many schedules; schedules that left something in flight."""
    rng = random.Random(seed)
    wrong = nan = right = left = 0
    for _ in range(runs):
        w = World(rng, rng.choice([0.0005, 0.003, 0.02]), 2 if pair else 1, old)
        tiles = rng.choice([1, 2, 3]) if pair else 1
        try:
            n = product(w, pair, tiles, rng.choice(NKB), *rings)
            assert w.wrong + w.nan + w.right == n
        except AssertionError:
            if not old:
                raise
            w.wrong += 1                    # the old rules even overrun a barrier
        wrong, nan, right, left = wrong + w.wrong, nan + w.nan, right + w.right, left + drain(w)
    return wrong, nan, right, left


@pytest.mark.parametrize("pair,rings", [(True, r) for r in PAIR] + [(False, r) for r in FEW])
def test_product_stores_nan_or_the_right_value_and_leaves_nothing_in_flight(pair, rings):
    wrong, nan, right, left = with_waits_that_run_out(pair, rings, (), 300, 3)
    assert nan > 0 and right > 0
    assert wrong == 0 and left == 0


@pytest.mark.parametrize("rings", FEW)
def test_a_producer_that_just_leaves_has_copies_in_flight(rings):
    assert with_waits_that_run_out(False, rings, ("leave",), 300, 5)[3] > 0


@pytest.mark.parametrize("pair,rings", [(True, PAIR[0]), (False, FEW[1])])
def test_an_arrival_of_a_role_that_gave_up_lets_wrong_values_through(pair, rings):
    wrong, _, _, _ = with_waits_that_run_out(pair, rings, ("arrive", "leave"), 300, 4)
    assert wrong > 0


# ------------------------------------------------------------------------------------------------
# norm backward: rows ahead in a ring
# ------------------------------------------------------------------------------------------------

def norm_ring(w, rows, stages, warps=3):
    full, empty = [Bar(1) for _ in range(stages)], [Bar(warps) for _ in range(stages)]
    named = Bar(warps)
    stage = [None] * stages
    row_ok, row_right = [True] * rows, [True] * rows     # what the row's sum is made of
    dw_ok = [True] * warps

    def producer():
        ring, ok, n = Ring(stages, 1), True, 0
        for row in range(rows):
            ok = (yield (0, empty[ring.at], ring.parity)) and ok
            if not ok:
                break
            full[ring.at].arrive(tx=1)

            def land(s=ring.at, row=row):
                stage[s] = row
                full[s].complete()
            w.flight.append(land)
            n += 1
            ring.step()
        if "leave" not in w.old:
            for i in last_turns(n, stages):
                yield ("drain", full[i % stages], i // stages & 1)

    def worker(k):
        ring, ok, turn = Ring(stages, 0), True, 0
        for row in range(rows):
            ok = (yield (0, full[ring.at], ring.parity)) and ok
            row_right[row] &= stage[ring.at] == row
            if ok or "stale" in w.old:
                empty[ring.at].arrive()
            else:
                row_ok[row] = False                      # NaN in the sum
            ring.step()
            named.arrive()
            yield ("threads", named, turn)
            turn ^= 1
            if "stale" in w.old and not ok:
                w.wrong += 1                             # its part of the row keeps what was there
            else:
                w.store(row_ok[row], row_right[row])
        named.arrive()
        yield ("threads", named, turn)
        dw_ok[k] = not w.abort[0]

    w.run([producer()] + [worker(k) for k in range(warps)])
    return warps * rows, dw_ok


def norm_with_waits_that_run_out(stages, old, runs, seed):
    rng = random.Random(seed)
    wrong = nan = right = left = 0
    for _ in range(runs):
        w = World(rng, rng.choice([0.0005, 0.003, 0.02]), 1, old)
        try:
            n, dw_ok = norm_ring(w, rng.choice([1, 2, 5, 9, 20]), stages)
            assert w.wrong + w.nan + w.right == n
            assert len(set(dw_ok)) == 1 and (not w.nan or not dw_ok[0])    # NaN in a row: NaN in every column of dw
        except AssertionError:
            if not old:
                raise
            w.wrong += 1
        wrong, nan, right, left = wrong + w.wrong, nan + w.nan, right + w.right, left + drain(w)
    return wrong, nan, right, left


@pytest.mark.parametrize("stages", [3, 5, 8])
def test_norm_ring_ends_and_is_right(stages):
    rng = random.Random(6)
    for _ in range(200):
        w = World(rng, 0.0, 1)
        n, dw_ok = norm_ring(w, rng.choice([1, 2, 5, 9, 20]), stages)
        assert w.right == n and all(dw_ok) and not drain(w)


@pytest.mark.parametrize("stages", [3, 5, 8])
def test_norm_ring_stores_nan_or_the_right_rows_and_leaves_nothing_in_flight(stages):
    wrong, nan, right, left = norm_with_waits_that_run_out(stages, (), 300, 7)
    assert nan > 0 and right > 0 and wrong == 0 and left == 0


def test_a_norm_producer_that_just_leaves_has_copies_in_flight():
    assert norm_with_waits_that_run_out(8, ("leave",), 600, 9)[3] > 0


def test_norm_ring_that_skips_rows_leaves_old_values():
    assert norm_with_waits_that_run_out(5, ("stale", "leave"), 300, 8)[0] > 0
