"""A CPU model of fa_cache_prefix_kernel's roles (loaders, MMA thread, the two softmax
warpgroups) and of its ring of slots: every item of a share runs to its end, whatever
role goes first, and each MMA reads the key or value tile that it is meant to.  Roles
are generators that yield what they wait for; a schedule picks who goes next at random.
A planted mistake has to be found: the softmax looking for the next K of a tile that has
key tiles of its own, with few slots, waits for itself."""
import random

import pytest


class Stuck(Exception):
    pass


class Barrier:
    def __init__(self, count=1):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        """mbarrier.try_wait.parity: the phase with this parity has completed."""
        return (self.phase & 1) != parity


def run(items, NS, raw, vouched, seed, mistake=False):
    """items: (key tiles, two row tiles) each."""
    full, empty = [Barrier() for _ in range(NS)], [Barrier() for _ in range(NS)]
    q_full, s_full, p_full, o_done = ([Barrier() for _ in range(2)] for _ in range(4))
    raw_full, raw_empty = [Barrier() for _ in range(3)], [Barrier() for _ in range(3)]
    slot, log = [None] * NS, []  # unit that a slot holds; reads of the MMAs
    p_of = [None, None]          # which tile's weights P_X holds

    def units():
        for n, (tiles, _) in enumerate(items):
            for j in range(tiles):
                yield n, j, "K"
                yield n, j, "V"

    def copies():  # e4m3: the codes' copies, ahead of the conversion
        for u, _ in enumerate(units()):
            yield lambda u=u: raw_empty[u % 3].passed(((u // 3) & 1) ^ 1)
            raw_full[u % 3].arrive()

    def loader():
        for u, unit in enumerate(units()):
            if raw:
                yield lambda u=u: raw_full[u % 3].passed((u // 3) & 1)
            yield lambda u=u: empty[u % NS].passed(((u // NS) & 1) ^ 1)
            slot[u % NS] = unit
            full[u % NS].arrive()
            if raw:
                raw_empty[u % 3].arrive()

    def mma():
        sk, sv, pk, pv, nq, np = 0, 1, 0, 0, [0, 0], [0, 0]
        for n, (tiles, two) in enumerate(items):
            step, first_b = (1, 0) if two else (2, 1)

            def s_mma(x, j, first, wait, last):
                nonlocal sk, pk
                if first:
                    yield lambda: q_full[x].passed(nq[x])
                    nq[x] ^= 1
                if wait:
                    yield lambda: full[sk].passed(pk)
                log.append((slot[sk], (n, j, "K")))
                p_of[x] = None  # S_X lies where P_X was
                s_full[x].arrive()
                if last:
                    empty[sk].arrive()
                    sk += 2
                    if sk >= NS:
                        sk, pk = sk - NS, pk ^ 1

            def pv_mma(x, j, wait, last):
                nonlocal sv, pv
                yield lambda: p_full[x].passed(np[x])
                np[x] ^= 1
                if wait:
                    yield lambda: full[sv].passed(pv)
                log.append((slot[sv], (n, j, "V")))
                log.append((p_of[x], (n, j, x)))
                if last:
                    empty[sv].arrive()
                    sv += 2
                    if sv >= NS:
                        sv, pv = sv - NS, pv ^ 1

            yield from s_mma(0, 0, True, True, not two)
            if first_b < tiles:
                yield from s_mma(1, first_b, True, not two, True)
            for j0 in range(0, tiles, step):
                for x in range(2):
                    j = j0 + first_b if x else j0
                    if j >= tiles:
                        break
                    mine, last = x == 0 or not two, x == 1 or not two
                    yield from pv_mma(x, j, not vouched and mine, last)
                    if j + step < tiles:
                        yield from s_mma(x, j + step, False, (mistake is False and not two) if vouched else mine, last)
                    else:
                        o_done[x].arrive()

    def softmax(x):
        base = ns = no = 0
        for n, (tiles, two) in enumerate(items):
            step, c0 = (1, 0) if two else (2, x)
            mine = list(range(c0, tiles, step))
            if mine:
                q_full[x].arrive()
            for k, j in enumerate(mine):
                yield lambda: s_full[x].passed(ns & 1)
                ns += 1
                if vouched and (x == 0 or not two):
                    at = base + 2 * j
                    yield lambda: full[(at + 1) % NS].passed(((at + 1) // NS) & 1)
                    if k + 1 < len(mine) and (two or mistake):
                        nxt = at + 2 * step
                        yield lambda: full[nxt % NS].passed((nxt // NS) & 1)
                p_of[x] = (n, j, x)
                p_full[x].arrive()
            if mine:
                yield lambda: o_done[x].passed(no & 1)
                no += 1
            base += 2 * tiles

    rng = random.Random(seed)
    roles = [loader(), mma(), softmax(0), softmax(1)] + ([copies()] if raw else [])
    waits = [next(r, None) for r in roles]
    while any(w is not None for w in waits):
        ready = [k for k, w in enumerate(waits) if w is not None and w()]
        if not ready:
            raise Stuck([k for k, w in enumerate(waits) if w is not None])
        k = rng.choice(ready)
        waits[k] = next(roles[k], None)
    for got, want in log:
        assert got == want
    assert len(log) == 3 * sum(tiles * (2 if two else 1) for tiles, two in items)


def shares():
    rng = random.Random(3)
    yield [(1, True)], [(1, False)], [(2, False)], [(3, False)], [(7, True)], [(8, False)]
    for _ in range(30):
        yield tuple([(rng.randrange(1, 9), rng.random() < 0.5) for _ in range(rng.randrange(1, 5))] for _ in range(4))


# bf16: five or six slots, the softmax looks for the MMA thread; e4m3: raw buffers, three to six slots
@pytest.mark.parametrize("NS, raw, vouched", [(5, False, True), (6, False, True), (3, True, False), (4, True, False),
                                              (5, True, True), (6, True, True)])
def test_every_share_ends_and_reads_what_it_should(NS, raw, vouched):
    for group in shares():
        for items in group:
            for seed in range(4):
                run(items, NS, raw, vouched, seed)


def test_the_planted_mistake_is_found():
    with pytest.raises(Stuck):
        run([(5, False)], 3, True, True, 0, mistake=True)
