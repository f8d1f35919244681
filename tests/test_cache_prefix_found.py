"""A CPU model of how fa_cache_prefix_kernel hands on, item by item, where values were not finite:
the loader resets a buffer, notes what it finds and hands it over; both softmax
warpgroups read it at the item's end and give it back.  Two buffers in turn.  Whatever role
goes first, every item's readers see what was noted for it, and every share ends.  Planted
mistakes have to be found: a warpgroup without key tiles that does not wait, and a
loader that does not."""
import random

import pytest


class Stuck(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != parity


def run(items, seed, NS=5, threads=3, mistake=""):
    """items: (key tiles, tile B has key tiles) each; `threads` stand for a warpgroup's 128."""
    full, free = [Barrier(1) for _ in range(2)], [Barrier(2 * threads) for _ in range(2)]
    slots = [0, 0]  # units loaded and consumed
    buffer, open_tiles = [None, None], [0] * len(items)
    q = [[0, 0] for _ in items]  # threads of each warpgroup that have brought their query rows

    def loader():
        for n, (tiles, _) in enumerate(items):
            if mistake != "loader":
                yield lambda: free[n & 1].passed(((n >> 1) & 1) ^ 1)
            buffer[n & 1] = (n, 0)
            for j in range(tiles):
                yield lambda: slots[0] - slots[1] < NS
                slots[0] += 1
                buffer[n & 1] = (n, j + 1)
            full[n & 1].arrive()

    def mma():
        at = 0
        for n, (tiles, b) in enumerate(items):
            yield lambda: q[n][0] == threads and (not b or q[n][1] == threads)
            for _ in range(tiles):
                at += 1
                yield lambda: slots[0] >= at
                slots[1] += 1
            open_tiles[n] = 1

    def thread(x):
        for n, (tiles, b) in enumerate(items):
            mine = x == 0 or b
            if mine:
                q[n][x] += 1
                yield lambda: open_tiles[n]
            if mine or mistake != "readers":
                yield lambda: full[n & 1].passed((n >> 1) & 1)
            if mine:
                assert buffer[n & 1] == (n, tiles), (n, buffer)
                yield lambda: True
                assert buffer[n & 1] == (n, tiles), (n, buffer)
            free[n & 1].arrive()

    rng = random.Random(seed)
    roles = [loader(), mma()] + [thread(x) for x in (0, 1) for _ in range(threads)]
    favoured = rng.randrange(len(roles))
    waits = [next(r, None) for r in roles]
    while any(w is not None for w in waits):
        ready = [k for k, w in enumerate(waits) if w is not None and w()]
        if not ready:
            raise Stuck([k for k, w in enumerate(waits) if w is not None])
        k = favoured if favoured in ready and rng.random() < 0.8 else rng.choice(ready)
        waits[k] = next(roles[k], None)


def shares(seed):
    rng = random.Random(seed)
    return [(n := rng.choice((1, 1, 2, 3, 9)), n > 1 and rng.random() < 0.7) for _ in range(rng.randrange(1, 9))]


@pytest.mark.parametrize("NS", [5, 6])
def test_every_item_reads_its_own(NS):
    for seed in range(400):
        run(shares(seed), seed, NS)


@pytest.mark.parametrize("mistake", ["loader", "readers"])
def test_planted_mistakes_are_found(mistake):
    found = 0
    for seed in range(400):
        try:
            run(shares(seed), seed, mistake=mistake)
        except (AssertionError, Stuck):
            found += 1
    assert found > 0
