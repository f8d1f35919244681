"""Model check of the hand-off between the parts of a split item of the
score-modified backward (fa_bwd_kernel.cuh, fa_bwd_main's dV / dK epilogue), run
on the CPU over random interleavings.

As for the two halves of test_bwd_split_handoff.py, with S parts: each part's
threads write their fp32 rows, fence, meet on a barrier, and one takes a ticket;
the part that draws ticket S - 1 fences and adds the other S - 1 parts' rows to
its own.  A part that finds the other S - 1 counted in before it writes is the last
one: it writes no rows and takes no ticket.  No part waits for another.  Stores drain to memory at random moments;
the partial area starts with the previous call's rows."""
import random

import pytest

ROWS = 3


class Err(Exception):
    pass


def run(seed, S, mutation=None):
    rnd = random.Random(seed)
    mem = {("part", h, r): (-1, 0.0) for h in range(S) for r in range(ROWS)}
    mem["cnt"] = 0
    for call in range(2):
        if mutation != "counter-not-zeroed":
            mem["cnt"] = 0  # the preprocess kernel of this call
        out = {}
        own = {(h, r): float(100 * call + 10 * h + r + 1) for h in range(S) for r in range(ROWS)}
        buf = {k: [] for k in own}
        arrived = {(h, b): 0 for h in range(S) for b in (0, 1, 2)}
        peeked = {}
        ticket = {}

        def drain(key):
            while buf[key]:
                addr, val = buf[key].pop(rnd.randrange(len(buf[key])))
                mem[addr] = val

        def thread(h, r):
            if r == 0:
                peeked[h] = mem["cnt"] >= (S - 2 if mutation == "peeks-one-early" else S - 1)
            arrived[(h, 0)] += 1
            while arrived[(h, 0)] < ROWS:
                yield
            if peeked[h]:
                ticket[h] = S - 1
                yield from finish(h, r)
                return
            buf[(h, r)].append((("part", h, r), (call, own[(h, r)])))
            yield
            if mutation != "no-writer-fence":
                drain((h, r))
            arrived[(h, 1)] += 1
            while arrived[(h, 1)] < ROWS:
                yield
            if r == 0:
                ticket[h] = mem["cnt"]
                mem["cnt"] += 1
            arrived[(h, 2)] += 1
            while arrived[(h, 2)] < ROWS:
                yield
            if ticket[h] == (1 if mutation == "second-finishes" else S - 1):
                yield from finish(h, r)

        def finish(h, r):
            yield
            total = own[(h, r)]
            for other in range(S):
                if other == h:
                    if mutation == "own-part-twice":
                        total += own[(h, r)]
                    continue
                got = mem[("part", other, r)]
                if got[0] != call:
                    raise Err(f"part {h} read a stale row of part {other}")
                total += got[1]
            if r in out:
                raise Err("two parts finished")
            out[r] = total

        live = [thread(h, r) for h in range(S) for r in range(ROWS)]
        while live:
            if rnd.random() < 0.2:
                drain(rnd.choice(list(buf)))
            i = rnd.randrange(len(live))
            try:
                next(live[i])
            except StopIteration:
                live.pop(i)
        for key in buf:
            drain(key)
        if out != {r: sum(own[(h, r)] for h in range(S)) for r in range(ROWS)}:
            raise Err(f"stored {out}")


@pytest.mark.parametrize("S", [2, 3, 8])
def test_the_last_part_stores_the_sum(S):
    for seed in range(400):
        run(seed, S)


@pytest.mark.parametrize("mutation", ["no-writer-fence", "second-finishes", "counter-not-zeroed", "own-part-twice", "peeks-one-early"])
def test_planted_mistakes_are_caught(mutation):
    caught = 0
    for seed in range(400):
        try:
            run(seed, 4, mutation)
        except Err:
            caught += 1
    assert caught > 0


def test_parts_cover_every_tile_once():
    """t0 = T part / S, T = T (part + 1) / S - t0 in whole tiles."""
    for T in range(0, 70):
        for S in range(2, 9):
            ranges = [(T * h // S, T * (h + 1) // S) for h in range(S)]
            assert ranges[0][0] == 0 and ranges[-1][1] == T
            assert all(a[1] == b[0] for a, b in zip(ranges, ranges[1:]))
