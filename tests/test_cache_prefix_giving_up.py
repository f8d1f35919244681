"""A CPU model of how fa_cache_prefix_kernel's bf16 loader leaves when a wait runs out: no copy may
be in flight when the CTA gives its shared memory up.  Tiles of values in whose rows zeros are
written arrive on a barrier of their own, and their slot's barrier is then passed on by
hand, so that it says nothing of the copy.  The mistake of not waiting for that barrier at the
end has to be found."""
import random

import pytest


def run(tails, give_up_at, seed, NS=5, mended=True):
    """tails: for each unit, whether it goes by way of the extra barrier; the wait number `give_up_at`
    runs out.  Returns the copies in flight at the CTA's end."""
    rng = random.Random(seed)
    full, raw = [0] * NS, 0     # completed phases
    flying = []                 # (barrier, slot) of copies on their way
    waits = 0

    def land(n):
        nonlocal raw
        for _ in range(n):
            if flying:
                kind, s = flying.pop(rng.randrange(len(flying)))
                if kind == "raw":
                    raw += 1
                else:
                    full[s] += 1

    def wait(done):  # False: it ran out
        nonlocal waits
        waits += 1
        if waits == give_up_at:
            return False
        while not done():
            land(1)
        return True

    def wait_to_the_end(done):  # bounded in the kernel, ignoring that somebody gave up
        while not done() and flying:
            land(1)

    u = zeroed = 0
    for u, tail in enumerate(tails):
        s = u % NS
        land(rng.randrange(2))
        if not wait(lambda: True):  # the slot is free
            break
        if tail:
            flying.append(("raw", s))
            zeroed += 1
            target = zeroed
            ok = wait(lambda: raw >= target)
            full[s] += 1  # by hand, given up or not
            if not ok:
                u += 1
                break
        else:
            flying.append(("full", s))
    else:
        u = len(tails)
    if mended and zeroed:
        wait_to_the_end(lambda: raw >= zeroed)
    for v in range(max(u - NS, 0), u):
        wait_to_the_end(lambda: full[v % NS] >= v // NS + 1)
    return len(flying)


def calls():
    for seed in range(300):
        rng = random.Random(seed)
        tails = [k % 2 == 1 and rng.random() < 0.5 for k in range(rng.randrange(1, 20))]
        for give_up_at in range(1, 2 * len(tails) + 2):
            yield tails, give_up_at, seed


def test_no_copy_is_left_in_flight():
    for call in calls():
        assert run(*call) == 0, call


def test_the_mistake_is_found():
    assert any(run(*call, mended=False) for call in calls())
