"""The forward kernel's synchronisation on the key-tile ranges of a mask plan.

A plan gives the two query tiles of a work item any two ranges: tile B may
start or end before tile A, and there may be a gap between them.  The kernel
walks the union of the two and stretches the earlier range over a gap
(fwd_item in fa_fwd_kernel.cuh).  The protocol model of test_fwd_protocol.py
is run on such items, with the union that the kernel takes there."""
import inspect
import random

import pytest

from tests import test_fwd_protocol as model

_CAUSAL_UNION = "((it[0][0] if it[0][1] > it[0][0] else it[1][0]), max(it[0][1], it[1][1]))"
_UNION = "(min([r[0] for r in it if r[1] > r[0]] or [0]), max(it[0][1], it[1][1]))"


@pytest.fixture(scope="module")
def run():
    source = inspect.getsource(model.run)
    assert _CAUSAL_UNION in source
    scope = dict(vars(model))
    exec(source.replace(_CAUSAL_UNION, _UNION), scope)
    return scope["run"]


def stretched(a, b):
    """fwd_item's rule: no key tile of the union is left out by both."""
    a, b = list(a), list(b)
    if a[1] > a[0] and b[1] > b[0]:
        if a[1] < b[0]:
            a[1] = b[0]
        if b[1] < a[0]:
            b[1] = a[0]
    return tuple(a), tuple(b)


def random_range(rnd):
    if rnd.random() < 0.15:
        return (0, 0)
    lo = rnd.randrange(0, 6)
    return (lo, lo + rnd.randrange(1, 4))


@pytest.mark.parametrize("NS", [2, 4])
def test_any_two_ranges(run, NS):
    rnd = random.Random(10 + NS)
    for trial in range(150):
        items = [stretched(random_range(rnd), random_range(rnd)) for _ in range(rnd.randrange(1, 6))]
        for seed in range(4):
            run(items, NS, seed=trial * 100 + seed, copy_prob=0.1 if seed % 3 == 0 else 1.0)


@pytest.mark.parametrize("items", [[((0, 2), (4, 5))], [((5, 6), (0, 2))]])
def test_an_unstretched_gap_stops_the_kernel(run, items):
    # the model knows the fault that the stretching is there for
    with pytest.raises(model.Err, match="deadlock"):
        run(items + [((0, 3), (0, 3))] * 2, 2, seed=1)
