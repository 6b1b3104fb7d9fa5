"""The bound that oracle.cache8.decode derives for decode8 is narrow enough to see what a
kernel that loses or repeats pieces of a long sequence does to its output."""

import numpy as np
import pytest

from oracle import cache8 as oc


def case(n, d, seed, pages_differ):
    """One sequence of n keys, one head; pages_differ: V of a page is near one of +-8."""
    rng = np.random.default_rng(seed)
    page = 64
    p = oc.pool(-(-n // page), 1, page, d, page, "e4m3", rng, 0.0)
    if pages_differ:
        sign = rng.choice([-8.0, 8.0], (len(p["v"]), 1, 1, d))
        p["v"] = oc.encode(sign + rng.standard_normal(p["v"].shape) / 4, "e4m3")
        p["v_scale"][:] = 1.0
    q = np.round(rng.standard_normal((1, 1, d)) * 64) / 64
    return p, list(range(len(p["v"]))), q


def outputs(p, pages, n, q):
    return oc.decode(p, [pages], [n], q, q.shape[-1] ** -0.5)


@pytest.mark.parametrize("n,d", [(9000, 128), (20000, 64), (40000, 64)])
def test_lost_and_halved_outputs_are_seen(n, d):
    p, pages, q = case(n, d, n, False)
    want, bound = outputs(p, pages, n, q)
    seen = lambda o: np.max(np.abs(o - want) / bound) > 2.0
    assert not seen(want * (1 + 2.0 ** -9))
    assert seen(want * 0.0) and seen(want / 2)
    # every third page lost; a sixteenth of the keys, as of one piece in sixteen
    left = [e for e in pages if e % 3]
    assert seen(outputs(p, left, 64 * (len(left) - 1), q)[0])
    part = pages[len(pages) // 16:]
    assert seen(outputs(p, part, n - 64 * (len(pages) // 16), q)[0])


@pytest.mark.parametrize("n,d", [(9000, 128), (20000, 64), (40000, 64)])
def test_a_page_lost_or_repeated_is_seen(n, d):
    p, pages, q = case(n, d, n + 1, True)
    want, bound = outputs(p, pages, n, q)
    seen = lambda o: np.max(np.abs(o - want) / bound) > 1.0
    for at in (0, len(pages) // 2, len(pages) - 2):
        assert seen(outputs(p, pages[:at] + pages[at + 1:], n - 64, q)[0])
        assert seen(outputs(p, pages[:at] + [pages[at]] + pages[at:], n + 64, q)[0])
