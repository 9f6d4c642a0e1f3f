"""The oracle of routing by scores: closed forms, the plain router as a special case,
brute force over all choices."""
import itertools
import math

import numpy as np
import pytest

import oracle as O
from oracle import scored


def test_softmax_renormalised_is_the_plain_router():
    logits = np.random.default_rng(0).standard_normal((50, 24)).astype(np.float32)
    a, b = scored.route_scored(logits, 5, 16), O.route(logits, 5, 16)
    for f in ("ids", "counts", "offsets", "perm", "inv", "tiles"):
        assert np.array_equal(getattr(a, f), getattr(b, f)), f
    # both in float64; b's are rounded to fp32 once (2^-24)
    assert np.all(np.abs(a.w - b.w) <= b.w * 2.0 ** -23)


def test_sigmoid_by_hand():
    ids, w = scored.choose([0.0, math.log(3.0), -math.log(3.0)], 2, sigmoid=True, renorm=False,
                           factor=2.0)
    assert ids == [1, 0] and w == pytest.approx([1.5, 1.0])
    # the bias chooses and does not weigh
    ids, w = scored.choose([0.0, math.log(3.0), -math.log(3.0)], 1, sigmoid=True, renorm=False,
                           bias=[0.0, 0.0, 1.0])
    assert ids == [2] and w == pytest.approx([0.25])


@pytest.mark.parametrize("best", [1, 2])
def test_groups_by_brute_force(best):
    rng = np.random.default_rng(best)
    for _ in range(30):
        z = rng.integers(-3, 4, 12).astype(np.float32) * 0.5
        ids, _ = scored.choose(z, 3, sigmoid=True, groups=4, top_groups=2, group_best=best)
        s = 1.0 / (1.0 + np.exp(-z.astype(np.float64)))
        rank = [sum(sorted(s[3 * g:3 * g + 3])[::-1][:best]) for g in range(4)]
        # the pair of groups and then the triple of experts that no other beats, the lowest
        # numbers among equals
        pair = max(itertools.combinations(range(4), 2),
                   key=lambda c: (sorted((rank[g] for g in c), reverse=True), [-g for g in c]))
        pool = [e for e in range(12) if e // 3 in pair]
        order = sorted(pool, key=lambda e: (-s[e], e))[:3]
        assert set(i // 3 for i in ids) <= set(pair) and ids == order


def test_values_out_of_range():
    inf = math.inf
    ids, w = scored.choose([math.nan, -inf, inf, 0.0], 4)
    assert ids == [2, 3, 0, 1] and w == [1.0, 0.0, 0.0, 0.0]
    ids, w = scored.choose([-800.0] * 4, 2, sigmoid=True)
    assert ids == [0, 1] and w == [0.0, 0.0]
    ids, _ = scored.choose([3.0, 2.0, 1.0], 2, bias=[-inf, 0.0, math.nan])
    assert ids == [1, 0]
