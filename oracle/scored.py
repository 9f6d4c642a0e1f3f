"""Routing by scores, bias and groups in float64, one token at a time (plain loops).

Non-finite logits and biases follow the library's rule: NaN and -inf count as the
least finite fp32 number, +inf as the largest. The arrays behind the choice
(histogram, offsets, permutation, block map) are those of :func:`oracle.route`.
"""
import math

import numpy as np

from . import Route

FMAX = float(np.finfo(np.float32).max)


def finite(v: float) -> float:
    return -FMAX if math.isnan(v) else max(-FMAX, min(FMAX, v))


def choose(logits, k, sigmoid=False, bias=None, groups=1, top_groups=1, group_best=1,
           renorm=True, factor=1.0):
    """(ids, fp64 weights) of one token."""
    z = [finite(float(v)) for v in logits]
    E = len(z)
    if sigmoid:
        # exp(-z) overflows where the score is 0 in float64
        score = [1.0 / (1.0 + math.exp(-v)) if v > -700.0 else math.exp(v) if v > -745.0 else 0.0
                 for v in z]
    else:
        top = max(z)
        score = [math.exp(v - top) for v in z]
        total = math.fsum(score)
        score = [s / total for s in score]
    # scores grow with the logits: where scores alone are compared, the logits tell their order
    # exactly, also where float64 rounds two scores to the same number
    if bias is None and (groups == 1 or group_best == 1):
        key = z
    else:
        key = [s + (0.0 if bias is None else finite(float(bias[e])))
               for e, s in enumerate(score)]
    per = E // groups
    if groups > 1:
        rank = [sum(sorted(key[g * per:g * per + per], reverse=True)[:group_best])
                for g in range(groups)]
        stay = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
        pool = [e for e in range(E) if e // per in stay]
    else:
        pool = range(E)
    ids = sorted(pool, key=lambda e: (-key[e], e))[:k]
    w = [score[e] for e in ids]
    total = math.fsum(w) if renorm else 1.0
    return ids, [factor * v / total if total > 0 else 0.0 for v in w]


def arrays(ids, E: int, block_m: int):
    """Histogram, offsets, permutation, inverse and block map of chosen experts [T][k]."""
    ids = np.asarray(ids, dtype=np.int32)
    T, k = ids.shape
    flat = ids.reshape(-1)
    counts = np.bincount(flat, minlength=E).astype(np.int32)
    offsets = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    perm = np.argsort(flat, kind="stable").astype(np.int32)
    inv = np.empty(T * k, dtype=np.int32)
    inv[perm] = np.arange(T * k, dtype=np.int32)
    tiles = [(e, int(offsets[e]) + s, min(block_m, int(counts[e]) - s))
             for e in range(E) for s in range(0, int(counts[e]), block_m)]
    return counts, offsets, perm, inv, np.array(tiles, dtype=np.int32).reshape(-1, 3)


def route_scored(logits, k, block_m=128, **how) -> Route:
    """:func:`choose` for every token; w stays float64."""
    logits = np.asarray(logits, dtype=np.float32)
    T, E = logits.shape
    rows = [choose(row, k, **how) for row in logits]
    ids = np.array([r[0] for r in rows], dtype=np.int32).reshape(T, k)
    w = np.array([r[1] for r in rows], dtype=np.float64).reshape(T, k)
    counts, offsets, perm, inv, tiles = arrays(ids, E, block_m)
    return Route(T, E, k, block_m, ids, w, counts, offsets, perm, inv, tiles)
