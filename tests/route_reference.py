"""The choice of experts in whole numbers, as include/fp8bs.h defines it: c = s + bias in
multiples of 2^-44, compared as Python integers, so that no bias is too large.

The library holds c within 2^-43, two units: a row counts only where what is told
apart is further apart than that (`clear`)."""
import math
from fractions import Fraction

import numpy as np

UNIT = 1 << 44
SLACK = 4                                       # units between two c's, each off by two at most


def scores(x, scoring):
    x = np.asarray(x, dtype=np.float64)
    if scoring == "sigmoid":
        return 1.0 / (1.0 + np.exp(-x))
    e = np.exp(x - x.max())
    return e / e.sum()


def choose(x, topk, scoring, bias, groups=1, topk_groups=1, group_top=1):
    """One row of logits -> (ids, s, clear).  A NaN c comes after every other, a group with one among its best after every
    group without."""
    s = scores(x, scoring)
    e = len(s)
    c = []
    for si, b in zip(s, bias):
        if math.isnan(b):
            c.append(None)
        else:
            c.append(round((Fraction(float(si)) + Fraction(float(min(max(b, -65536.0), 65536.0)))) * UNIT))
    order = lambda i: (1, 0, i) if c[i] is None else (0, -c[i], i)
    clear = True
    live = list(range(e))
    if groups > 1:
        per = e // groups
        best = []
        for g in range(groups):
            top = sorted(range(g * per, (g + 1) * per), key=order)[:group_top]
            nans = sum(c[i] is None for i in top)
            best.append((nans, -sum(c[i] for i in top if c[i] is not None), g))
        ranked = sorted(best)
        if topk_groups < groups:
            a, b = ranked[topk_groups - 1], ranked[topk_groups]
            clear &= a[0] != b[0] or a[0] == group_top or b[1] - a[1] > 2 * SLACK
        opened = {r[2] for r in ranked[:topk_groups]}
        live = [i for i in live if i // per in opened]
    ranked = sorted(live, key=order)
    for i, j in zip(ranked[:topk], ranked[1:topk + 1]):
        same = c[i] == c[j] and (c[i] is None or (x[i] == x[j] and bias[i] == bias[j]))
        clear &= same or (c[i] is None) != (c[j] is None) or abs(c[i] - c[j]) > SLACK
    return ranked[:topk], s, clear
