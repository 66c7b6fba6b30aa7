"""The routing's definition in 64 bits, one token at a time, and the tolerance
of its fp32 weights."""
import math

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)
HALF_STEP = 2.0 ** -24  # largest relative error of one fp32 rounding


def _score_log(z, live, scoring):
    if scoring == "softmax":
        m = max(z[e] for e in live)
        s = sum(math.exp(z[e] - m) for e in live)
        return {e: z[e] - m - math.log(s) for e in live}
    return {e: -np.logaddexp(0.0, -z[e]) for e in live}


def route_row(logits, k, scoring="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True,
              scale=1.0):
    """(ids, weights) of one token; logits and bias as float64 values."""
    E = len(logits)
    z = [min(float(v), FLT_MAX) if v > -math.inf else -math.inf for v in logits]
    live = [e for e in range(E) if z[e] > -math.inf]
    ids, w = [-1] * k, [0.0] * k
    if not live:
        return ids, w
    logs = _score_log(z, live, scoring)
    score = {e: math.exp(logs[e]) for e in live}
    if bias is None:
        choice = {e: z[e] for e in live}
    else:
        choice = {e: score[e] + float(bias[e]) for e in live if score[e] + float(bias[e]) > -math.inf}
    S = E // n_group
    if n_group > 1:
        value = []
        for g in range(n_group):
            have = [score[e] if bias is None and group_top == 2 else choice[e]
                    for e in range(g * S, (g + 1) * S) if e in choice]
            have.sort(reverse=True)
            value.append((-sum(have[:group_top]) if have else math.inf, g))
        keep = {g for _, g in sorted(value)[:topk_group]}
        choice = {e: c for e, c in choice.items() if e // S in keep}
    order = sorted(choice, key=lambda e: (-choice[e], e))[:k]
    if not order:
        return ids, w
    if renormalize:
        m = max(logs[e] for e in order)
        part = [math.exp(logs[e] - m) for e in order]
        part = [v / sum(part) for v in part]
    else:
        part = [score[e] for e in order]
    for i, e in enumerate(order):
        ids[i], w[i] = e, part[i] * scale
    return ids, w


def route_rows(logits, k, **kw):
    rows = [route_row(r, k, **kw) for r in np.asarray(logits, np.float64)]
    return np.array([r[0] for r in rows], np.int32).reshape(-1, k), np.array([r[1] for r in rows]).reshape(-1, k)


def weight_tolerance(logits, ids, want, scale):
    """Largest error of an fp32 weight, per element.  Its exponential's argument is
    a rounded difference (relative error |d| half steps, where the weight
    does not vanish: |d| <= 110), the exponential itself is off by at most 2
    half steps and 2 more for a sigmoid's sum and quotient.  The sum over the experts
    takes 9 roundings (512 terms in a tree), its terms' errors weigh at most
    ln(512) + 3 half steps together; quotient and scale are one each: under 32
    in all besides |d|.  Below the normal range of fp32 the error is absolute."""
    z = np.asarray(logits, np.float64)
    z = np.where(z > -np.inf, np.minimum(z, FLT_MAX), -np.inf)
    top = z.max(axis=1, keepdims=True)
    at = np.where(ids >= 0, np.take_along_axis(z, np.maximum(ids, 0).astype(np.int64), 1), 0.0)
    d = np.where(ids >= 0, np.minimum(np.where(top > -np.inf, top, 0.0) - at, 110.0), 0.0)
    return np.abs(want) * (2.0 * d + 32.0) * HALF_STEP + scale * 2.0 ** -120
