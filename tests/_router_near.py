"""The renormalized weights' gradient with tolerances that follow the result: nothing where a token has one scored slot."""
import numpy as np

from tests import _router as R


def scored(l, ids):
    """(which slots have an id with a logit, their ids or 0, the logarithms of their scores less the token's largest's)"""
    E = l.shape[1]
    use = (ids >= 0) & (ids < E)
    at = np.where(use, ids, 0)
    return use & (np.take_along_axis(l, at, 1) > -np.inf), at


def grad(l, ids, score, scale, gw, mask=None, **losses):
    """(gradient of the logits, magnitudes that its rounding is relative to) of renormalized weights, d_j = gw[t, j].

    a_j = scale w_j (d_j - sum_i w_i d_i) = scale w_j (D_j - sum_i w_i D_i) with D_i = d_i - d_0, 0 a slot with the largest
    score.  A rounding of a difference, a weight or a sum of these is relative to |D_j| + sum_i w_i |D_i|, which is 0 where
    all slots with a score have the same d: then the result is 0, exactly for one such slot."""
    d, mag = R.grad(l, ids, score, True, scale, None, mask=mask, **losses)
    T, K = ids.shape
    on = R.live(l, mask)
    use, at = scored(l, ids)
    use &= on[:, None]
    q = np.where(use, np.take_along_axis(R.log_scores(l, score), at, 1), -np.inf)
    g = np.where(use, gw, 0.0)
    top = q.argmax(1)[:, None]
    m = np.where(use.any(1, keepdims=True), np.take_along_axis(q, top, 1), 0.0)
    with np.errstate(invalid="ignore"):
        e = np.where(use, np.exp(q - m), 0.0)
    w = e / np.where(e.sum(1, keepdims=True) > 0, e.sum(1, keepdims=True), 1.0)
    D = np.where(use, g - np.take_along_axis(g, top, 1), 0.0)
    a = scale * w * (D - (w * D).sum(1, keepdims=True))
    am = abs(scale) * w * (np.abs(D) + (w * np.abs(D)).sum(1, keepdims=True))
    slope = 1.0
    if score == R.SIGMOID:
        with np.errstate(over="ignore"):
            slope = np.take_along_axis(np.where(l > -np.inf, 1 / (1 + np.exp(np.minimum(l, 700.0))), 0.0), at, 1)
    rows = np.repeat(np.arange(T), K)
    np.add.at(d, (rows, at.ravel()), (a * slope).ravel())
    np.add.at(mag, (rows, at.ravel()), (am * slope).ravel())
    return d, mag


def lone_slots(r, l, K, how):
    """ids [T, K] and logits of tokens with one scored slot: "one" chosen id, the others "dropped", or "without a logit"."""
    T, E = l.shape
    if how == "one":
        return l, r.integers(0, E, (T, 1)).astype(np.int32)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :K].astype(np.int32)
    keep = r.integers(0, K, T)
    others = np.arange(K)[None] != keep[:, None]
    if how == "dropped":
        return l, np.where(others, -1, ids).astype(np.int32)
    l = np.array(l)
    t, j = np.nonzero(others)
    l[t, ids[t, j]] = -np.inf
    return l, ids
