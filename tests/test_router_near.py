"""The tolerances of the renormalized weights' gradient tell a division from a product with a rounded reciprocal, and the mean
of the gradients from the mean about one of them (numpy in fp32, no GPU)."""
import numpy as np
import pytest

from tests import _router as R
from tests import _router_near as N

f32 = np.float32


def weights_grad(l, ids, score, scale, gw, by_reciprocal=False, about_largest=True):
    """The gradient in fp32, step by step: scores, their sum, the weights, the mean, back to the logits."""
    use, at = N.scored(l, ids)
    lj = np.where(use, np.take_along_axis(l, at, 1), -np.inf)
    top = lj.argmax(1)[:, None]
    with np.errstate(over="ignore", invalid="ignore"):
        s = np.exp(lj - np.take_along_axis(lj, top, 1)) if score == R.SOFTMAX else 1 / (1 + np.exp(-lj))
        slope = 1.0 if score == R.SOFTMAX else 1 / (1 + np.exp(lj))
    s, slope = np.where(use, s, 0.0).astype(f32), f32(1) * np.asarray(slope, f32)
    one = s.sum(1, keepdims=True, dtype=f32)
    w = s * (f32(1) / one) if by_reciprocal else s / one
    g = np.where(use, gw, 0).astype(f32)
    D = np.where(use, g - np.take_along_axis(g, top, 1), f32(0)) if about_largest else g
    a = f32(scale) * w * (D - (w * D).sum(1, keepdims=True, dtype=f32)) * slope
    d = np.zeros(l.shape, f32)
    np.add.at(d, (np.repeat(np.arange(len(l)), ids.shape[1]), at.ravel()), np.where(use, a, 0).ravel())
    return d


def inside(l, ids, score, gw, **kw):
    l64 = l.astype(np.float64)
    d, mag = N.grad(l64, ids, score, 1.5, gw.astype(np.float64))
    got = weights_grad(l, ids, score, 1.5, gw, **kw).astype(np.float64)
    return bool((np.abs(got - d) <= R.grad_tol(mag, d, l64, False)).all())


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("how", ["one", "dropped", "without a logit"])
def test_one_scored_slot(how, score):
    r = np.random.default_rng(1)
    l, ids = N.lone_slots(r, r.standard_normal((2000, 33)).astype(f32), 5, how)
    gw = r.standard_normal(ids.shape).astype(f32)
    assert inside(l, ids, score, gw)
    assert inside(l, ids, score, gw, by_reciprocal=True)  # the difference is 0, whatever the weight
    if score == R.SIGMOID:  # softmax's only score is 1, whose reciprocal is exact
        assert not inside(l, ids, score, gw, by_reciprocal=True, about_largest=False)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
def test_a_slot_that_carries_the_sum(score):
    r = np.random.default_rng(2)
    T, E, K = 2000, 33, 4
    l = r.standard_normal((T, E)).astype(f32) - f32(14)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :K].astype(np.int32)
    l[np.arange(T), ids[:, 0]] += f32(14)
    gw = (r.standard_normal((T, K)) + 1000).astype(f32)
    assert inside(l, ids, score, gw)
    assert not inside(l, ids, score, gw, about_largest=False)
    assert not inside(l, ids, score, gw, by_reciprocal=True, about_largest=False)
