"""The gate and its gradient where the logistic function leaves fp32 but its products with large factors do not."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X
from tests.test_gpu_swiglu import logistic

pytestmark = pytest.mark.gpu

STEP32, HALF = X.STEP32, X.BF16_HALF
TOP = float(torch.finfo(torch.bfloat16).max) * (1 + HALF)


def agrees(name, got, ref, steps):
    """Below -80 a result is good to (2 |g| + 16) steps of fp32 (its exponent's rounding, |g| / 8 of 8 factors, and the rest) and
    rounded to fp32 and then bf16, or subnormal to half of 2^-133 and of 2^-149."""
    err = np.abs(ref) * steps * STEP32
    tol = err + (HALF + STEP32) * (np.abs(ref) + err) + 2.0 ** -134 + 2.0 ** -150
    big = np.abs(ref) > TOP
    bad = np.where(big, got != np.sign(ref) * np.inf, ~(np.abs(got - ref) <= tol))
    near = np.abs(np.abs(ref) / TOP - 1) < 0.01  # rounded to infinity or to the largest
    assert not (bad & ~near).any(), (name, [(i, got[i], ref[i]) for i in np.argwhere(bad & ~near)[:4].tolist() for i in [tuple(i)]])


@pytest.mark.parametrize("w", [2.0 ** -20, 1.0, 2.0 ** 60, 2.0 ** 120])
@pytest.mark.parametrize("seed", [0, 1])
def test_large_factors(w, seed):
    """g down to -366, u, d and the routing weight up to the largest: every product that bf16 holds, whatever lies between."""
    r = np.random.default_rng([seed, int(np.log2(w)) + 50])
    rows, n = 96, 264
    sign = lambda *s: np.where(r.random(s) < 0.5, -1.0, 1.0)  # noqa: E731
    g = torch.from_numpy(-r.uniform(80.5, 366, (rows, n)).astype(np.float32)).bfloat16()
    u = torch.from_numpy((sign(rows, n) * 2.0 ** r.uniform(-60, 126, (rows, n))).astype(np.float32)).bfloat16()
    d = torch.from_numpy((sign(rows, n) * 2.0 ** r.uniform(-60, 126, (rows, n))).astype(np.float32)).bfloat16()
    h0 = torch.cat((g, u), 1)
    ws = torch.full((rows,), w)
    f = mg.swiglu(h0.to(X.DEV), ws.to(X.DEV))
    b = mg.swiglu_grad(d.to(X.DEV), h0.to(X.DEV), row_weights=ws.to(X.DEV))
    assert torch.equal(f.out, b.out)
    g, u, d = X.f64(g), X.f64(u), X.f64(d)
    s, rest = logistic(g)
    steps = 2 * np.abs(g) + 16
    with np.errstate(over="ignore"):
        agrees("out", X.f64(f.out.cpu()), w * g * s * u, steps)
        got = X.f64(b.grad_h0.cpu())
        agrees("dg", got[:, :n], w * d * u * s * (1 + g * rest), steps)
        agrees("du", got[:, n:], w * d * g * s, steps)
    # the weight's gradient: the terms' roundings and n / 8 + 16 additions
    term = d * g * s * u
    tol = (np.abs(term) * (steps + n / 8 + 16)).sum(1) * STEP32 + n * 2.0 ** -149
    got = b.grad_row_weights.cpu().double().numpy()
    fits = np.abs(term).sum(1) < 2.0 ** 127
    assert (np.abs(got - term.sum(1)) <= tol)[fits].all()
    assert w != 2.0 ** 60 or ((np.abs(w * d * u * s * g) > 2.0 ** -120) & (np.abs(w * d * u * s * g) < 2.0 ** 120) & (g < -208)).any()


def test_lowest_values():
    """-inf gives NaN, as the formula does; the lowest finite value a zero."""
    low = float(torch.finfo(torch.bfloat16).min)
    h0 = torch.ones(2, 16, dtype=torch.bfloat16)
    h0[0, 0], h0[1, 0] = low, -float("inf")
    d = torch.ones(2, 8, dtype=torch.bfloat16)
    f = mg.swiglu(h0.to(X.DEV)).out.cpu()
    b = mg.swiglu_grad(d.to(X.DEV), h0.to(X.DEV))
    assert f[0, 0] == 0 and f[1, 0].isnan() and bool(f[:, 1:].isfinite().all())
    g = b.grad_h0.cpu()
    assert g[0, 0] == 0 and g[0, 8] == 0 and g[1, 0].isnan() and g[1, 8].isnan()
    assert torch.equal(torch.nan_to_num(b.out.cpu(), nan=7.0), torch.nan_to_num(f, nan=7.0))


def test_infinite_factors():
    """An infinite gradient or u beside a small logistic function: infinities, as the products are, and no NaN."""
    inf = float("inf")
    g = [-79.0, -81.0, -100.0, -150.0]
    h0 = torch.ones(8, 16, dtype=torch.bfloat16)
    d = torch.ones(8, 8, dtype=torch.bfloat16)
    for k, v in enumerate(g):
        h0[k, 3], h0[4 + k, 3] = v, v
        d[k, 3] = inf
        h0[4 + k, 11] = inf
    w = torch.ones(8, device=X.DEV)
    b = mg.swiglu_grad(d.to(X.DEV), h0.to(X.DEV), row_weights=w)
    gw, gr, out = b.grad_row_weights.cpu(), b.grad_h0.cpu(), b.out.cpu()
    assert (gw == -inf).all()
    assert (gr[:4, 3] == -inf).all() and (gr[:4, 11] == -inf).all() and (gr[4:, 3] == -inf).all()
    assert (out[4:, 3] == -inf).all() and bool(out[:4].isfinite().all())
    assert torch.equal(mg.swiglu(h0.to(X.DEV), w).out.cpu(), out)
