"""Every tile that the expert stage's products are built for, selected by its sizes, with several ragged tiles for a
workgroup, against 64-bit references."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X
from tests import _tiles

pytestmark = pytest.mark.gpu


def _case(case):
    op, ty, act, tile, E, mean, K, N = case
    print(f"[experts tiles] {_tiles.name(case)} E={E} mean={mean} N={N}", flush=True)
    rows = _tiles.rows_of(E, mean)
    assert mg.experts_tile(rows.shape(K, N), op, ty, act) == tile
    return rows, K, N, np.random.default_rng([15, op, ty, act, K, N])


@pytest.mark.parametrize("case", [c for c in _tiles.CASES if c[0] == _tiles.F], ids=_tiles.name)
def test_forward(case):
    rows, K, N, r = _case(case)
    ty, act = case[1:3]
    nw, t = N * (1 + act), torch.from_numpy
    xs = ws = None
    if ty == mg.ROWS_BF16:
        x, w = X.bf16(r, rows.rows, K), X.bf16(r, rows.E, nw, K, scale=K ** -0.5)
        x64, w64 = X.f64(x), X.f64(w)
    elif ty == mg.ROWS_INT8:
        x, w = (t(r.integers(-127, 128, s, dtype=np.int8)) for s in ((rows.rows, K), (rows.E, nw, K)))
        xs, ws = (t(r.uniform(0.5, 2, s).astype(np.float32) / 70) for s in ((rows.rows,), (rows.E, nw)))
        ws /= K ** 0.5
        x64, w64 = X.f64(x) * X.f64(xs)[:, None], X.f64(w) * X.f64(ws)[..., None]
    else:
        x, w = (t(r.integers(0, 256, s, dtype=np.uint8)) for s in ((rows.rows, K // 2), (rows.E, nw, K // 2)))
        xs = t(r.integers(122, 129, (rows.rows, K // 32), dtype=np.uint8))
        ws = t(r.integers(116, 123, (rows.E, nw, K // 32), dtype=np.uint8))
        x64, w64 = X.unpack_mx(x.numpy(), xs.numpy()), X.unpack_mx(w.numpy(), ws.numpy())
    ref, tol = X.product(rows, x64, w64, bool(act))
    d = lambda a: None if a is None else a.to(X.DEV)  # noqa: E731
    xd, wd, xsd, wsd = d(X.poison(x, rows.used)), d(w), d(xs), d(ws)
    outs = [mg.experts_matmul(rows.shape(K, N), xd, wd, rows.dev_off(), xsd, wsd, act, X.canary(rows.rows, N)) for _ in range(2)]
    X.check(outs[0], ref, tol, rows.used, _tiles.name(case))
    assert torch.equal(*outs), "the same call twice"


@pytest.mark.parametrize("case", [c for c in _tiles.CASES if c[0] == _tiles.D], ids=_tiles.name)
def test_dgrad(case):
    rows, K, N, r = _case(case)
    w, dy = X.bf16(r, rows.E, N, K, scale=K ** -0.5), X.bf16(r, rows.rows, N)
    ref, tol = X.product(rows, X.f64(dy), np.ascontiguousarray(X.f64(w).transpose(0, 2, 1)), False)
    args = rows.shape(K, N), X.poison(dy, rows.used).to(X.DEV), w.to(X.DEV), rows.dev_off()
    outs = [mg.experts_matmul_dgrad(*args, out=X.canary(rows.rows, K)) for _ in range(2)]
    X.check(outs[0], ref, tol, rows.used, _tiles.name(case))
    assert torch.equal(*outs), "the same call twice"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", [c for c in _tiles.CASES if c[0] == _tiles.W], ids=_tiles.name)
def test_wgrad(case, dtype):
    rows, K, N, r = _case(case)
    x, dy = X.bf16(r, rows.rows, K), X.bf16(r, rows.rows, N)
    ref, tol = np.zeros((rows.E, N, K)), np.zeros((rows.E, N, K))
    for e, lo, hi in rows.spans():  # zeros, exactly, where there are no rows
        a, b = X.f64(dy[lo:hi]), X.f64(x[lo:hi])
        ref[e] = a.T @ b
        if hi > lo:
            err = (hi - lo + 8) * X.STEP32 * (np.abs(a).T @ np.abs(b))
            tol[e] = err + X.TINY + (X.BF16_HALF * (np.abs(ref[e]) + err) if dtype == torch.bfloat16 else 0)
    args = rows.shape(K, N), X.poison(dy, rows.used).to(X.DEV), X.poison(x, rows.used).to(X.DEV), rows.dev_off()
    outs = [mg.experts_matmul_wgrad(*args, out=torch.full((rows.E, N, K), -7.0, dtype=dtype, device=X.DEV)) for _ in range(2)]
    X.check(outs[0], ref, tol, np.ones(rows.E, bool), _tiles.name(case))
    assert torch.equal(*outs), "the same call twice"
