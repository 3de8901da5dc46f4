"""The gate far out: silu(g) u where exp(g) is near the end of fp32 and past it, but the product is not."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X

pytestmark = pytest.mark.gpu

G = [-200.0, -187.0, -181.0, -176.0, -174.0, -150.0, -120.0, -100.0, -89.0, -88.5, -88.0, -87.5, -87.0, -86.5, -60.0, -17.0,
     -1.0, -2.0 ** -100, 0.0, 2.0 ** -100, 1.0, 17.0, 88.0, 100.0, 2.0 ** 100]
U = [s * 2.0 ** e for e in (-100, -20, 0, 20, 60, 100, 115, 127) for s in (1.0, -1.5)]


@pytest.mark.parametrize("rows", [1, 40, 200])
@pytest.mark.parametrize("row_type", ["bf16", "int8"])
def test_gate_over_the_range(rows, row_type):
    """Rows that pick the weights' first element: g and u are the products themselves, without a rounding (int8: the
    channel's scale)."""
    print(f"[gate] {rows} {row_type}", flush=True)
    pairs = np.array([(g, u) for g in G for u in U])
    n, K = len(pairs), 16
    values = torch.from_numpy(np.concatenate((pairs[:, 0], pairs[:, 1])))[None]  # [1, 2 n]
    assert torch.equal(values.bfloat16().double(), values)
    shape, off = mg.make_experts_shape(rows, 1, K, n), torch.tensor([0, rows], dtype=torch.int32, device=X.DEV)
    if row_type == "bf16":
        x, w = torch.zeros(rows, K, dtype=torch.bfloat16), torch.zeros(1, 2 * n, K, dtype=torch.bfloat16)
        x[:, 0], w[:, :, 0] = 1, values.bfloat16()
        scales = None
    else:
        x, w = torch.zeros(rows, K, dtype=torch.int8), torch.zeros(1, 2 * n, K, dtype=torch.int8)
        x[:, 0], w[:, :, 0] = 1, 1
        scales = values.float().to(X.DEV)
    got = mg.experts_matmul(shape, x.to(X.DEV), w.to(X.DEV), off, w_scales=scales, act=mg.ACT_SWIGLU).cpu().double().numpy()
    g, u = pairs[:, 0], pairs[:, 1]
    # g / (1 + exp(-g)) u, with 1 + exp(-g) = exp(-g) (1 + exp(g)) below zero
    ref = np.where(g < 0, g * np.exp(-np.abs(g)), g) * u / (1 + np.exp(-np.abs(g)))
    # silu to (|g| + 8) steps of fp32 and a step for each of the two products behind it; below -174 each half of the
    # exponential is subnormal, with 2^-149 / 2 of error and, for a result that bf16 holds, at least 2^-134 large
    err = np.abs(ref) * ((np.abs(g) + 10) * X.STEP32 + np.where(g < -174, 2.0 ** -15, 0.0))
    with np.errstate(invalid="ignore"):
        tol = err + X.BF16_HALF * (np.abs(ref) + err) + X.TINY
        over = np.abs(ref) > float(torch.finfo(torch.bfloat16).max) * (1 + X.BF16_HALF)
        bad = np.where(over, got != np.sign(ref) * np.inf, ~(np.abs(got - ref) <= tol))
    assert not bad.any(), [(*pairs[i], got[r, i], ref[i]) for r, i in np.argwhere(bad)[:5]]
