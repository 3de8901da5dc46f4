"""A row of the gate depends on its own inputs alone, bit for bit, and the gradient's `out` is the forward's result again."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X

pytestmark = pytest.mark.gpu


def world(rows, n):
    r = np.random.default_rng([rows, n])
    h0, d = X.bf16(r, rows, 2 * n).to(X.DEV), X.bf16(r, rows, n).to(X.DEV)
    w = torch.from_numpy(r.uniform(0.5, 1, rows).astype(np.float32)).to(X.DEV)
    h0[:, :n] *= 4  # some of every size between -20 and 20
    return h0, d, w


def results(h0, d, w, kept):
    f = mg.swiglu(h0, w, checkpoint=kept)
    g = mg.swiglu_grad(d, row_weights=w, **(dict(codes=f.codes, scales=f.scales) if kept else dict(h0=h0)))
    return [t for t in (f.out, f.codes, f.scales, g.grad_h0, g.out, g.grad_row_weights) if t is not None]


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("far", [-81.0, -100.0, -200.0, -3e38])
@pytest.mark.parametrize("rows,n", [(64, 8), (64, 128), (61, 256), (33, 520), (16, 1024), (9, 2056)])
def test_beside_a_row_that_is_far_out(rows, n, far, kept):
    h0, d, w = world(rows, n)
    want = results(h0, d, w, kept)
    other = h0.clone()
    other[1::2, 0] = far
    for a, b in zip(want, results(other, d, w, kept)):
        assert torch.equal(a[::2], b[::2])


@pytest.mark.parametrize("far", [-81.0, -100.0, -200.0])
@pytest.mark.parametrize("rows,n", [(64, 8), (61, 256), (33, 520), (9, 2056)])
def test_beside_a_column_that_is_far_out(rows, n, far):
    h0, d, w = world(rows, n)
    out, grad, again, _ = results(h0, d, w, False)
    other = h0.clone()
    other[:, 3] = far
    o, g, a, _ = results(other, d, w, False)
    keep = torch.arange(n, device=X.DEV) != 3
    assert torch.equal(o[:, keep], out[:, keep]) and torch.equal(a[:, keep], again[:, keep])
    assert torch.equal(g.view(rows, 2, n)[:, :, keep], grad.view(rows, 2, n)[:, :, keep])


@pytest.mark.parametrize("rows,n", [(64, 8), (61, 128), (1000, 256), (33, 520), (300, 2048), (9, 8200)])
@pytest.mark.parametrize("far", [None, -81.0, -150.0])
def test_the_forwards_result_again(rows, n, far):
    h0, d, w = world(rows, n)
    if far is not None:
        h0[::3, ::5] = far
    out, _, again, _ = results(h0, d, w, False)
    assert torch.equal(out, again)
