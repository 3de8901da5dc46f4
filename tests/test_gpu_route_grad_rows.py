"""The logits' gradient from receive rows of any number: a slot whose row is not there has none."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,K", [(50, 16, 4), (33, 134, 8), (9, 2048, 16), (1, 8, 1)])
@pytest.mark.parametrize("part", [0.0, 0.3, 1.0, 1.5])
def test_rows_that_are_not_there(T, E, K, part):
    r = np.random.default_rng([T, E])
    logits = torch.from_numpy(r.standard_normal((T, E)).astype(np.float32)).to(X.DEV)
    shape, bal = mg.make_route_shape(T, E, K, scale=2.0), mg.make_balance(1, 0.5, 0.1)
    ids = mg.route(shape, logits).topk_idx
    loss = mg.balance_loss(shape, bal, logits, ids)
    dst = r.permutation(T * K).reshape(T, K).astype(np.int32)
    dst[r.random((T, K)) < 0.1] = -1
    dst[r.random((T, K)) < 0.1] = 2 ** 31 - 1
    n = int(part * T * K)
    buf = torch.full((2 * T * K,), np.nan, device=X.DEV)  # behind the rows: not looked at
    buf[:n] = torch.from_numpy(r.standard_normal(n).astype(np.float32))
    there = torch.from_numpy((dst >= 0) & (dst < n)).to(X.DEV)
    dst = torch.from_numpy(dst).to(X.DEV)
    slots = torch.where(there, buf[dst.clamp(0, 2 * T * K - 1).long()], 0.0)
    for more in ((), (bal, loss)):
        want = mg.route_grad(shape, logits, ids, slots, *more)
        got = mg.route_grad(shape, logits, ids, buf[:n], *more, dst_row=dst)
        assert torch.equal(got, want) and bool(got.isfinite().all())
