"""The sums of probabilities: at most 64 tokens' are added in fp32, everything above in 64 bits."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24


@pytest.mark.parametrize("E,T", [(8, 16), (64, 128), (8, 144), (64, 1000), (100, 16), (100, 300), (200, 16), (200, 48), (200, 512),
                                 (400, 8), (400, 64), (1000, 4), (1000, 40), (2048, 60)])
@pytest.mark.parametrize("S", [1, 3])
def test_small_terms_beside_a_large_one(E, T, S):
    """One token of each segment has p = 1 at id 0, the others 0.9 of half a step of it shared by all of a lane's: added to the
    one in fp32 each would be lost.  The workgroup's sum and the result are rounded, the small terms are good to 72 steps."""
    print(f"[sums] {E} {T} {S}", flush=True)
    lanes = 16 if E <= 256 else 32 if E <= 512 else 64
    at_once = 4 * 64 // lanes
    p = 0.9 * HALF / -(-T // at_once)
    l = torch.full((S, T, E), -np.inf)
    l[:, :, 1] = 0.0
    l[:, :, 0] = float(np.log(p / (1 - p)))
    l[:, 0, 0], l[:, 0, 1] = 0.0, -np.inf
    l = l.view(S * T, E)
    s64 = torch.softmax(l.double(), 1).view(S, T, E)
    want = s64.sum(1).numpy()
    ids = torch.zeros(S * T, 1, dtype=torch.int32)
    shape = mg.make_route_shape(S * T, E, 1)
    b = mg.balance_loss(shape, mg.make_balance(S, 1.0, 0.0), l.to(X.DEV), ids.to(X.DEV))
    small = float(s64[0, 1:, 0].sum())
    got = b.prob_sums.cpu().double().numpy()
    assert (np.abs(got[:, 0] - want[:, 0]) <= 2 * HALF * want[:, 0] + 72 * 2 * HALF * small).all(), (got[:, 0] - want[:, 0]) / HALF
    assert b.counts[:, 0].tolist() == [T] * S and b.segment_tokens.tolist() == [T] * S
    loss = E / (S * T) * want[:, 0].sum()  # c = T of T_g = T tokens, at id 0 alone
    assert abs(float(b.losses[0]) - loss) <= 2 * HALF * loss + 72 * 2 * HALF * loss * small
