"""The losses that the logits' gradient is given have to be of its own segments and ids (no GPU)."""
import pytest
import torch

import combine_moe_get_amd as mg
from combine_moe_get_amd import router


def loss(S, E):
    return mg.BalanceLoss(torch.zeros(2), torch.zeros(S, E, dtype=torch.int32), torch.zeros(S, E), torch.zeros(S, dtype=torch.int32))


@pytest.mark.parametrize("made,ok", [((4, 8), True), ((1, 8), False), ((2, 8), False), ((8, 8), False), ((64, 8), False),
                                     ((4, 16), False), ((4, 4), False), ((2, 16), False), ((8, 4), False)])
def test_segments_and_ids(made, ok, monkeypatch):
    monkeypatch.setattr(router, "_device_of", lambda t, name: t.device)
    s = mg.make_route_shape(64, 8, 2)
    l, ids = torch.zeros(64, 8), torch.zeros(64, 2, dtype=torch.int32)
    for gw in (None, torch.zeros(64, 2)):
        if ok:
            mg.prepare_route_grad(s, l, ids, gw, mg.make_balance(4), loss(*made))
        else:
            with pytest.raises(ValueError, match="4 segments of 8 ids"):
                mg.prepare_route_grad(s, l, ids, gw, mg.make_balance(4), loss(*made))
