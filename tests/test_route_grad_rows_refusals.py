"""What the logits' gradient from receive rows refuses and how the binding counts the rows, on a machine without a GPU."""
import ctypes

import pytest
import torch

import combine_moe_get_amd as mg
from combine_moe_get_amd import experts, router

ARG, SHAPE = -1, -2
p = ctypes.c_void_p(4096)  # an aligned address that is never read
odd2 = ctypes.c_void_p(4098)
n = None


def call(T=64, fp32=1, balance=None, **kw):
    a = dict(logits=p, ids=p, gw=p, rows=512, dst=p, mask=n, balance=balance, counts=n, tokens=n, gl=n, out=p)
    a.update(kw)
    return router._lib().moe_route_grad_rows(ctypes.byref(mg.make_route_shape(T, 64, 8)), fp32, *a.values(), n)


def test_refusals():
    assert router._lib().moe_route_grad_rows(None, 1, p, p, p, 1, p, *[n] * 5, p, n) == ARG
    assert call(rows=-1) == SHAPE and call(rows=-2 ** 40) == SHAPE
    assert call(dst=n) == ARG and call(gw=n) == ARG and call(rows=0, dst=n) == ARG
    assert call(fp32=2) == ARG
    for k in ("logits", "ids", "gw", "dst", "out"):
        assert call(**{k: odd2}) == ARG
    for k in ("logits", "ids", "out"):
        assert call(**{k: n}) == ARG
    b = ctypes.byref(mg.make_balance(4))
    assert call(counts=p) == ARG and call(gl=p) == ARG                # losses without their coefficients
    assert call(balance=b, counts=p) == ARG and call(balance=b, tokens=p) == ARG
    assert call(balance=ctypes.byref(mg.make_balance(5)), counts=p, tokens=p) == SHAPE
    assert call(T=0, rows=0, gw=n, dst=n, logits=n, ids=n, out=n) == 0
    assert call(T=0, rows=-1) == SHAPE


@pytest.mark.parametrize("rows", [0, 1, 5, 8, 100])
def test_the_binding_gives_the_rows_that_there_are(rows, monkeypatch):
    monkeypatch.setattr(router, "_device_of", lambda t, name: t.device)
    s = mg.make_route_shape(4, 8, 2)
    l, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    c = mg.prepare_route_grad(s, l, ids, torch.zeros(rows), dst_row=ids)
    assert c._fn is experts._lib().moe_route_grad_rows and c._args[5] == rows
    assert c._args[6] == ids.data_ptr() and c._args[4] == (c._keep[3].data_ptr() or None)
    c = mg.prepare_route_grad(s, l, ids, torch.zeros(4, 2))
    assert c._fn is experts._lib().moe_route_grad and len(c._args) == 13
    with pytest.raises(ValueError):
        mg.prepare_route_grad(s, l, ids, torch.zeros(rows), dst_row=torch.zeros(7, dtype=torch.int32))


def test_more_rows_than_a_map_can_name():
    assert call(rows=2 ** 31) == -4 and call(rows=2 ** 62) == -4 and call(T=0, rows=2 ** 31) == -4
