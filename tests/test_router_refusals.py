"""What the router and the gate refuse, on a machine without a GPU: the C entry points return their status before any
device work; the binding raises before a call is made."""
import ctypes

import pytest
import torch

import combine_moe_get_amd as mg
from combine_moe_get_amd import binding as B
from combine_moe_get_amd import experts, router

ARG, SHAPE, CAPACITY, UNSUPPORTED = -1, -2, -3, -4
p = ctypes.c_void_p(4096)  # an aligned address that is never read
odd = ctypes.c_void_p(4104)
odd2 = ctypes.c_void_p(4098)
n = None


@pytest.mark.parametrize("kw,want", [
    (dict(), 0), (dict(T=0), 0), (dict(T=-1), SHAPE), (dict(T=(1 << 24) - 1), 0), (dict(T=1 << 24), UNSUPPORTED),
    (dict(E=0), SHAPE), (dict(E=2048), 0), (dict(E=2049), UNSUPPORTED), (dict(E=33), 0), (dict(E=4, K=4), 0),
    (dict(E=4, K=5), SHAPE), (dict(K=0), SHAPE), (dict(K=16), 0), (dict(K=17), UNSUPPORTED),
    (dict(groups=0), SHAPE), (dict(groups=3, topk_groups=1), SHAPE), (dict(groups=4, topk_groups=2), 0),
    (dict(groups=4, topk_groups=5), SHAPE), (dict(topk_groups=0), SHAPE), (dict(groups=64, topk_groups=64), 0),
    (dict(E=128, groups=128, topk_groups=128), UNSUPPORTED), (dict(groups=8, topk_groups=1, K=8), 0),
    (dict(groups=8, topk_groups=1, K=9), SHAPE), (dict(score=2), ARG), (dict(score=-1), ARG), (dict(group_score=2), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(scale=0.0), 0), (dict(scale=-1.0), 0),
])
def test_shapes(kw, want):
    a = dict(T=64, E=64, K=8)
    a.update(kw)
    assert mg.check_route_shape(mg.make_route_shape(**a)) == want


def test_shape_flags():
    L = router._lib()
    assert L.moe_route_check_shape(None) == ARG
    s = mg.make_route_shape(64, 64, 8)
    s.renormalize = 2
    assert mg.check_route_shape(s) == ARG


@pytest.mark.parametrize("S,T,some", [(1, 64, True), (64, 64, True), (0, 64, False), (-1, 64, False), (3, 64, False),
                                      (4096, 4096, True), (8192, 8192, False), (7, 0, True)])
def test_workspace(S, T, some):
    n = mg.balance_workspace_size(mg.make_route_shape(T, 64, 8), mg.make_balance(S))
    assert (n > 0) == some
    assert mg.balance_workspace_size(mg.make_route_shape(T, 64, 65), mg.make_balance(1)) == 0


def test_route_refuses():
    L = router._lib()
    s = ctypes.byref(mg.make_route_shape(64, 64, 8))
    f = L.moe_route
    assert f(None, 1, p, n, n, p, p, n) == ARG
    assert f(ctypes.byref(mg.make_route_shape(64, 64, 65)), 1, p, n, n, p, p, n) == SHAPE
    assert f(s, 2, p, n, n, p, p, n) == ARG and f(s, -1, p, n, n, p, p, n) == ARG
    for a in ([n, n, p, p], [odd, n, p, p], [p, odd2, p, p], [p, n, n, p], [p, n, odd2, p], [p, n, p, n], [p, n, p, odd2]):
        assert f(s, 1, a[0], a[1], n, a[2], a[3], n) == ARG
    assert f(ctypes.byref(mg.make_route_shape(0, 64, 8)), 1, n, n, n, n, n, n) == 0


def test_balance_refuses():
    L = router._lib()
    shape, bal = mg.make_route_shape(64, 64, 8), mg.make_balance(4)
    s, b = ctypes.byref(shape), ctypes.byref(bal)
    need = mg.balance_workspace_size(shape, bal)
    f = L.moe_balance_loss

    def call(shape=s, balance=b, fp32=1, bytes=need, **kw):
        a = dict(logits=p, ids=p, mask=n, losses=p, counts=p, sums=p, tokens=p, ws=p)
        a.update(kw)
        return f(shape, balance, fp32, *a.values(), bytes, n)

    assert call(shape=None) == ARG and call(balance=None) == ARG and call(fp32=3) == ARG
    assert call(balance=ctypes.byref(mg.make_balance(5))) == SHAPE
    assert call(balance=ctypes.byref(mg.make_balance(0))) == SHAPE
    big = ctypes.byref(mg.make_route_shape(8192, 64, 8))
    assert call(shape=big, balance=ctypes.byref(mg.make_balance(8192))) == UNSUPPORTED
    assert call(bytes=need - 1) == ARG and call(bytes=0) == ARG
    for k in ("logits", "ids", "losses", "counts", "sums", "tokens", "ws"):
        assert call(**{k: n}) == ARG
        assert call(**{k: odd2}) == ARG
    assert call(logits=odd) == ARG and call(ws=odd) == ARG


def test_route_grad_refuses():
    L = router._lib()
    s, b = ctypes.byref(mg.make_route_shape(64, 64, 8)), ctypes.byref(mg.make_balance(4))
    f = L.moe_route_grad

    def call(shape=s, fp32=1, balance=b, **kw):
        a = dict(logits=p, ids=p, gw=p, dst=n, mask=n, balance=balance, counts=p, tokens=p, gl=n, out=p)
        a.update(kw)
        return f(shape, fp32, *a.values(), n)

    assert call(shape=None) == ARG and call(fp32=2) == ARG
    assert call(balance=ctypes.byref(mg.make_balance(5))) == SHAPE
    assert call(balance=None) == ARG and call(balance=None, counts=n) == ARG and call(balance=None, tokens=n) == ARG
    assert call(balance=None, counts=n, tokens=n, gl=p) == ARG
    assert call(balance=None, counts=n, tokens=n, gw=n) == ARG       # nothing to go back through
    assert call(gw=n, dst=p) == ARG                                  # a map of nothing
    for k in ("logits", "ids", "counts", "tokens", "out"):
        assert call(**{k: n}) == ARG
        assert call(**{k: odd2}) == ARG
    for k in ("gw", "dst", "gl"):
        assert call(**{k: odd2}) == ARG
    assert call(logits=odd) == ARG and call(out=odd) == ARG
    assert call(shape=ctypes.byref(mg.make_route_shape(0, 64, 8)), logits=n, ids=n, gw=n, counts=n, tokens=n, out=n) == 0


def test_swiglu_refuses():
    L = experts._lib()
    f = L.moe_swiglu
    s = ctypes.byref(mg.make_experts_shape(64, 8, 64, 8))
    ok = dict(rows=64, features=64, h0=p, w=n, shape=None, off=n, out=p, codes=n, scales=n)

    def call(**kw):
        return f(*dict(ok, **kw).values(), n)

    assert call(rows=-1) == SHAPE and call(features=0) == SHAPE and call(features=-8) == SHAPE
    assert call(features=12) == UNSUPPORTED and call(features=65544) == UNSUPPORTED and call(rows=1 << 40) == UNSUPPORTED
    assert call(rows=0, h0=n, out=n) == 0
    for k in ("h0", "out"):
        assert call(**{k: n}) == ARG and call(**{k: odd}) == ARG
    assert call(w=odd2) == ARG
    assert call(codes=p) == ARG and call(scales=p) == ARG            # a checkpoint is both
    assert call(codes=odd, scales=p) == ARG and call(codes=p, scales=odd2) == ARG
    assert call(shape=s) == ARG and call(off=p) == ARG and call(shape=s, off=odd2) == ARG
    assert call(rows=65, shape=s, off=p) == SHAPE and call(features=32, shape=s, off=p) == SHAPE
    bad = ctypes.byref(mg.make_experts_shape(64, 8, 64, 8, P=3))
    assert call(shape=bad, off=p) == SHAPE
    assert call(shape=ctypes.byref(mg.make_experts_shape(64, 8, 64, 8, P=2, rank_stride=40)), off=p) == CAPACITY


def test_swiglu_grad_refuses():
    L = experts._lib()
    f = L.moe_swiglu_grad
    s = ctypes.byref(mg.make_experts_shape(64, 8, 64, 8))
    ok = dict(rows=64, features=64, go=p, h0=p, codes=n, scales=n, w=n, shape=None, off=n, gh0=p, out=n, gw=n)

    def call(**kw):
        return f(*dict(ok, **kw).values(), n)

    assert call(rows=-1) == SHAPE and call(features=0) == SHAPE and call(features=12) == UNSUPPORTED
    assert call(rows=0, go=n, h0=n, gh0=n) == 0
    assert call(go=n) == ARG and call(go=odd) == ARG and call(h0=odd) == ARG
    assert call(h0=n) == ARG                                         # neither
    assert call(codes=p, scales=p) == ARG                            # both
    assert call(h0=n, codes=p) == ARG and call(h0=n, scales=p) == ARG and call(codes=p) == ARG and call(scales=p) == ARG
    assert call(h0=n, codes=odd, scales=p) == ARG and call(h0=n, codes=p, scales=odd2) == ARG
    assert call(gh0=n) == ARG                                        # nothing asked for
    assert call(gh0=odd) == ARG and call(out=odd) == ARG and call(gw=odd2) == ARG and call(w=odd2) == ARG
    assert call(shape=s) == ARG and call(off=p) == ARG and call(rows=65, shape=s, off=p) == SHAPE


def test_binding_refuses():
    s = mg.make_route_shape(4, 8, 2)
    l, ids, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for f in (lambda: mg.route(s, l), lambda: mg.balance_loss(s, mg.make_balance(), l, ids),
              lambda: mg.route_grad(s, l, ids, w), lambda: mg.swiglu(torch.zeros(2, 16, dtype=torch.bfloat16)),
              lambda: mg.swiglu_grad(torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(2, 16, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="device"):
            f()
    with pytest.raises(TypeError):
        mg.route(s, None)
    with pytest.raises(TypeError):
        mg.swiglu(None)



@pytest.fixture
def on_device(monkeypatch):
    monkeypatch.setattr(router, "_device_of", lambda t, name: t.device)
    monkeypatch.setattr(experts, "_device_of", lambda t, name: t.device)


def test_binding_refuses_arguments_that_do_not_go_together(on_device):
    s = mg.make_route_shape(4, 8, 2)
    l, ids, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    bal = mg.make_balance()
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        mg.prepare_route(s, l.half())
    with pytest.raises(B.MoeGetError):
        mg.prepare_route(mg.make_route_shape(4, 8, 9), l)
    with pytest.raises(B.MoeGetError):
        mg.prepare_balance_loss(s, mg.make_balance(3), l, ids)
    with pytest.raises(ValueError, match="go together"):
        mg.prepare_route_grad(s, l, ids, w, balance=bal)
    with pytest.raises(ValueError, match="needed where there are no losses"):
        mg.prepare_route_grad(s, l, ids)
    with pytest.raises(ValueError, match="grad_losses needs"):
        mg.prepare_route_grad(s, l, ids, w, grad_losses=torch.ones(2))
    with pytest.raises(ValueError, match="dst_row needs"):
        mg.prepare_route_grad(s, l, ids, None, bal, (None,), dst_row=ids)
    h, d = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(2, 16, dtype=torch.bfloat16)
    e, off = mg.make_experts_shape(2, 1, 16, 8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: mg.prepare_swiglu(h, shape=e), lambda: mg.prepare_swiglu(h, expert_offsets=off),
                 lambda: mg.prepare_swiglu_grad(d, h, shape=e)):
        with pytest.raises(ValueError, match="go together"):
            call()
    with pytest.raises(ValueError, match="multiple of 16"):
        mg.prepare_swiglu(torch.zeros(2, 24, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="2 \\* features"):
        mg.prepare_swiglu(torch.zeros(32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="results of a checkpoint"):
        mg.prepare_swiglu(h, codes=h.to(torch.int8))
    with pytest.raises(ValueError, match="either h0 or codes"):
        mg.prepare_swiglu_grad(d)
    with pytest.raises(ValueError, match="either h0 or codes"):
        mg.prepare_swiglu_grad(d, h, codes=h.to(torch.int8), scales=torch.zeros(2, 2, 1))
    with pytest.raises(ValueError, match="need_out"):
        mg.prepare_swiglu_grad(d, h, out=d, need_out=False)


NAMES = {"route": (router, 2), "balance_loss": (router, 4), "route_grad": (router, 3), "swiglu": (experts, 1),
         "swiglu_grad": (experts, 1)}


@pytest.mark.parametrize("name", list(NAMES))
def test_the_functions_go_through_call_on(name, monkeypatch):
    seen = []
    module, required = NAMES[name]
    monkeypatch.setattr(B, "call_on", lambda stream, prepare, *args: seen.append((stream, prepare)))
    getattr(module, name)(*[None] * required, stream="s")
    assert seen == [("s", getattr(module, "prepare_" + name))]
