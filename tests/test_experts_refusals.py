"""What the expert stage refuses, on a machine without a GPU: the C entry points return their status
before any device work; the binding raises before a call is made."""
import ctypes

import pytest
import torch

import combine_moe_get_amd as mg

ARG, SHAPE, CAPACITY, UNSUPPORTED = -1, -2, -3, -4
p = ctypes.c_void_p(4096)  # an aligned address that is never read
odd = ctypes.c_void_p(4104)
n = None


def _lib():
    from combine_moe_get_amd import experts

    return experts._lib()


@pytest.mark.parametrize("kw,row_type,want", [
    (dict(), 0, 0), (dict(), 1, 0), (dict(), 2, 0),
    (dict(rows=0), 0, 0),
    (dict(rows=-1), 0, SHAPE),
    (dict(rows=1 << 27), 0, UNSUPPORTED),
    (dict(E=0), 0, SHAPE), (dict(E=2049), 0, SHAPE), (dict(E=2048), 0, 0),
    (dict(P=0), 0, SHAPE), (dict(P=3), 0, SHAPE),
    (dict(P=2, rank_stride=32), 0, 0), (dict(P=2, rank_stride=33), 0, CAPACITY), (dict(rank_stride=-1), 0, SHAPE),
    (dict(in_features=0), 0, SHAPE), (dict(out_features=0), 0, SHAPE), (dict(in_features=-8), 0, SHAPE),
    (dict(in_features=72), 0, 0), (dict(in_features=72), 1, UNSUPPORTED), (dict(in_features=80), 1, 0),
    (dict(in_features=80), 2, UNSUPPORTED), (dict(in_features=68), 0, UNSUPPORTED),
    (dict(out_features=12), 0, UNSUPPORTED), (dict(in_features=65544), 0, UNSUPPORTED), (dict(in_features=65536), 0, 0),
    (dict(out_features=65544), 0, UNSUPPORTED), (dict(), 3, ARG), (dict(), -1, ARG),
])
def test_shapes(kw, row_type, want):
    a = dict(rows=64, E=8, in_features=64, out_features=24)
    a.update(kw)
    assert mg.check_experts_shape(mg.make_experts_shape(**a), row_type) == want


def test_null_shape():
    assert _lib().moe_experts_check_shape(None, 0) == ARG


def test_products_refuse():
    L, s = _lib(), ctypes.byref(mg.make_experts_shape(64, 8, 64, 24))
    mm = L.moe_experts_matmul
    assert mm(s, 0, 2, p, n, p, n, p, p, n) == ARG       # no such activation
    assert mm(s, 3, 0, p, n, p, n, p, p, n) == ARG       # no such type
    assert mm(s, 0, 0, p, p, p, n, p, p, n) == ARG       # bf16 rows take no scales
    for i in range(4):                                   # a buffer missing, a buffer misaligned
        for bad in (n, odd):
            if i == 2 and bad is odd:
                continue
            a = [p, p, p, p]
            a[i] = bad
            assert mm(s, 0, 0, a[0], n, a[1], n, a[2], a[3], n) == ARG
    assert mm(s, 0, 0, p, n, p, n, ctypes.c_void_p(4098), p, n) == ARG
    assert mm(s, 1, 0, p, ctypes.c_void_p(4098), p, n, p, p, n) == ARG
    assert mm(s, 2, 0, p, n, p, p, p, p, n) == ARG       # 4-bit rows need both scales
    assert mm(s, 2, 0, p, p, p, n, p, p, n) == ARG
    for a in ([n, p, p, p], [p, n, p, p], [p, p, n, p], [p, p, p, n], [odd, p, p, p], [p, odd, p, p], [p, p, p, odd]):
        assert L.moe_experts_matmul_dgrad(s, *a, n) == ARG
        assert L.moe_experts_matmul_wgrad(s, 0, *a, n) == ARG
    assert L.moe_experts_matmul_wgrad(s, 2, p, p, p, p, n) == ARG
    none = ctypes.byref(mg.make_experts_shape(0, 8, 64, 24))
    assert mm(none, 0, 0, n, n, n, n, n, n, n) == 0      # no rows: nothing to do, no buffer looked at
    assert L.moe_experts_matmul_dgrad(none, n, n, n, n, n) == 0
    assert L.moe_experts_matmul_wgrad(none, 0, n, n, n, n, n) == ARG  # its zeros have to go somewhere


def test_quantize_refuses():
    L = _lib()
    q = L.moe_quantize_rows
    s = ctypes.byref(mg.make_experts_shape(64, 8, 64, 24))
    assert q(0, 64, 64, p, p, p, None, n, n) == ARG
    assert q(1, -1, 64, p, p, p, None, n, n) == SHAPE
    assert q(1, 64, 0, p, p, p, None, n, n) == SHAPE
    assert q(1, 64, 72, p, p, p, None, n, n) == UNSUPPORTED
    assert q(2, 64, 80, p, p, p, None, n, n) == UNSUPPORTED
    assert q(2, 64, 65568, p, p, p, None, n, n) == UNSUPPORTED
    assert q(1, 1 << 40, 64, p, p, p, None, n, n) == UNSUPPORTED
    for a in ([n, p, p], [p, n, p], [p, p, n], [odd, p, p], [p, odd, p]):
        assert q(1, 64, 64, *a, None, n, n) == ARG
    assert q(1, 64, 64, p, p, ctypes.c_void_p(4098), None, n, n) == ARG
    assert q(1, 64, 64, p, p, p, s, n, n) == ARG
    assert q(1, 64, 64, p, p, p, None, p, n) == ARG
    assert q(1, 65, 64, p, p, p, s, p, n) == SHAPE
    assert q(1, 64, 32, p, p, p, s, p, n) == SHAPE
    assert q(1, 0, 64, n, n, n, None, n, n) == 0


def test_combine_grad_refuses():
    L = _lib()
    cg = L.moe_combine_grad
    plain, special = mg.make_shape(64, 64, 4, 8, 2), mg.make_shape(64, 64, 4, 8, 2, 0, 1, 1)

    def call(shape, **kw):
        a = dict(go=p, y=p, ids=p, w=p, mask=n, dst=p, x=p, a1=p, a2=p, v=p, gy=p, gw=p, gx=n, ga1=n, ga2=n, gv=n)
        a.update(kw)
        return cg(ctypes.byref(shape), *a.values(), n)

    assert call(mg.make_shape(64, 60, 4, 8, 2)) == UNSUPPORTED
    assert call(mg.make_shape(65, 64, 4, 8, 2)) == SHAPE
    assert call(plain, gy=n, gw=n) == ARG               # nothing asked for
    assert call(plain, ga1=p) == ARG                    # no constant expert to have a gradient
    for k in ("go", "y", "ids", "w", "dst"):
        assert call(plain, **{k: n}) == ARG
    for k in ("go", "y", "gy"):
        assert call(plain, **{k: odd}) == ARG
    assert call(plain, gw=ctypes.c_void_p(4098)) == ARG
    for k in ("x", "a1", "a2", "v"):
        assert call(special, **{k: n}) == ARG
        assert call(special, **{k: odd}) == ARG
    assert call(special, gx=odd) == ARG


def test_binding_refuses_what_is_not_on_the_device_or_of_another_type():
    s = mg.make_experts_shape(4, 2, 64, 24)
    x, w, off = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 24, 64, dtype=torch.bfloat16), \
        torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        mg.experts_matmul(s, x, w, off)
    with pytest.raises(TypeError):
        mg.experts_matmul(s, None, w, off)
    with pytest.raises(ValueError, match="device"):
        mg.quantize_rows(x, mg.ROWS_INT8)
    with pytest.raises(ValueError, match="device"):
        mg.combine_grad(mg.make_shape(4, 64, 2, 4, 1), x, x, off, off, off)
