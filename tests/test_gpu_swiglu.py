"""The gate, its 8-bit checkpoint and its gradient against the definitions: codes and scales exactly, the rest in 64 bits."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X

pytestmark = pytest.mark.gpu

STEP32, HALF = X.STEP32, X.BF16_HALF


def logistic(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, e) / (1 + e), np.where(g >= 0, e, 1.0) / (1 + e)  # and 1 - it


def forward(h0, w):
    """(reference, error before the rounding): the logistic function is good to |g| + 8 steps, four products follow."""
    n = h0.shape[1] // 2
    g, u = h0[:, :n], h0[:, n:]
    s, _ = logistic(g)
    ref = s * g * u * w[:, None]
    return ref, np.abs(ref) * (np.abs(g) + 13) * STEP32 + X.TINY


def backward(h0, w, d):
    n = h0.shape[1] // 2
    g, u = h0[:, :n], h0[:, n:]
    s, rest = logistic(g)
    w = w[:, None]
    dg, du = w * d * u * s * (1 + g * rest), w * d * g * s
    # 1 + g (1 - s): its terms' sizes, each good to |g| + 9 steps
    eg = np.abs(w * d * u * s) * (1 + np.abs(g) * rest) * (np.abs(g) + 16) * STEP32 + X.TINY
    eu = np.abs(du) * (np.abs(g) + 13) * STEP32 + X.TINY
    row = d * s * g * u
    gw = row.sum(1)
    ew = (np.abs(row) * (np.abs(g) + 13 + n / 8 + 16)).sum(1) * STEP32 + X.TINY * n
    return np.concatenate((dg, du), 1), np.concatenate((eg, eu), 1), gw, ew


def codes_of(h0):
    """The checkpoint of h0 float32 [rows, 2 n], each operation rounded once to binary32: codes, scales, values."""
    rows, n = h0.shape[0], h0.shape[1] // 2
    nb = (n + 127) // 128
    x = np.zeros((rows, 2, nb * 128), np.float32)
    x[:, :, :n] = h0.reshape(rows, 2, n)
    x = x.reshape(rows, 2, nb, 128)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        amax = np.fmax.reduce(np.abs(x), 3)
        amax = np.where(np.isnan(amax), np.float32(0), amax)
        dyn = np.where(amax > 0, np.float32(127) * (np.float32(1) / amax), np.float32(0)).astype(np.float32)
        p = np.rint(x * dyn[..., None])
        code = np.clip(np.where(np.isnan(p), 0, p), -127, 127).astype(np.int8)
        scale = np.where(amax > 0, np.float32(1) / dyn, np.float32(0)).astype(np.float32)
        value = code.astype(np.float32) * scale[..., None]
    cut = lambda a: a.reshape(rows, 2, nb * 128)[:, :, :n].reshape(rows, 2 * n)  # noqa: E731
    return cut(code), scale, cut(value)


def close(got, ref, err, used, what):
    X.check(got, ref, err + HALF * (np.abs(ref) + err), used, what)


def world(seed, rows, n, weights=True):
    r = np.random.default_rng(seed)
    h0 = X.bf16(r, rows, 2 * n) * torch.from_numpy(np.exp(r.uniform(-2, 2, (rows, 1)))).bfloat16()
    w = torch.from_numpy(r.uniform(-1, 1, rows).astype(np.float32)) if weights else None
    return r, h0, w, X.bf16(r, rows, n)


def run(L, n, weights, seed, kept):
    """Forward and backward over the rows of a layout, everything compared."""
    r, h0, w, d = world(seed, L.rows, n, weights)
    w64 = np.ones(L.rows) if w is None else X.f64(w)
    shape, off, used = L.shape(n, 8), L.dev_off(), L.used
    poisoned = X.poison(h0, used).to(X.DEV)
    wd = None if w is None else X.poison(w, used).to(X.DEV)
    nb = (n + 127) // 128
    out = X.canary(L.rows, n)
    codes = torch.full((L.rows, 2 * n), 99, dtype=torch.int8, device=X.DEV)
    scales = torch.full((L.rows, 2, nb), -7.0, device=X.DEV)
    f = mg.swiglu(poisoned, wd, checkpoint=kept, shape=shape, expert_offsets=off, out=out,
                  codes=codes if kept else None, scales=scales if kept else None)
    ref, err = forward(X.f64(h0), w64)
    close(f.out, ref, err, used, "out")
    at = h0.float().numpy()
    if kept:
        c, s, at = codes_of(at)
        got = f.codes.cpu().numpy()
        assert np.array_equal(got[used], c[used]) and (got[~used] == 99).all()
        got = f.scales.cpu().numpy()
        assert np.array_equal(got[used], s[used]) and (got[~used] == -7).all()
    at = at.astype(np.float64)
    gw = torch.full((L.rows,), -7.0, device=X.DEV) if weights else None
    keep = dict(codes=f.codes, scales=f.scales) if kept else dict(h0=poisoned)
    g = mg.swiglu_grad(X.poison(d, used).to(X.DEV), **keep, row_weights=wd, shape=shape, expert_offsets=off,
                       grad_h0=X.canary(L.rows, 2 * n), out=X.canary(L.rows, n), grad_row_weights=gw)
    dh, eh, dw, ew = backward(at, w64, X.f64(d))
    close(g.grad_h0, dh, eh, used, "grad_h0")
    ref, err = forward(at, w64)
    close(g.out, ref, err, used, "out again")
    if weights:
        got = g.grad_row_weights.cpu().double().numpy()
        assert (np.abs(got - dw)[used] <= ew[used]).all() and (got[~used] == -7).all()
    else:
        assert g.grad_row_weights is None


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("n", [8, 16, 120, 128, 136, 256, 520, 1024, 1032, 2056, 4096, 8200])
@pytest.mark.parametrize("window", [False, True])
def test_rows_of_experts(n, kept, window):
    print(f"[swiglu] {n} {kept} {window}", flush=True)
    L = X.Rows([3, 0, 1, 9, 0, 17], P=2 if window else 1, slack=4 if window else None)
    run(L, n, True, [n, 1], kept)
    run(L, n, False, [n, 2], kept)


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("rows,n", [(1, 8), (1, 65536), (2, 128), (1000, 72), (4097, 136), (300, 2048)])
def test_all_rows(rows, n, kept):
    print(f"[swiglu] {rows} {n} {kept}", flush=True)
    r, h0, w, d = world([rows, n], rows, n)
    f = mg.swiglu(h0.to(X.DEV), w.to(X.DEV), checkpoint=kept)
    used = np.ones(rows, bool)
    close(f.out, *forward(X.f64(h0), X.f64(w)), used, "out")
    at = h0.float().numpy()
    if kept:
        c, s, at = codes_of(at)
        assert np.array_equal(f.codes.cpu().numpy(), c) and np.array_equal(f.scales.cpu().numpy(), s)
        g = mg.swiglu_grad(d.to(X.DEV), codes=f.codes, scales=f.scales, row_weights=w.to(X.DEV))
    else:
        assert f.codes is None and f.scales is None
        g = mg.swiglu_grad(d.to(X.DEV), h0.to(X.DEV), row_weights=w.to(X.DEV))
    at = at.astype(np.float64)
    dh, eh, dw, ew = backward(at, X.f64(w), X.f64(d))
    close(g.grad_h0, dh, eh, used, "grad_h0")
    close(g.out, *forward(at, X.f64(w)), used, "out again")
    assert (np.abs(g.grad_row_weights.cpu().double().numpy() - dw) <= ew).all()


def test_no_rows():
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=X.DEV)  # noqa: E731
    f = mg.swiglu(e(0, 32), checkpoint=True)
    assert f.out.shape == (0, 16) and f.codes.shape == (0, 32) and f.scales.shape == (0, 2, 1)
    g = mg.swiglu_grad(e(0, 16), codes=f.codes, scales=f.scales)
    assert g.grad_h0.shape == (0, 32)
    L = X.Rows([0, 0, 0])
    out = mg.swiglu(e(L.rows, 32), shape=L.shape(16, 8), expert_offsets=L.dev_off(), out=X.canary(L.rows, 16)).out
    assert bool((out == -7).all())


def test_results_one_by_one():
    r, h0, w, d = world(3, 40, 264)
    h0, w, d = h0.to(X.DEV), w.to(X.DEV), d.to(X.DEV)
    whole = mg.swiglu_grad(d, h0, row_weights=w)
    assert mg.swiglu_grad(d, h0, row_weights=w, need_out=False).out is None
    assert torch.equal(mg.swiglu_grad(d, h0, row_weights=w, need_out=False).grad_h0, whole.grad_h0)
    from combine_moe_get_amd import experts

    s = torch.cuda.current_stream().cuda_stream
    for k in range(3):  # through the C entry point: each output alone
        o = [torch.empty_like(t) if i == k else None for i, t in enumerate(whole)]
        p = [t.data_ptr() if t is not None else None for t in o]
        assert experts._lib().moe_swiglu_grad(40, 264, d.data_ptr(), h0.data_ptr(), None, None, w.data_ptr(), None, None, *p, s) == 0
        assert torch.equal(o[k], whole[k])


def test_against_differences():
    """grad_h0 against central differences of the definition in 64 bits, h = 1e-3: off by h^2 / 6 times a third derivative
    of at most 1, and by the gradient's own bf16 rounding."""
    r, h0, w, d = world(5, 6, 24)
    g = mg.swiglu_grad(d.to(X.DEV), h0.to(X.DEV), row_weights=w.to(X.DEV))
    base, w64, d64, h = X.f64(h0), X.f64(w), X.f64(d), 1e-3
    f = lambda x, ww: (forward(x, ww)[0] * d64).sum(1)  # noqa: E731
    got = X.f64(g.grad_h0.cpu())
    for i in range(48):
        up, down = base.copy(), base.copy()
        up[:, i] += h
        down[:, i] -= h
        want = (f(up, w64) - f(down, w64)) / (2 * h)
        size = np.abs(w64 * d64[:, i % 24]) * (1 + np.abs(base[:, (i + 24) % 48]))
        assert (np.abs(got[:, i] - want) <= HALF * np.abs(want) + (h * h + 2 ** -18) * size + 1e-9).all()
    want = (f(base, w64 + h) - f(base, w64 - h)) / (2 * h)
    assert np.allclose(X.f64(g.grad_row_weights.cpu()), want, rtol=1e-5, atol=1e-5 * np.abs(want).max())


G = [-200.0, -187.0, -181.0, -176.0, -174.0, -150.0, -120.0, -100.0, -89.0, -88.0, -87.0, -60.0, -17.0, -2.0, -1.25, -1.0,
     -2.0 ** -100, 0.0, 2.0 ** -100, 1.0, 17.0, 88.0, 100.0, 2.0 ** 100]
U = [s * 2.0 ** e for e in (-100, -20, 0, 20, 60, 100, 115, 127) for s in (1.0, -1.5)]


def test_over_the_range():
    """g and u far out: where exp(g) leaves fp32 but the results do not."""
    pairs = np.array([(g, u) for g in G for u in U])
    pairs = np.concatenate((pairs, np.zeros(((-len(pairs)) % 8, 2))))
    g, u = pairs.T
    h0 = torch.from_numpy(np.concatenate((g, u))[None]).bfloat16()
    assert np.array_equal(X.f64(h0)[0], np.concatenate((g, u)))
    s, rest = logistic(g)
    got = [X.f64(mg.swiglu(h0.to(X.DEV)).out.cpu())[0]]
    d = torch.ones(1, len(g), dtype=torch.bfloat16)
    gr = mg.swiglu_grad(d.to(X.DEV), h0.to(X.DEV))
    got += [X.f64(gr.out.cpu())[0], *X.f64(gr.grad_h0.cpu())[0].reshape(2, -1)]
    top = float(torch.finfo(torch.bfloat16).max) * (1 + HALF)
    # below -174 each half of the exponential is subnormal, with 2^-149 / 2 of error and, for a result that bf16 holds, at
    # least 2^-134 large
    far = np.where(g < -174, 2.0 ** -15, 0.0)
    with np.errstate(over="ignore", invalid="ignore"):
        for name, y, ref, size in (("out", got[0], g * s * u, 1.0), ("again", got[1], g * s * u, 1.0),
                                   ("dg", got[2], u * s * (1 + g * rest), (1 + np.abs(g) * rest) / np.abs(1 + g * rest)),
                                   ("du", got[3], g * s, 1.0)):
            err = np.abs(ref) * size * ((np.abs(g) + 16) * STEP32 + far)
            tol = err + HALF * (np.abs(ref) + err) + X.TINY
            bad = np.where(np.abs(ref) > top, y != np.sign(ref) * np.inf, ~(np.abs(y - ref) <= tol))
            assert not bad.any(), (name, [(*pairs[i], y[i], ref[i]) for i in np.flatnonzero(bad)[:5]])


def test_blocks_that_are_zero_or_not_finite():
    n = 272
    r = np.random.default_rng(11)
    h0 = X.bf16(r, 6, 2 * n)
    h0[0, :128] = 0
    h0[1, n:] = 0
    h0[2] *= torch.tensor(2.0 ** -130).bfloat16()  # amaxes whose reciprocals leave fp32
    h0[3, 5] = float("inf")
    h0[4, 300] = float("nan")
    h0[5, :] = 3.0e38
    f = mg.swiglu(h0.to(X.DEV), checkpoint=True)
    c, s, _ = codes_of(h0.float().numpy())
    assert np.array_equal(f.codes.cpu().numpy(), c)
    assert np.array_equal(f.scales.cpu().numpy(), s)


def test_every_amax():
    """Blocks with every finite bf16 as their largest: dyn and scale are two roundings of it, the codes one more."""
    top = torch.from_numpy(np.arange(1, 0x7f80, dtype=np.int16)).view(torch.bfloat16)
    top = torch.cat((top, top[-1:]))  # an even number: two halves a row
    r = np.random.default_rng(17)
    x = torch.from_numpy(r.uniform(-1, 1, (len(top), 128)).astype(np.float32)) * top.float()[:, None]
    x = x.bfloat16()
    x[:, 7] = top
    x[:, 50] = -top / 2  # half of it, exactly
    h0 = x.view(-1, 256)
    f = mg.swiglu(h0.to(X.DEV), checkpoint=True)
    c, s, _ = codes_of(h0.float().numpy())
    assert np.array_equal(f.scales.cpu().numpy(), s)
    assert np.array_equal(f.codes.cpu().numpy(), c)


def test_gradient_from_the_largest_and_the_smallest_checkpoints():
    """Blocks of bf16's largest values, whose scale times 128 leaves fp32, and of its smallest."""
    n = 136
    r = np.random.default_rng(13)
    h0 = X.bf16(r, 6, 2 * n)
    h0[0, n:] = 3.3895e38 * torch.sign(h0[0, n:])
    h0[1, n:] *= 2.0 ** 124  # finite still
    h0[2, n:] = 3.3895e38
    h0[3] *= torch.tensor(2.0 ** -118).bfloat16()
    h0[4, :n] = -3.3895e38
    w, d = torch.ones(6), X.bf16(r, 6, n, scale=2.0 ** -20)
    f = mg.swiglu(h0.to(X.DEV), checkpoint=True)
    c, s, at = codes_of(h0.float().numpy())
    assert np.array_equal(f.codes.cpu().numpy(), c) and np.array_equal(f.scales.cpu().numpy(), s)
    g = mg.swiglu_grad(d.to(X.DEV), codes=f.codes, scales=f.scales)
    at = at.astype(np.float64)
    assert np.isfinite(at).all()
    dh, eh, _, _ = backward(at, X.f64(w), X.f64(d))
    close(g.grad_h0, dh, eh, np.ones(6, bool), "grad_h0")


def test_rows_beyond_32_bits_of_offset():
    """Rows whose bytes begin past 2^32, in every buffer."""
    n, rows = 32768, 69000
    r, h0, w, d = world(8, 64, n)
    big = lambda k, dt: torch.zeros(rows, k, dtype=dt, device=X.DEV)  # noqa: E731
    hb, db, wb = big(2 * n, torch.bfloat16), big(n, torch.bfloat16), torch.zeros(rows, device=X.DEV)
    hb[-64:], db[-64:], wb[-64:] = h0.to(X.DEV), d.to(X.DEV), w.to(X.DEV)
    f = mg.swiglu(hb, wb, checkpoint=True)
    g = mg.swiglu_grad(db, codes=f.codes, scales=f.scales, row_weights=wb)
    sf = mg.swiglu(h0.to(X.DEV), w.to(X.DEV), checkpoint=True)
    sg = mg.swiglu_grad(d.to(X.DEV), codes=sf.codes, scales=sf.scales, row_weights=w.to(X.DEV))
    for a, b in zip((*f, *g), (*sf, *sg)):
        assert torch.equal(a[-64:], b)
        assert bool((a[-128:-64] == 0).all())
