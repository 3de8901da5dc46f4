"""The combine's gradient against its definition in 64 bits: masks, dropped and bad ids, repeated experts,
zero / copy / constant experts, windows, odd hidden sizes; rows that hold no copy keep their values."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X
from tests import _gpu as G

pytestmark = pytest.mark.gpu


def _world(seed, T, H, K, E, Z, C, Kc, mask, repeat=False, bad=False):
    r = np.random.default_rng(seed)
    etot = E + Z + C + Kc
    ids = r.integers(0, etot, (T, K)) if repeat else np.argsort(r.random((T, etot)), axis=1)[:, :K]
    ids = ids.astype(np.int32)
    ids[r.random((T, K)) < 0.05] = -1
    if bad:
        ids[r.random((T, K)) < 0.05] = etot + 7
    m = (r.random(T) < mask).astype(np.uint8) if mask < 1 else None
    b = lambda *s: X.bf16(r, *s)  # noqa: E731
    return dict(ids=ids, mask=m, w=r.uniform(-1, 1, (T, K)).astype(np.float32), go=b(T, H), x=b(T, H), a1=b(Kc, H),
                a2=b(Kc, H), v=b(Kc, H), r=r)


def _definition(d, y, dst, E, Z, C, Kc):
    """Reference values, and the sums of magnitudes that bound their errors."""
    T, K = d["ids"].shape
    go, x, a1, a2, v, y = (X.f64(t) for t in (d["go"], d["x"], d["a1"], d["a2"], d["v"], y))
    H = go.shape[1]
    w = d["w"].astype(np.float64)
    gy, gw, gx = np.zeros_like(y), np.zeros((T, K)), np.zeros((T, H))
    mw, mx = np.zeros((T, K)), np.zeros((T, H))
    ga1, ga2, gv, m1, mg_ = (np.zeros((Kc, H)) for _ in range(5))
    named = np.zeros(len(y), bool)
    for t in range(T):
        if d["mask"] is not None and not d["mask"][t]:
            continue
        for j in range(K):
            i, g = int(d["ids"][t, j]), go[t]
            if 0 <= i < E and dst[t, j] >= 0:
                named[dst[t, j]] = True
                gy[dst[t, j]] = w[t, j] * g
                gw[t, j], mw[t, j] = g @ y[dst[t, j]], np.abs(g) @ np.abs(y[dst[t, j]])
            elif E + Z <= i < E + Z + C:
                gw[t, j], mw[t, j] = g @ x[t], np.abs(g) @ np.abs(x[t])
                gx[t] += w[t, j] * g
                mx[t] += np.abs(w[t, j] * g)
            elif E + Z + C <= i < E + Z + C + Kc:
                k = i - E - Z - C
                gw[t, j] = g @ (a1[k] * x[t] + a2[k] * v[k])
                mw[t, j] = np.abs(g) @ (np.abs(a1[k] * x[t]) + np.abs(a2[k] * v[k]))
                gx[t] += w[t, j] * a1[k] * g
                mx[t] += np.abs(w[t, j] * a1[k] * g)
                ga1[k] += w[t, j] * g * x[t]
                m1[k] += np.abs(w[t, j] * g * x[t])
                ga2[k] += w[t, j] * g * v[k]
                gv[k] += w[t, j] * g * a2[k]
                mg_[k] += np.abs(w[t, j] * g)
    return dict(gy=gy, gw=gw, gx=gx, ga1=ga1, ga2=ga2, gv=gv, named=named, mw=mw, mx=mx, m1=m1,
                m2=mg_ * np.abs(v), mv=mg_ * np.abs(a2))


def _near(got, ref, tol, what):
    got = got.cpu().double().numpy()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, by up to {np.abs(got - ref)[bad].max()}"


CASES = [
    (1, 64, 1, 4, 1, 0, 0, 0, 1.0),
    (3, 8, 2, 6, 1, 0, 0, 0, 1.0),
    (40, 1032, 8, 16, 4, 0, 0, 0, 0.8),
    (64, 520, 4, 8, 2, 1, 2, 3, 0.7),
    (24, 7168, 8, 32, 8, 2, 2, 2, 1.0),
    (130, 264, 16, 32, 2, 1, 1, 1, 0.5),
    (600, 96, 3, 8, 2, 0, 1, 0, 1.0),
    (520, 72, 5, 4, 2, 0, 0, 4, 0.9),
    (12, 8192, 6, 8, 1, 1, 0, 0, 0.0),
]


@pytest.mark.parametrize("window", [False, True], ids=["compact", "window"])
@pytest.mark.parametrize("repeat", [False, True], ids=["distinct", "repeat"])
@pytest.mark.parametrize("T,H,K,E,P,Z,C,Kc,mask", CASES)
def test_against_the_definition(T, H, K, E, P, Z, C, Kc, mask, repeat, window):
    print(f"[combine_grad] T={T} H={H} K={K} E={E} P={P} Z={Z} C={C} Kc={Kc} mask={mask} {repeat} {window}", flush=True)
    d = _world([T, H, K], T, H, K, E, Z, C, Kc, mask, repeat, bad=True)
    shape = mg.make_shape(T, H, K, E, P, Z, C, Kc)
    A = mg.rank_capacity(shape) if window else 0
    ids, m = G.dev(d["ids"]), G.dev(d["mask"])
    lay = mg.layout(shape, ids, m, rank_stride=A)
    dst = lay.dst_row.cpu().numpy()
    rows = P * A if window else T * K
    y = X.bf16(d["r"], rows, H)
    ref = _definition(d, y, dst, E, Z, C, Kc)
    gy = X.canary(rows, H)
    to = lambda t: t.to(X.DEV) if t.numel() else None  # noqa: E731
    some = C + Kc > 0
    g = mg.combine_grad(shape, to(d["go"]), to(X.poison(y, ref["named"])), ids, G.dev(d["w"]), lay.dst_row, m,
                        to(d["x"]) if some else None, to(d["a1"]), to(d["a2"]), to(d["v"]), gy, rows=rows)
    n = ref["named"]
    # rows: the product rounded to fp32 and to bf16
    X.check(g.grad_expert_out, ref["gy"], np.abs(ref["gy"]) * (X.BF16_HALF + 2 * X.STEP32) + X.TINY, n, "rows")
    # fp32 sums of at most H terms (three roundings a term of a constant expert)
    _near(g.grad_topk_weights, ref["gw"], (H + 8) * X.STEP32 * ref["mw"] + X.TINY * (ref["mw"] > 0), "weights")
    if some:
        err = (2 * K + 4) * X.STEP32 * ref["mx"]
        _near(g.grad_ori_x, ref["gx"], err + X.BF16_HALF * (np.abs(ref["gx"]) + err) + X.TINY * (err > 0), "ori_x")
    if Kc:
        per = (T * K + 8) * X.STEP32
        _near(g.grad_alpha1, ref["ga1"], per * ref["m1"], "alpha1")
        _near(g.grad_alpha2, ref["ga2"], per * ref["m2"], "alpha2")
        _near(g.grad_v, ref["gv"], per * ref["mv"], "v")


def test_twice_the_same():
    d = _world(3, 512, 512, 8, 16, 1, 1, 2, 0.9)
    shape = mg.make_shape(512, 512, 8, 16, 2, 1, 1, 2)
    ids, m = G.dev(d["ids"]), G.dev(d["mask"])
    lay = mg.layout(shape, ids, m)
    y = X.bf16(d["r"], 512 * 8, 512).to(X.DEV)
    a = [mg.combine_grad(shape, d["go"].to(X.DEV), y, ids, G.dev(d["w"]), lay.dst_row, m, d["x"].to(X.DEV),
                         d["a1"].to(X.DEV), d["a2"].to(X.DEV), d["v"].to(X.DEV), torch.zeros_like(y)) for _ in range(2)]
    for p, q in zip(*a):
        assert torch.equal(p, q)


def test_against_differences():
    """Along random directions the gradient equals central differences of the combine's definition in 64
    bits, to within the rounding of its elements (the combine is linear in y, in w and in x)."""
    T, H, K, E, C = 10, 48, 3, 6, 1
    d = _world(5, T, H, K, E, 0, C, 0, 1.0)
    shape = mg.make_shape(T, H, K, E, 1, 0, C, 0)
    ids = G.dev(d["ids"])
    lay = mg.layout(shape, ids)
    dst = lay.dst_row.cpu().numpy()
    y = X.bf16(d["r"], T * K, H)
    g = mg.combine_grad(shape, d["go"].to(X.DEV), y.to(X.DEV), ids, G.dev(d["w"]), lay.dst_row, ori_x=d["x"].to(X.DEV),
                        grad_expert_out=torch.zeros(T * K, H, dtype=torch.bfloat16, device=X.DEV))
    go = X.f64(d["go"])

    def loss(y, w, x):
        out = np.zeros((T, H))
        for t in range(T):
            for j in range(K):
                if dst[t, j] >= 0:
                    out[t] += w[t, j] * y[dst[t, j]]
                elif d["ids"][t, j] == E:
                    out[t] += w[t, j] * x[t]
        return float((out * go).sum())

    at = [X.f64(y), d["w"].astype(np.float64), X.f64(d["x"])]
    for i, (grad, half) in enumerate(zip((g.grad_expert_out, g.grad_topk_weights, g.grad_ori_x),
                                         (X.BF16_HALF, (H + 8) * X.STEP32 * 8, X.BF16_HALF))):
        v = d["r"].standard_normal(at[i].shape)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + v, at[i] - v
        terms = grad.cpu().double().numpy() * v
        assert abs(terms.sum() - (loss(*up) - loss(*down)) / 2) <= 2 * half * np.abs(terms).sum() + 1e-9


@pytest.mark.parametrize("H", [72, 1032, 8192])
def test_only_what_is_asked_for(H):
    """Every subset of the six results is what the whole call gives; the others' buffers are not needed."""
    T, K, E, C, Kc = 38, 4, 8, 2, 3
    d = _world([6, H], T, H, K, E, 1, C, Kc, 0.8)
    shape = mg.make_shape(T, H, K, E, 2, 1, C, Kc)
    ids, m, w = G.dev(d["ids"]), G.dev(d["mask"]), G.dev(d["w"])
    lay = mg.layout(shape, ids, m)
    y = X.bf16(d["r"], T * K, H).to(X.DEV)
    ins = [d[k].to(X.DEV) for k in ("go", "x", "a1", "a2", "v")]
    call = mg.prepare_combine_grad(shape, ins[0], y, ids, w, lay.dst_row, m, *ins[1:], X.canary(T * K, H))
    full = [t.clone() for t in call()]
    at = range(11, 17)  # the results among the arguments
    all_args = list(call._args)
    for subset in range(1, 64):
        for t in call.result:
            t.fill_(-7)
        for i, a in enumerate(at):
            call._args[a] = all_args[a] if subset >> i & 1 else None
        for i, (got, want) in enumerate(zip(call(), full)):
            assert torch.equal(got, want if subset >> i & 1 else torch.full_like(got, -7)), (subset, i)


def test_gradient_of_dispatch_beside_special_experts():
    """The combine with unit weights and without the special experts: each token's rows added up."""
    T, H, K, E, C, Kc = 48, 264, 4, 8, 2, 2
    d = _world(7, T, H, K, E, 1, C, Kc, 0.8)
    ids, m = G.dev(d["ids"]), G.dev(d["mask"])
    lay = mg.layout(mg.make_shape(T, H, K, E, 2, 1, C, Kc), ids, m)
    dst = lay.dst_row.cpu().numpy()
    y = X.bf16(d["r"], T * K, H)
    routed = torch.where(ids < E, ids, -1).contiguous()
    got = mg.combine(mg.make_shape(T, H, K, E, 2), y.to(X.DEV), routed, torch.ones(T, K, device=X.DEV), lay.dst_row, m)
    rows = np.where(dst[:, :, None] >= 0, X.f64(y)[np.maximum(dst, 0)], 0.0)
    ref, err = rows.sum(1), K * X.STEP32 * np.abs(rows).sum(1)
    _near(got, ref, err + X.BF16_HALF * (np.abs(ref) + err), "tokens")


def test_no_tokens():
    shape = mg.make_shape(0, 64, 2, 4, 2, 0, 0, 2)
    e = torch.empty(0, dtype=torch.bfloat16, device=X.DEV)
    i = torch.empty(0, 2, dtype=torch.int32, device=X.DEV)
    a = torch.ones(2, 64, dtype=torch.bfloat16, device=X.DEV)
    g = mg.combine_grad(shape, e, e, i, torch.empty(0, 2, device=X.DEV), i, None, e, a, a, a)
    for t in (g.grad_alpha1, g.grad_alpha2, g.grad_v):
        assert torch.all(t == 0)
