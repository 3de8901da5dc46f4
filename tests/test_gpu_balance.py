"""The balance losses and the gradient of the logits, against their definitions in 64 bits and against differences."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X
from tests import _router as R
from tests.test_gpu_route import logits

pytestmark = pytest.mark.gpu

INF, NAN = np.inf, np.nan


def dev(a, dtype=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a if dtype is None else a.astype(dtype))).to(X.DEV)


def run(l, ids, score, renorm=True, scale=1.0, gw=None, S=1, bc=0.7, zc=0.0, gl=None, mask=None, losses=True):
    """Both calls and both references, compared."""
    T, E = l.shape
    K = ids.shape[1]
    shape = mg.make_route_shape(T, E, K, score, renorm, scale)
    l64 = R.usable(l.double().numpy())
    if mask is not None:
        l64 = np.where(np.asarray(mask)[:, None] > 0, l64, -np.inf)
    bal = b = None
    ref = {}
    if losses:
        bal = mg.make_balance(S, bc, zc)
        b = mg.balance_loss(shape, bal, l.to(X.DEV), dev(ids, np.int32), dev(mask))
        ref = R.losses(l64, ids, score, S, np.float32(bc).astype(float), np.float32(zc).astype(float), mask)
        assert np.array_equal(b.counts.cpu().numpy(), ref["counts"])
        assert np.array_equal(b.segment_tokens.cpu().numpy(), ref["tokens"])
        spread = np.abs(np.where(l64 > -np.inf, l64, 0.0)).max() if T else 0.0
        # a probability is good to (4 |l| + E / 8 + 32) steps; 64 of them at most are added in fp32
        rel = (4 * min(spread, 200.0) + E / 8 + 32 + 64) * R.STEP32
        sums = b.prob_sums.cpu().double().numpy()
        assert (np.abs(sums - ref["sums"]) <= rel * ref["sums"] + T * R.TINY + 2.0 ** -126).all()
        got = b.losses.cpu().double().numpy()
        assert (np.abs(got - ref["losses"]) <= rel * np.abs(ref["losses"]) + R.TINY).all(), (got, ref["losses"])
    g = mg.route_grad(shape, l.to(X.DEV), dev(ids, np.int32), dev(gw, np.float32), bal, b, dev(gl, np.float32), dev(mask))
    d, mag = R.grad(l64, ids, score, renorm, np.float32(scale).astype(float),
                    None if gw is None else gw.astype(np.float32).astype(float), S, np.float32(bc).astype(float),
                    np.float32(zc).astype(float), (1.0, 1.0) if gl is None else gl.astype(np.float32).astype(float),
                    ref.get("counts"), ref.get("tokens"), mask)
    got = g.cpu().double().numpy()
    off = np.abs(got - d) - R.grad_tol(mag, d, l64, l.dtype == torch.bfloat16)
    i = np.unravel_index(np.argmax(np.where(np.isnan(off), np.inf, off)), off.shape) if off.size else None
    assert (off <= 0).all(), (i, got[i], d[i], mag[i])
    return b, g


def some_ids(r, l, K, dropped=0.0):
    ids = np.argsort(-l.double().numpy() + 0.3 * r.standard_normal(l.shape), axis=1)[:, :K].astype(np.int32)
    ids[r.random(ids.shape) < dropped] = -1
    return ids


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,K,S", [(1, 1, 1, 1), (1, 8, 2, 1), (3, 7, 3, 3), (130, 33, 4, 2), (64, 64, 16, 8), (6, 65, 1, 1),
                                     (96, 128, 6, 4), (77, 134, 6, 7), (512, 256, 8, 2), (12, 257, 5, 3), (36, 512, 8, 1),
                                     (20, 1000, 8, 4), (24, 2048, 16, 2), (5000, 40, 2, 1), (8192, 100, 3, 4), (8300, 128, 8, 1),
                                     (40, 1022, 3, 1), (700, 1024, 8, 2), (300, 2047, 8, 1)])
def test_against_the_definitions(T, E, K, S, bf16, renorm, score):
    print(f"[balance] {T} {E} {K} {S} {bf16} {renorm} {score}", flush=True)
    r = np.random.default_rng([T, E, K, S])
    l = logits(r, T, E, bf16)
    ids = some_ids(r, l, K, 0.1)
    gw = r.standard_normal((T, K))
    run(l, ids, score, renorm, 2.5, gw, S, 0.7, 0.3, np.array([1.5, -0.5]))
    run(l, ids, score, renorm, 1.0, None, S, 0.7, 0.0)
    run(l, ids, score, renorm, 1.0, gw, losses=False)
    run(l, ids, score, renorm, 1.0, gw, S, 0.7, 0.3, mask=(r.random(T) < 0.6).astype(np.uint8))


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_against_differences(score, renorm):
    """The fp32 gradient against central differences of the definition in 64 bits: (f(l + h) - f(l - h)) / 2 h with h = 1e-4 is
    off by h^2 / 6 of the third derivative (at most some 30 of the terms' size) and 1e-16 / h of the value."""
    r = np.random.default_rng(9)
    T, E, K, S = 12, 10, 3, 3
    l = logits(r, T, E)
    ids = some_ids(r, l, K, 0.1)
    gw, gl = r.standard_normal((T, K)), np.array([2.0, 0.5])
    mask = np.ones(T, np.uint8)
    mask[[2, 7]] = 0
    _, g = run(l, ids, score, renorm, 1.5, gw, S, 0.7, 0.3, gl, mask)
    gw32 = gw.astype(np.float32).astype(float)

    def f(l64):
        w, _ = R.weights(l64, ids, score, renorm, 1.5)
        v = R.losses(l64, ids, score, S, float(np.float32(0.7)), float(np.float32(0.3)), mask)["losses"]
        return (w * gw32 * mask[:, None]).sum() + (v * gl).sum()

    base, h = l.double().numpy(), 1e-4
    want = np.zeros((T, E))
    for t in range(T):
        for e in range(E):
            up, down = base.copy(), base.copy()
            up[t, e] += h
            down[t, e] -= h
            want[t, e] = (f(up) - f(down)) / (2 * h)
    assert np.abs(g.cpu().double().numpy() - want).max() <= 1e-6


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_logits_that_are_no_numbers(score, renorm):
    r = np.random.default_rng(6)
    T, E, K = 12, 70, 4
    l = logits(r, T, E)
    ids = some_ids(r, l, K)
    l[0] = -INF
    l[1] = NAN
    l[2, 5:] = -INF
    l[3, 1:] = NAN                 # chosen ids without a logit
    l[4, 2:] = float(torch.finfo(torch.float32).min)
    l[5] = -1000.0                 # all scores vanish in fp32
    l[5, 7] = -1002.0
    l[7, ::2] = -INF
    l[11] = NAN
    gw = r.standard_normal((T, K))
    mask = np.ones(T, np.uint8)
    mask[[8, 11]] = 0
    gw[8] = NAN                    # of a masked token: not looked at
    ids[9, 1] = -1
    gw[9, 1] = NAN                 # of a slot without an id
    b, g = run(l, ids, score, renorm, 1.0, np.nan_to_num(gw), 2, 0.7, 0.0, mask=mask)
    shape = mg.make_route_shape(T, E, K, score, renorm)
    again = mg.route_grad(shape, l.to(X.DEV), dev(ids), dev(gw, np.float32), mg.make_balance(2, 0.7, 0.0), b, None, dev(mask))
    assert torch.equal(again, g)
    for t in (0, 1, 8, 11):
        assert bool((g[t] == 0).all())
    assert bool((g.cpu()[~(l > -INF)] == 0).all())


def test_ids_that_are_not_counted_and_ids_that_stand_twice():
    r = np.random.default_rng(7)
    T, E, K = 30, 20, 4
    l = logits(r, T, E)
    ids = some_ids(r, l, K)
    ids[:, 1] = ids[:, 0]
    ids[::3, 2] = [E, E + 7, 2 ** 31 - 1, -2, -2 ** 31, -1, E, E, E, E]
    for score in (mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID):
        for renorm in (False, True):
            run(l, ids, score, renorm, 1.0, r.standard_normal((T, K)), 3, 0.7, 0.1)


def test_segments_without_a_live_token_and_no_tokens():
    r = np.random.default_rng(3)
    l = logits(r, 12, 16)
    mask = np.ones(12, np.uint8)
    mask[4:8] = 0
    ids = some_ids(r, l, 2)
    b, _ = run(l, ids, mg.SCORE_SOFTMAX, gw=r.standard_normal((12, 2)), S=3, zc=0.2, mask=mask)
    assert b.segment_tokens.tolist() == [4, 0, 4] and bool((b.prob_sums[1] == 0).all())
    b, g = run(l, ids, mg.SCORE_SIGMOID, gw=r.standard_normal((12, 2)), S=3, zc=0.2, mask=np.zeros(12, np.uint8))
    assert b.losses.tolist() == [0, 0] and bool((g == 0).all())
    for E in (16, 18, 130, 1026):
        s = mg.make_route_shape(0, E, 2)
        bal = mg.make_balance(2, 1.0, 1.0)
        e = torch.empty(0, E, device=X.DEV)
        i = torch.empty(0, 2, dtype=torch.int32, device=X.DEV)
        b = mg.balance_loss(s, bal, e, i)
        assert b.losses.tolist() == [0, 0] and bool((b.counts == 0).all()) and b.segment_tokens.tolist() == [0, 0]
        assert bool((b.prob_sums == 0).all())
        assert mg.route_grad(s, e, i, torch.empty(0, 2, device=X.DEV), bal, b).shape == (0, E)


def test_many_segments():
    r = np.random.default_rng(4)
    T, E, K = 4096, 24, 2
    l = logits(r, T, E)
    run(l, some_ids(r, l, K), mg.SCORE_SIGMOID, gw=r.standard_normal((T, K)), S=4096, zc=0.2, mask=(r.random(T) < 0.5).astype(np.uint8))


def test_gradients_of_receive_rows():
    """grad_topk_weights of rows with the layout's map is the same as of slots; slots without a row have none."""
    r = np.random.default_rng(12)
    T, E, K = 50, 16, 4
    l = logits(r, T, E)
    ids = some_ids(r, l, K, 0.1)
    shape = mg.make_route_shape(T, E, K)
    lay = mg.layout(mg.make_shape(T, 64, K, E, 2), dev(ids))
    rows = torch.randn(T * K, device=X.DEV)
    rows[int(lay.expert_offsets[-1]):] = NAN
    slots = torch.where(lay.dst_row >= 0, rows[lay.dst_row.clamp(min=0).long()], 0.0)
    a = mg.route_grad(shape, l.to(X.DEV), dev(ids), slots)
    b = mg.route_grad(shape, l.to(X.DEV), dev(ids), rows, dst_row=lay.dst_row)
    assert torch.equal(a, b) and bool(a.isfinite().all())


def test_results_do_not_change_and_a_workspace_is_what_it_is_given():
    r = np.random.default_rng(14)
    T, E, K, S = 6144, 64, 8, 4
    l, shape, bal = logits(r, T, E).to(X.DEV), mg.make_route_shape(T, E, K), mg.make_balance(S, 1.0, 0.1)
    ids = mg.route(shape, l).topk_idx
    ws = torch.full((mg.balance_workspace_size(shape, bal) + 64,), 255, dtype=torch.uint8, device=X.DEV)
    first = mg.balance_loss(shape, bal, l, ids)
    for _ in range(4):
        b = mg.balance_loss(shape, bal, l, ids, workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(first, b))
    assert bool((ws[-64:] == 255).all())


def test_a_million_tokens():
    """More tokens than fp32 adds one by one without loss."""
    T, E, K = 1 << 20, 8, 2
    l = torch.randn(T, E, device=X.DEV, generator=torch.Generator(device=X.DEV).manual_seed(3))
    shape, bal = mg.make_route_shape(T, E, K), mg.make_balance(1, 1.0, 1.0)
    ids = mg.route(shape, l).topk_idx
    b = mg.balance_loss(shape, bal, l, ids)
    p = torch.softmax(l.double(), 1)
    counts = torch.bincount(ids.flatten().long(), minlength=E)
    assert torch.equal(b.counts[0].long(), counts) and int(b.segment_tokens) == T
    rel = (4 * float(l.abs().max()) + 1 + 32 + 64) * R.STEP32
    assert bool(((b.prob_sums[0].double() - p.sum(0)).abs() <= rel * p.sum(0)).all())
    want = torch.stack((E / (K * T * T) * (counts * p.sum(0)).sum(), torch.logsumexp(l.double(), 1).square().mean()))
    assert bool(((b.losses.double() - want).abs() <= rel * want).all())


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
@pytest.mark.parametrize("T,E", [(7, 33), (5, 64), (9, 134), (3, 257), (5, 1000), (2, 2046)])
def test_rows_behind_the_last_and_tokens_that_are_not_live(T, E, score):
    """A larger buffer keeps what lies behind; losses whose gradient is not finite leave rows of masked tokens zeros."""
    r = np.random.default_rng([T, E])
    for bf16 in (False, True):
        l = logits(r, T, E, bf16)
        ids = some_ids(r, l, 2)
        mask = np.ones(T, np.uint8)
        mask[0] = 0
        shape, bal = mg.make_route_shape(T, E, 2, score), mg.make_balance(1, 1.0, 1.0)
        b = mg.balance_loss(shape, bal, l.to(X.DEV), dev(ids), dev(mask))
        for bad in (INF, NAN):
            out = torch.full((T * E + 40,), 7.0, dtype=l.dtype, device=X.DEV)
            mg.route_grad(shape, l.to(X.DEV), dev(ids), torch.ones(T, 2, device=X.DEV), bal, b,
                          torch.tensor([bad, bad], device=X.DEV), dev(mask), out=out)
            assert bool((out[T * E:] == 7).all()) and bool((out[:E] == 0).all())
            assert not bool(out[E:T * E].isfinite().all())
