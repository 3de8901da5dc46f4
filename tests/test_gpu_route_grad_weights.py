"""The gradient through renormalized weights, held to what its own result allows: where one slot of a token has a score its
weight is a constant, and nothing goes back."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X
from tests import _router as R
from tests import _router_near as N

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a if dtype is None else a.astype(dtype))).to(X.DEV)


def world(r, T, E, bf16):
    l = torch.from_numpy((r.standard_normal((T, E)) * r.uniform(0.3, 3.0, (T, 1))).astype(np.float32))
    return (l.bfloat16() if bf16 else l).float().numpy(), torch.bfloat16 if bf16 else torch.float32


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("how", ["one", "dropped", "without a logit"])
@pytest.mark.parametrize("T,E", [(700, 64), (300, 33), (200, 256), (60, 2048)])
def test_one_scored_slot_gives_nothing_back(T, E, how, bf16, score):
    print(f"[lone] {T} {E} {how} {bf16} {score}", flush=True)
    r = np.random.default_rng([T, E])
    l, dtype = world(r, T, E, bf16)
    l, ids = N.lone_slots(r, l, 5, how)
    K = ids.shape[1]
    lt, it = dev(l).to(dtype), dev(ids)
    shape = mg.make_route_shape(T, E, K, score, True, 2.5)
    bal = mg.make_balance(1, 1e-2, 1e-3)
    b = mg.balance_loss(shape, bal, lt, it)
    gw = torch.randn(T, K, device=X.DEV)
    assert torch.equal(mg.route_grad(shape, lt, it, gw, bal, b), mg.route_grad(shape, lt, it, None, bal, b))
    assert bool((mg.route_grad(shape, lt, it, gw) == 0).all())


def test_one_chosen_id_of_a_mean_over_tokens():
    """4096 tokens of 64 ids: the balance loss's part is of the order of 1e-2 / T and is what is left."""
    r = np.random.default_rng(15)
    T, E = 4096, 64
    l, _ = world(r, T, E, False)
    ids = l.argmax(1)[:, None].astype(np.int32)
    for score in (mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID):
        shape, bal = mg.make_route_shape(T, E, 1, score), mg.make_balance(1, 1e-2, 0.0)
        b = mg.balance_loss(shape, bal, dev(l), dev(ids))
        gw = (r.standard_normal((T, 1)) / T).astype(np.float32)
        g = mg.route_grad(shape, dev(l), dev(ids), dev(gw), bal, b).cpu().double().numpy()
        l64 = l.astype(np.float64)
        ref = R.losses(l64, ids, score, 1, float(np.float32(1e-2)), 0.0)
        d, mag = N.grad(l64, ids, score, 1.0, gw.astype(np.float64), bc=float(np.float32(1e-2)), counts=ref["counts"], tokens=ref["tokens"])
        assert (np.abs(g - d) <= R.grad_tol(mag, d, l64, False)).all()
        # eight roundings of a probability and of its factor, each half a step, as if all of one sign
        assert np.linalg.norm(g - d) <= 8 * 2.0 ** -24 * np.linalg.norm(mag)


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,K", [(130, 33, 2), (64, 64, 16), (77, 134, 6), (64, 256, 8), (36, 512, 4), (20, 1000, 8), (9, 2048, 3)])
@pytest.mark.parametrize("lift", [0.0, 6.0, 14.0])
def test_slots_of_any_weight(T, E, K, bf16, score, lift):
    """One slot's score above the others': from even ones to one that carries the sum, the rest a millionth."""
    r = np.random.default_rng([T, E, K])
    l, dtype = world(r, T, E, bf16)
    l -= lift if score == mg.SCORE_SIGMOID else 0.0
    ids = np.argsort(r.random((T, E)), axis=1)[:, :K].astype(np.int32)
    l[np.arange(T), ids[np.arange(T), r.integers(0, K, T)]] += lift
    ids[r.random(ids.shape) < 0.1] = -1
    lt = dev(l).to(dtype)
    l64 = lt.cpu().double().numpy()
    gw = r.standard_normal((T, K)).astype(np.float32)
    gw[::3] += 1000.0  # what all slots have in common does not matter
    shape = mg.make_route_shape(T, E, K, score, True, 1.5)
    g = mg.route_grad(shape, lt, dev(ids), dev(gw)).cpu().double().numpy()
    d, mag = N.grad(l64, ids, score, 1.5, gw.astype(np.float64))
    off = np.abs(g - d) - R.grad_tol(mag, d, l64, bf16)
    assert (off <= 0).all(), np.unravel_index(off.argmax(), off.shape)


@pytest.mark.parametrize("bad", [np.inf, np.nan])
def test_ids_without_a_logit_stay_zeros(bad):
    """Also where a gradient of the token's weights is not finite."""
    T, E, K = 8, 40, 4
    r = np.random.default_rng(4)
    l, _ = world(r, T, E, False)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :K].astype(np.int32)
    l[np.arange(T), ids[:, 1]] = -np.inf
    gw = r.standard_normal((T, K)).astype(np.float32)
    gw[::2, 0] = bad
    for score in (mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID):
        g = mg.route_grad(mg.make_route_shape(T, E, K, score), dev(l), dev(ids), dev(gw)).cpu().numpy()
        assert (g[np.arange(T), ids[:, 1]] == 0).all()
        assert np.isfinite(g[1::2]).all() and not np.isfinite(g[::2]).all(1).any()
