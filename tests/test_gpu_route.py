"""The router's choice against its definition in 64 bits: ids exactly, weights within what fp32 arithmetic allows."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X
from tests import _router as R

pytestmark = pytest.mark.gpu

INF, NAN = np.inf, np.nan


def logits(r, T, E, bf16=False, grid=None):
    l = r.standard_normal((T, E)) * r.uniform(0.3, 3.0, (T, 1)) + r.standard_normal(E)
    if grid:
        l = np.round(l / grid) * grid  # ties
    t = torch.from_numpy(l.astype(np.float32))
    return t.bfloat16() if bf16 else t


def check(l, K, score, renorm=True, scale=1.0, bias=None, mask=None, groups=1, keep=1, two=False, what=""):
    T, E = l.shape
    shape = mg.make_route_shape(T, E, K, score, renorm, scale, groups, keep, mg.GROUP_TOP2 if two else mg.GROUP_MAX)
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(X.DEV)  # noqa: E731
    # a little more room than the results need: what lies behind them stays
    ids = torch.full((T * K + 5,), 77, dtype=torch.int32, device=X.DEV)
    w = torch.full((T * K + 5,), 77.0, device=X.DEV)
    mg.route(shape, l.to(X.DEV), bias=dev(bias), x_active_mask=dev(mask), topk_idx=ids, topk_weights=w)
    ids, w = ids.cpu().numpy(), w.cpu().double().numpy()
    assert (ids[T * K:] == 77).all() and (w[T * K:] == 77).all()
    ids, w = ids[:T * K].reshape(T, K), w[:T * K].reshape(T, K)
    l64 = R.usable(l.double().numpy())
    if mask is not None:
        l64 = np.where(np.asarray(mask)[:, None] > 0, l64, -np.inf)
    want = R.choose(l64, K, score, bias, mask, groups, keep, R.TOP2 if two else R.MAX)
    bad = np.argwhere((ids != want).any(1)).ravel()
    assert len(bad) == 0, (what, bad[:5], ids[bad[0]], want[bad[0]])
    ref, tol = R.weights(l64, want, score, renorm, scale)
    off = np.abs(w - ref) - tol
    assert (off <= 0).all(), (what, np.unravel_index(off.argmax(), off.shape), w.ravel()[off.argmax()], ref.ravel()[off.argmax()])
    return ids


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 2, 2), (3, 7, 3), (130, 33, 4), (65, 64, 16), (2, 65, 1), (9, 127, 8),
                                   (5, 128, 6), (77, 134, 6), (33, 200, 5), (64, 256, 8), (6, 257, 16), (4, 511, 2),
                                   (4, 512, 8), (3, 1000, 9), (2, 1024, 8), (3, 2047, 16), (2, 2048, 8)])
def test_sizes(T, E, K, bf16, score):
    print(f"[route] {T} {E} {K} {bf16} {score}", flush=True)
    r = np.random.default_rng([T, E, K])
    check(logits(r, T, E, bf16), K, score, renorm=False, scale=2.5)
    bias = (0.3 * r.standard_normal(E)).astype(np.float32)
    check(logits(r, T, E, bf16), K, score, renorm=True, bias=bias, mask=(r.random(T) < 0.8).astype(np.uint8))


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,G,keep,K", [(8, 2, 1, 4), (64, 8, 3, 8), (256, 8, 4, 8), (256, 8, 8, 8), (96, 3, 2, 7),
                                        (134, 2, 1, 6), (64, 64, 16, 16), (60, 5, 2, 3), (256, 16, 2, 16), (512, 8, 1, 4),
                                        (1024, 32, 5, 8), (2048, 64, 9, 16), (130, 13, 4, 8), (128, 64, 8, 16), (320, 5, 2, 8)])
def test_groups(E, G, keep, K, biased, two, score):
    print(f"[groups] {E} {G} {keep} {K} {biased} {two} {score}", flush=True)
    r = np.random.default_rng([E, G, keep])
    T = 21
    bias = (0.3 * r.standard_normal(E)).astype(np.float32) if biased else None
    check(logits(r, T, E), K, score, groups=G, keep=keep, two=two, bias=bias)
    l = logits(r, T, E, bf16=True, grid=0.5)  # ties within and between groups
    check(l, K, score, groups=G, keep=keep, two=two)
    l = logits(r, T, E)
    l[torch.from_numpy(r.random((T, E)) < 0.9)] = -INF  # groups with one id left, or none
    check(l, K, score, groups=G, keep=keep, two=two, bias=bias)


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
def test_ties_go_to_the_lowest_id(score):
    for E in (5, 64, 100, 256, 600, 2048):
        K = min(E, 16)
        l = torch.zeros(4, E)
        l[1] = -3.5
        l[2, E // 2:] = 1.0
        l[3] = torch.arange(E) % 2
        ids = check(l, K, score)
        assert (ids[0] == np.arange(K)).all() and (ids[1] == np.arange(K)).all()
        check(l, K, score, bias=np.zeros(E, np.float32))
        check(l, K, score, bias=np.where(np.arange(E) % 3 == 0, 0.5, 0.0).astype(np.float32))
        check(-l * 0.0, K, score)  # zeros of both signs are the same


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_logits_that_are_no_numbers(score, renorm, bf16):
    low = float(torch.finfo(torch.bfloat16).min)
    r = np.random.default_rng(5)
    E, K = 70, 4
    l = logits(r, 12, E, bf16)
    l[0] = -INF                     # nothing left
    l[1] = NAN
    l[2, 3:] = -INF                 # fewer than K left
    l[3, 1:] = NAN
    l[4, 2:] = low                  # masked by the lowest value: finite, chosen last
    l[5] = low
    l[6, 17] = INF                  # counts as the largest finite one
    l[7, ::2] = -INF
    l[8, 5], l[8, 6] = INF, INF
    l[9] = -1000.0                  # scores that vanish in fp32, their ratios do not
    l[9, 11] = -1003.0
    l[10] = 300.0
    mask = np.ones(12, np.uint8)
    mask[11] = 0
    l[11] = NAN                     # a masked token's logits are not looked at
    ids = check(l, K, score, renorm, mask=mask)
    assert (ids[[0, 1, 11]] == -1).all() and (ids[2] == -1).sum() == 1 and (ids[3] == -1).sum() == 3
    bias = np.zeros(E, np.float32)
    bias[:8] = [NAN, -INF, INF, 5.0, -5.0, 1e30, -1e30, 0.0]
    l[9] = logits(r, 1, E, bf16)
    l[10] = logits(r, 1, E, bf16)
    ids = check(l, K, score, renorm, mask=mask, bias=bias)
    assert not np.isin(ids, [0, 1]).any() and ids[7, 0] != 2 and ids[9, 0] == 2 and ids[9, 1] == 5


@pytest.mark.parametrize("T,E,K,groups,keep", [(8200, 100, 6, 1, 1), (8192, 128, 8, 8, 3), (9000, 65, 16, 5, 2)])
def test_many_tokens(T, E, K, groups, keep):
    r = np.random.default_rng([T, E])
    mask = (r.random(T) < 0.9).astype(np.uint8)
    check(logits(r, T, E, bf16=True), K, mg.SCORE_SIGMOID, groups=groups, keep=keep, two=True, mask=mask)
    check(logits(r, T, E), K, mg.SCORE_SOFTMAX, groups=groups, keep=keep, bias=(0.1 * r.standard_normal(E)).astype(np.float32))


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,K", [(64, 8), (128, 16), (256, 8), (512, 8), (1024, 16), (2048, 16)])
def test_rows_with_many_near_the_best(E, K, biased):
    """The best ids lie together in few lanes, or many ids share the best values: from a handful of candidates to all ids."""
    r = np.random.default_rng([E, K, biased])
    bias = (2.0 ** -26 * r.integers(0, 4, E)).astype(np.float32) if biased else None
    rows = []
    for width in (1, 3, K - 1, K, K + 1, 17, 33, 60, 64, 65, 130, 260, E):
        for first in (0, E - min(width, E), r.integers(0, E)):
            l = r.standard_normal(E) - 8
            at = (first + np.arange(min(width, E))) % E
            rows.append(l.copy())
            rows[-1][at] = 3.0                                            # ties
            rows.append(l.copy())
            rows[-1][at] = 3.0 + 0.01 * r.permutation(len(at))            # in any order
            rows.append(l.copy())
            rows[-1][at] = 3.0 + 2.0 ** -22 * r.permutation(len(at))      # neighbours in fp32
    l = torch.from_numpy(np.array(rows, np.float32))
    for score in (mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID):
        check(l, K, score, bias=bias)
        check(l, K, score, bias=bias, groups=8, keep=5, two=True)


@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
@pytest.mark.parametrize("E,G", [(64, 8), (256, 8), (96, 3), (512, 4)])
def test_groups_next_to_one_another(E, G, score):
    """Group scores that differ by some 1e-9, which 32 bits do not hold, tie, or are set apart by a bias of any size."""
    r = np.random.default_rng([E, G])
    T, per, keep, K = 64, E // G, max(1, G // 2), 4
    l = r.standard_normal((T, E)) - 3
    for t in range(T):
        for g in range(G):
            at = g * per + r.permutation(per)[:2]
            l[t, at] = [1.5, 1.0 + 2.0 ** -23 * r.integers(0, 3)]
    l = torch.from_numpy(l.astype(np.float32))
    check(l, K, score, groups=G, keep=keep, two=True)
    check(l, K, score, groups=G, keep=keep, two=True, bias=(2.0 ** -28 * r.integers(0, 8, E)).astype(np.float32))
    check(l, K, score, groups=G, keep=keep, two=False, bias=(2.0 ** -28 * r.integers(0, 8, E)).astype(np.float32))
    bias = (0.1 * r.standard_normal(E)).astype(np.float32)
    bias[[0, 5, per, E - 1]] = [3.0e38, -3.0e38, INF, -1e20]
    for two in (False, True):
        check(l, K, score, groups=G, keep=keep, two=two, bias=bias)
    bias[:] = -3.4e38
    check(l, K, score, groups=G, keep=keep, two=False, bias=bias)


def test_near_scores_are_told_apart():
    """Sigmoids of neighbouring fp32 logits, and sums with a bias that differ by less than fp32 holds."""
    r = np.random.default_rng(8)
    T, E = 40, 64
    base = r.uniform(-2, 2, (T, 1)).astype(np.float32)
    l = base + (r.permuted(np.tile(np.arange(E), (T, 1)), axis=1) * 2.0 ** -22).astype(np.float32)
    check(torch.from_numpy(l), 8, mg.SCORE_SIGMOID, bias=np.full(E, 7.0, np.float32))
    check(torch.from_numpy(l), 8, mg.SCORE_SOFTMAX, bias=np.full(E, 3.0, np.float32))
    bias = (r.permutation(E) * 2.0 ** -24).astype(np.float32)
    check(torch.from_numpy(l), 8, mg.SCORE_SIGMOID, bias=bias)


def test_no_tokens():
    s = mg.make_route_shape(0, 8, 2)
    out = mg.route(s, torch.empty(0, 8, device=X.DEV))
    assert out.topk_idx.shape == (0, 2) and out.topk_weights.shape == (0, 2)


def test_beyond_32_bits_of_offset():
    """Rows whose bytes begin past 2^32: the last tokens of 2.2e9 logits."""
    T, E, K = (1 << 21) + 37, 1024, 8
    l = torch.zeros(T, E, dtype=torch.bfloat16, device=X.DEV)
    r = np.random.default_rng(2)
    tail = logits(r, 64, E, bf16=True)
    l[-64:] = tail.to(X.DEV)
    ids, w = mg.route(mg.make_route_shape(T, E, K), l)
    want = R.choose(R.usable(tail.double().numpy()), K, R.SOFTMAX)
    assert np.array_equal(ids[-64:].cpu().numpy(), want)
    assert bool((ids[:-64] == torch.arange(K, device=X.DEV)).all())
    assert bool(((w[:-64] - 1 / K).abs() <= 4 * R.STEP32).all())
    shape = mg.make_route_shape(T, E, K)
    g = mg.route_grad(shape, l, ids, grad_topk_weights=torch.ones(T, K, device=X.DEV) * torch.arange(K, device=X.DEV))
    d, mag = R.grad(R.usable(tail.double().numpy()), want, R.SOFTMAX, True, 1.0, np.tile(np.arange(K), (64, 1)))
    off = np.abs(g[-64:].cpu().double().numpy() - d) - R.grad_tol(mag, d, tail.double().numpy(), True)
    assert (off <= 0).all()
