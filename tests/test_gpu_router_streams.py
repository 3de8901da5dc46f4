"""The router's and the gate's calls on another stream, prepared, and captured into graphs that are replayed."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X

pytestmark = pytest.mark.gpu

T, E, K, S, N = 512, 64, 8, 4, 264


def _world():
    r = np.random.default_rng(33)
    shape, bal = mg.make_route_shape(T, E, K, mg.SCORE_SIGMOID, groups=8, topk_groups=3, group_score=mg.GROUP_TOP2), \
        mg.make_balance(S, 0.5, 0.1)
    f = lambda *s: torch.from_numpy(r.standard_normal(s, dtype=np.float32)).to(X.DEV)  # noqa: E731
    logits, bias = f(T, E), 0.1 * f(E)
    ids = mg.route(shape, logits, bias).topk_idx
    h0, d, w = f(T, 2 * N).bfloat16(), f(T, N).bfloat16(), f(T)
    kept = mg.swiglu(h0, w, checkpoint=True)
    return dict(shape=shape, bal=bal, logits=logits, bias=bias, ids=ids, gw=f(T, K), gl=f(2), h0=h0, d=d, w=w,
                codes=kept.codes, scales=kept.scales, loss=mg.balance_loss(shape, bal, logits, ids))


CALLS = {
    "route": (("logits", "bias"), lambda d, t, s: mg.route(d["shape"], t["logits"], t["bias"], stream=s)),
    "balance_loss": (("logits", "ids"), lambda d, t, s: mg.balance_loss(d["shape"], d["bal"], t["logits"], t["ids"], stream=s)),
    "route_grad": (("logits", "ids", "gw", "gl"),
                   lambda d, t, s: mg.route_grad(d["shape"], t["logits"], t["ids"], t["gw"], d["bal"], d["loss"], t["gl"], stream=s)),
    "swiglu": (("h0", "w"), lambda d, t, s: mg.swiglu(t["h0"], t["w"], checkpoint=True, stream=s)),
    "swiglu_grad": (("d", "codes", "scales", "w"),
                    lambda d, t, s: mg.swiglu_grad(t["d"], codes=t["codes"], scales=t["scales"], row_weights=t["w"], stream=s)),
}


def _tensors(out):
    return [out] if isinstance(out, torch.Tensor) else [t for o in out for t in _tensors(o)] if isinstance(out, tuple) else []


@pytest.mark.parametrize("name", list(CALLS))
def test_arguments_and_results_dropped_at_once(name):
    d = _world()
    keys, call = CALLS[name]
    want = [t.clone() for t in _tensors(call(d, d, None))]
    side, spin = torch.cuda.Stream(), 20_000_000  # some 10 ms
    for _ in range(3):
        t = {k: d[k].clone() for k in keys}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(spin)
        out = _tensors(call(d, t, side))
        spare = _tensors(call(d, t, side))
        taken = {o.data_ptr() for o in spare} | {v.data_ptr() for v in t.values()}
        sizes = [(o.shape, o.dtype) for o in spare] + [(v.shape, v.dtype) for v in t.values()]
        del spare, t
        fresh = [torch.ones(s, dtype=dt, device=X.DEV) for s, dt in sizes for _ in range(2)]
        if not side.query():  # still under way: its memory must not be handed out
            assert not taken & {f.data_ptr() for f in fresh}
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(out, want))
        assert all(bool((f == 1).all()) for f in fresh)


@pytest.mark.parametrize("joined", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_captured_and_replayed(name, joined):
    """Two calls of a kind in each of two graphs, on the capture's stream or on one that joins it; replayed in turn with new
    inputs, eager calls and synchronizations between."""
    d = _world()
    keys, call = CALLS[name]
    call(d, d, None)
    torch.cuda.synchronize()
    t = {k: d[k].clone() for k in keys}
    graphs = []
    for _ in range(2):
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if joined:
                side.wait_stream(torch.cuda.current_stream())
            call(d, t, side if joined else None)
            got = _tensors(call(d, t, side if joined else None))
            if joined:
                torch.cuda.current_stream().wait_stream(side)
        graphs.append((graph, got))
    for k in range(4):
        for key, v in t.items():
            if v.dtype.is_floating_point:
                v.copy_(d[key] * (1 + 0.25 * k))
        want = [w.clone() for w in _tensors(call(d, t, None))]
        torch.cuda.synchronize()
        graph, got = graphs[k % 2]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want)), k
        torch.ones(1 << 20, device=X.DEV).sum()


def test_two_streams_at_once():
    """Two batches' losses on two streams, each with a workspace that its call makes."""
    d = _world()
    big = mg.make_route_shape(1 << 17, E, K)
    logits = [torch.randn(1 << 17, E, device=X.DEV) for _ in range(2)]
    bal = mg.make_balance(8, 0.5, 0.1)
    ids = [mg.route(big, l).topk_idx for l in logits]
    want = [mg.balance_loss(big, bal, l, i) for l, i in zip(logits, ids)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [mg.balance_loss(big, bal, logits[k], ids[k], stream=streams[k]) for k in range(2)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))
    del d


def test_prepared_calls():
    """A prepared call reads what its tensors hold when it is issued."""
    d = _world()
    r = mg.prepare_route(d["shape"], d["logits"], d["bias"])
    b = mg.prepare_balance_loss(d["shape"], d["bal"], d["logits"], r.result.topk_idx)
    g = mg.prepare_route_grad(d["shape"], d["logits"], r.result.topk_idx, d["gw"], d["bal"], b.result, d["gl"])
    for k in range(3):
        d["logits"].mul_(1.5).add_(k)
        for call in (r, b, g):
            call()
        again = mg.route(d["shape"], d["logits"], d["bias"])
        loss = mg.balance_loss(d["shape"], d["bal"], d["logits"], again.topk_idx)
        assert torch.equal(again.topk_idx, r.result.topk_idx) and torch.equal(again.topk_weights, r.result.topk_weights)
        assert all(torch.equal(x, y) for x, y in zip(loss, b.result))
        assert torch.equal(mg.route_grad(d["shape"], d["logits"], again.topk_idx, d["gw"], d["bal"], loss, d["gl"]), g.result)
