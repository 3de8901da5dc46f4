"""The expert stage as it is used: between dispatch and combine, forward and back, on other streams and
in captured graphs."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X
from tests import _gpu as G

pytestmark = pytest.mark.gpu

T, H, I, K, E, P = 96, 256, 128, 4, 16, 4


def _world(seed):
    r = np.random.default_rng(seed)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :K].astype(np.int32)
    ids[r.random((T, K)) < 0.05] = -1
    w = r.random((T, K)).astype(np.float32)
    return dict(ids=G.dev(ids), w=G.dev(w / w.sum(1, keepdims=True)), x=X.bf16(r, T, H).to(X.DEV),
                w1=X.bf16(r, E, 2 * I, H, scale=H ** -0.5).to(X.DEV), w2=X.bf16(r, E, H, I, scale=I ** -0.5).to(X.DEV),
                mask=G.dev((r.random(T) < 0.9).astype(np.uint8)), go=X.bf16(r, T, H).to(X.DEV))


def _gated64(h):
    g, u = h[:, :I], h[:, I:]
    return g / (1 + np.exp(-g)) * u


def _reference(d, q=lambda a: a, q2=None):
    """The layer in 64 bits; q: what the first product's rows go through, q2: the second's."""
    ids, w, m = d["ids"].cpu().numpy(), d["w"].cpu().double().numpy(), d["mask"].cpu().numpy()
    x, w1, w2 = q(X.f64(d["x"].cpu())), d.get("w1_64", X.f64(d["w1"].cpu())), d.get("w2_64", X.f64(d["w2"].cpu()))
    out = np.zeros((T, H))
    for t in range(T):
        for j in range(K):
            if m[t] and ids[t, j] >= 0:
                h = _gated64(x[t:t + 1] @ w1[ids[t, j]].T)
                out[t] += w[t, j] * ((q2 or q)(h) @ w2[ids[t, j]].T)[0]
    return out


def _shapes(stride=0):
    rows = P * stride if stride else T * K
    return mg.make_experts_shape(rows, E, H, I, P, stride), mg.make_experts_shape(rows, E, I, H, P, stride), rows


def _norm(a):
    return float(np.sqrt((a ** 2).mean()))


@pytest.mark.parametrize("window", [False, True])
def test_bf16_layer(window):
    d = _world(1)
    shape = mg.make_shape(T, H, K, E, P)
    A = mg.rank_capacity(shape) if window else 0
    s1, s2, rows = _shapes(A)
    lay, ex, _, _ = mg.layout_dispatch(shape, mg.QUANT_NONE, d["x"], d["ids"], d["mask"], rank_stride=A)
    h = mg.experts_matmul(s1, ex, d["w1"], lay.expert_offsets, act=mg.ACT_SWIGLU)
    y = mg.experts_matmul(s2, h, d["w2"], lay.expert_offsets)
    out = mg.combine(shape, y, d["ids"], d["w"], lay.dst_row, d["mask"], rows=rows)
    got, ref = X.f64(out.cpu()), _reference(d)
    # three roundings to bf16, of h, of y and of the sum: in the mean each is far below half a step
    assert _norm(got - ref) <= 3 * X.BF16_HALF * _norm(ref)


def test_int8_layer():
    """Dynamic int8 rows from dispatch into int8 weights, the second product's rows quantised between."""
    d = _world(2)
    shape = mg.make_shape(T, H, K, E, P)
    s1, s2, rows = _shapes()
    q1, c1 = mg.quantize_rows(d["w1"], mg.ROWS_INT8)
    q2, c2 = mg.quantize_rows(d["w2"], mg.ROWS_INT8)
    lay, ex, xs, _ = mg.layout_dispatch(shape, mg.QUANT_DYNAMIC_INT8, d["x"], d["ids"], d["mask"])
    h = mg.experts_matmul(s1, ex, q1, lay.expert_offsets, xs, c1, mg.ACT_SWIGLU)
    hq, hs = mg.quantize_rows(h, mg.ROWS_INT8, shape=s2, expert_offsets=lay.expert_offsets)
    y = mg.experts_matmul(s2, hq, q2, lay.expert_offsets, hs, c2)
    out = mg.combine(shape, y, d["ids"], d["w"], lay.dst_row, d["mask"])
    d["w1_64"] = q1.cpu().double().numpy() * c1.cpu().double().numpy()[..., None]
    d["w2_64"] = q2.cpu().double().numpy() * c2.cpu().double().numpy()[..., None]

    def q(a):  # rows to the values of their codes
        amax = np.abs(a).max(1, keepdims=True)
        return np.rint(a * 127 / amax) * amax / 127

    ref = _reference(d, q)
    # h is rounded to bf16 before its codes are made: a code may move by one where the rounding crosses a
    # half, an error of at most one code step, amax / 127, in an element; each row's quantization
    # error is itself of that size, so the layer's is bounded by the layer of unquantised rows
    assert _norm(X.f64(out.cpu()) - ref) <= 3 * X.BF16_HALF * _norm(ref) + _norm(_reference(d) - ref)


def test_mxfp4_layer():
    d = _world(3)
    shape = mg.make_shape(T, H, K, E, P)
    s1, s2, rows = _shapes()
    q1, c1 = mg.quantize_rows(d["w1"], mg.ROWS_MXFP4)
    q2, c2 = mg.quantize_rows(d["w2"], mg.ROWS_MXFP4)
    lay, ex, _, _ = mg.layout_dispatch(shape, mg.QUANT_NONE, d["x"], d["ids"], d["mask"])
    xq, xs = mg.quantize_rows(ex, mg.ROWS_MXFP4, shape=s1, expert_offsets=lay.expert_offsets)
    h = mg.experts_matmul(s1, xq, q1, lay.expert_offsets, xs, c1, mg.ACT_SWIGLU)
    hq, hs = mg.quantize_rows(h, mg.ROWS_MXFP4, shape=s2, expert_offsets=lay.expert_offsets)
    y = mg.experts_matmul(s2, hq, q2, lay.expert_offsets, hs, c2)
    out = mg.combine(shape, y, d["ids"], d["w"], lay.dst_row, d["mask"])
    d["w1_64"] = X.unpack_mx(q1.cpu().numpy(), c1.cpu().numpy())
    d["w2_64"] = X.unpack_mx(q2.cpu().numpy(), c2.cpu().numpy())
    q = lambda a: X.unpack_mx(*X.quant_mx(a))  # noqa: E731
    ref = _reference(d, q)
    # as for int8: a moved code is an error of the size of the quantization's own
    assert _norm(X.f64(out.cpu()) - ref) <= 3 * X.BF16_HALF * _norm(ref) + _norm(_reference(d, q, lambda a: a) - ref)


def _train(d, stride=0):
    """Forward and backward of y = combine(relu(dispatch(x) w1^T) w2^T), the activation in torch."""
    shape = mg.make_shape(T, H, K, E, P)
    w1 = d["w1"][:, :I].contiguous()
    s1, s2, rows = _shapes(stride)
    lay, ex, _, _ = mg.layout_dispatch(shape, mg.QUANT_NONE, d["x"], d["ids"], d["mask"], rank_stride=stride)
    off = lay.expert_offsets
    h0 = mg.experts_matmul(s1, ex, w1, off)
    h = torch.relu(h0)
    y = mg.experts_matmul(s2, h, d["w2"], off)
    out = mg.combine(shape, y, d["ids"], d["w"], lay.dst_row, d["mask"], rows=rows)
    g = mg.combine_grad(shape, d["go"], y, d["ids"], d["w"], lay.dst_row, d["mask"], rows=rows)
    gw2 = mg.experts_matmul_wgrad(s2, g.grad_expert_out, h, off, dtype=torch.float32)
    gh = mg.experts_matmul_dgrad(s2, g.grad_expert_out, d["w2"], off)
    gh0 = torch.where(h0 > 0, gh, torch.zeros_like(gh))
    gw1 = mg.experts_matmul_wgrad(s1, gh0, ex, off, dtype=torch.float32)
    gex = mg.experts_matmul_dgrad(s1, gh0, w1, off)
    gx = mg.combine(shape, gex, d["ids"], torch.ones_like(d["w"]), lay.dst_row, d["mask"], rows=rows)
    return dict(out=out, gw=g.grad_topk_weights, gw1=gw1, gw2=gw2, gx=gx)


@pytest.mark.parametrize("window", [False, True])
def test_training_step_against_autograd_in_64_bits(window):
    d = _world(4)
    got = _train(d, mg.rank_capacity(mg.make_shape(T, H, K, E, P)) if window else 0)
    ids, m = d["ids"].cpu().long(), d["mask"].cpu()
    x, w, w1, w2 = (t.cpu().double().requires_grad_() for t in (d["x"], d["w"], d["w1"][:, :I], d["w2"]))
    out = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(K):
            if m[t] and ids[t, j] >= 0:
                h = torch.relu(x[t] @ w1[ids[t, j]].t())
                out[t] = out[t] + w[t, j] * (h @ w2[ids[t, j]].t())
    out.backward(d["go"].cpu().double())
    want = dict(out=out.detach(), gw=w.grad, gw1=w1.grad, gw2=w2.grad, gx=x.grad)
    for name, ref in want.items():
        # at most five tensors between the leaves and a result are rounded to bf16; a rounded h0 keeps its
        # sign, so the activation's gradient is the same
        err = (got[name].cpu().double() - ref).norm() / ref.norm()
        assert err <= 5 * X.BF16_HALF, (name, float(err))


def test_captured_and_replayed():
    """The training step and the quantised products in one graph, replayed with new inputs in place and
    eager work between the replays."""
    d, other = _world(5), [_world(6), _world(7), _world(8)]
    shape = mg.make_shape(T, H, K, E, P)
    s1, s2, rows = _shapes()
    q2, c2 = mg.quantize_rows(d["w2"], mg.ROWS_MXFP4)
    q1, c1 = mg.quantize_rows(d["w1"], mg.ROWS_INT8)

    def step(d):
        out = _train(d)
        lay, ex, xs, _ = mg.layout_dispatch(shape, mg.QUANT_DYNAMIC_INT8, d["x"], d["ids"], d["mask"])
        h = mg.experts_matmul(s1, ex, q1, lay.expert_offsets, xs, c1, mg.ACT_SWIGLU)
        hq, hs = mg.quantize_rows(h, mg.ROWS_MXFP4, shape=s2, expert_offsets=lay.expert_offsets)
        y = mg.experts_matmul(s2, hq, q2, lay.expert_offsets, hs, c2)
        out["q"] = mg.combine(shape, y, d["ids"], d["w"], lay.dst_row, d["mask"])
        return out

    step(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(d)
    for o in other + other[:1]:
        want = {k: v.clone() for k, v in step(o).items()}
        for k in ("ids", "w", "x", "w1", "w2", "mask", "go"):
            d[k].copy_(o[k])
        # the quantised weights are the first world's in both
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in want.items():
            assert torch.equal(got[k], v), k


def test_two_streams_at_once():
    """Two training steps on two streams give what each gives alone."""
    worlds = [_world(9), _world(10)]
    want = [{k: v.clone() for k, v in _train(d).items()} for d in worlds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in worlds]
    got = [None, None]
    for _ in range(5):
        for i, (d, s) in enumerate(zip(worlds, streams)):
            with torch.cuda.stream(s):
                got[i] = _train(d)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for k, v in w.items():
            assert torch.equal(g[k], v), k


def test_prepared_calls_and_given_streams():
    d = _world(11)
    s1, _, rows = _shapes()
    shape = mg.make_shape(T, H, K, E, P)
    lay, ex, _, _ = mg.layout_dispatch(shape, mg.QUANT_NONE, d["x"], d["ids"])
    call = mg.prepare_experts_matmul(s1, ex, d["w1"], lay.expert_offsets, act=mg.ACT_SWIGLU,
                                     out=torch.zeros(rows, I, dtype=torch.bfloat16, device=X.DEV))
    want = call().clone()
    torch.cuda.synchronize()
    call.result.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    assert torch.equal(call.result, want)
