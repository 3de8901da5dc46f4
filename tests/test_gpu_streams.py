"""Calls on a stream that is not the current one, whose arguments and results the caller drops at once while the
stream is still busy with something else."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X
from tests import _gpu as G

pytestmark = pytest.mark.gpu

T, H, I, K, E = 64, 256, 128, 4, 8


def _world():
    r = np.random.default_rng(21)
    b = lambda *s: X.bf16(r, *s).to(X.DEV)  # noqa: E731
    shape = mg.make_shape(T, H, K, E, 2, 0, 1, 1)
    ids = G.dev(np.argsort(r.random((T, E + 2)), axis=1)[:, :K].astype(np.int32))
    lay = mg.layout(shape, ids)
    s = mg.make_experts_shape(T * K, E, H, I)
    return dict(shape=shape, s=s, ids=ids, dst=lay.dst_row, off=lay.expert_offsets, w=G.dev(r.random((T, K)).astype(np.float32)),
                x=b(T, H), y=b(T * K, H), rows=b(T * K, H), wt=b(E, I, H), dy=b(T * K, I), a=[b(1, H) for _ in range(3)])


# the arguments that a call reads, and the call
CALLS = {
    "experts_matmul": (("rows", "wt", "off"),
                       lambda d, t, s: mg.experts_matmul(d["s"], t["rows"], t["wt"], t["off"], stream=s)),
    "experts_matmul_dgrad": (("dy", "wt", "off"),
                             lambda d, t, s: mg.experts_matmul_dgrad(d["s"], t["dy"], t["wt"], t["off"], stream=s)),
    "experts_matmul_wgrad": (("dy", "rows", "off"),
                             lambda d, t, s: mg.experts_matmul_wgrad(d["s"], t["dy"], t["rows"], t["off"], stream=s)),
    "quantize_rows": (("rows",), lambda d, t, s: mg.quantize_rows(t["rows"], mg.ROWS_INT8, stream=s)),
    "combine_grad": (("x", "y", "ids", "w", "dst"),
                     lambda d, t, s: mg.combine_grad(d["shape"], t["x"], t["y"], t["ids"], t["w"], t["dst"], None, t["x"],
                                                     *d["a"], stream=s)[1:]),
}


def _tensors(out):
    return [out] if isinstance(out, torch.Tensor) else [t for o in out for t in _tensors(o)] if isinstance(out, tuple) else []


@pytest.mark.parametrize("name", list(CALLS))
def test_arguments_and_results_dropped_at_once(name):
    d = _world()
    keys, call = CALLS[name]
    used = int(d["off"][-1])
    cut = lambda t: t[:used] if t.shape[0] == T * K else t  # noqa: E731  rows of no expert: not written
    want = [cut(t).clone() for t in _tensors(call(d, d, None))]
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
        assert all(torch.equal(cut(o), w) for o, w in zip(out, want))
        assert all(bool((f == 1).all()) for f in fresh)


def test_a_layer_on_a_side_stream():
    """Layout (whose status word is cleared by the call), dispatch and combine on a stream that is busy, with the workspace
    and the arguments gone."""
    d = _world()
    shape = mg.make_shape(T, H, K, E, 2)
    ids, x, w = (d[k].clone() for k in ("ids", "x", "w"))
    ids[ids >= E] = -1

    def layer(ids, x, w, s):
        lay, ex, _, _ = mg.layout_dispatch(shape, mg.QUANT_NONE, x, ids, stream=s)
        again = mg.layout(shape, ids, stream=s)
        ex2 = mg.dispatch(shape, mg.QUANT_NONE, x, again.dst_row, stream=s)[0]
        noalloc = mg.layout_noalloc(shape, ids, stream=s)
        out = mg.combine(shape, ex2, ids, w, noalloc.dst_row, stream=s)
        n = int((ids >= 0).sum())
        return [lay.dst_row, lay.status, again.dst_row, again.status, noalloc.status, ex[:n], ex2[:n], out]

    want = [t.clone() for t in layer(ids, x, w, None)]
    side = torch.cuda.Stream()
    for _ in range(3):
        args = [t.clone() for t in (ids, x, w)]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = layer(*args, side)
        del args
        fresh = [torch.full((n,), 3, dtype=torch.int32, device=X.DEV) for n in (1, 1, 1, T * K, T * K, T * H // 2, 1 << 16)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(bool((f == 3).all()) for f in fresh)


@pytest.mark.parametrize("name", list(CALLS))
def test_captured_on_a_stream_that_joins_the_capture(name):
    """Two calls on a side stream inside a capture, the first one's results dropped there; replayed with eager work and
    synchronizations between the replays."""
    d = _world()
    keys, call = CALLS[name]
    used = int(d["off"][-1])
    cut = lambda t: t[:used] if t.shape[0] == T * K else t  # noqa: E731  rows of no expert: not written
    call(d, d, None)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    t = {k: d[k].clone() for k in keys}
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        call(d, t, side)
        got = _tensors(call(d, t, side))
        torch.cuda.current_stream().wait_stream(side)
    for k in range(3):
        for key, v in t.items():
            if v.dtype == torch.bfloat16:
                v.copy_(d[key] * (k + 1))
        want = [cut(w).clone() for w in _tensors(call(d, t, None))]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(cut(g), w) for g, w in zip(got, want)), k
        torch.ones(1 << 20, device=X.DEV).sum()
