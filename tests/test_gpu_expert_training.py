"""A training step of a gated layer: the first product without the gate, the activation and its gradient in torch,
everything else in the library; against autograd in 64 bits."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X
from tests import _gpu as G

pytestmark = pytest.mark.gpu

T, H, I, K, E, P = 96, 256, 128, 4, 16, 4


def _step(x, topk_idx, topk_w, w_up, w_down, grad_out, stride):
    shape = mg.make_shape(T, H, K, E, P)
    lay, ex, _, _ = mg.layout_dispatch(shape, mg.QUANT_NONE, x, topk_idx, rank_stride=stride)
    rows, off = P * stride or T * K, lay.expert_offsets
    eu = mg.make_experts_shape(rows, E, H, 2 * I, P, stride)
    ed = mg.make_experts_shape(rows, E, I, H, P, stride)
    h0 = mg.experts_matmul(eu, ex, w_up, off).requires_grad_()
    h = torch.nn.functional.silu(h0[:, :I]) * h0[:, I:]
    hd = h.detach()
    y = mg.experts_matmul(ed, hd, w_down, off)
    out = mg.combine(shape, y, topk_idx, topk_w, lay.dst_row, rows=rows)

    g = mg.combine_grad(shape, grad_out, y, topk_idx, topk_w, lay.dst_row, rows=rows)
    gw_down = mg.experts_matmul_wgrad(ed, g.grad_expert_out, hd, off, dtype=torch.float32)
    gh = mg.experts_matmul_dgrad(ed, g.grad_expert_out, w_down, off)
    gh0, = torch.autograd.grad(h, h0, gh)
    gw_up = mg.experts_matmul_wgrad(eu, gh0, ex, off, dtype=torch.float32)
    grad_rows = mg.experts_matmul_dgrad(eu, gh0, w_up, off)
    gx = mg.combine(shape, grad_rows, topk_idx, torch.ones_like(topk_w), lay.dst_row, rows=rows)
    return dict(out=out, topk_w=g.grad_topk_weights, w_down=gw_down, w_up=gw_up, x=gx)


@pytest.mark.parametrize("window", [False, True])
def test_gated_training_step(window):
    r = np.random.default_rng(31)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :K].astype(np.int32)
    ids[r.random((T, K)) < 0.05] = -1
    w = r.random((T, K)).astype(np.float32)
    x, go = X.bf16(r, T, H), X.bf16(r, T, H)
    w_up, w_down = X.bf16(r, E, 2 * I, H, scale=H ** -0.5), X.bf16(r, E, H, I, scale=I ** -0.5)
    stride = mg.rank_capacity(mg.make_shape(T, H, K, E, P)) if window else 0
    got = _step(x.to(X.DEV), G.dev(ids), G.dev(w), w_up.to(X.DEV), w_down.to(X.DEV), go.to(X.DEV), stride)
    leaves = dict(x=x, topk_w=torch.from_numpy(w), w_up=w_up, w_down=w_down)
    leaves = {k: v.double().requires_grad_() for k, v in leaves.items()}
    out = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(K):
            if ids[t, j] >= 0:
                h0 = leaves["x"][t] @ leaves["w_up"][ids[t, j]].t()
                h = torch.nn.functional.silu(h0[:I]) * h0[I:]
                out[t] = out[t] + leaves["topk_w"][t, j] * (h @ leaves["w_down"][ids[t, j]].t())
    out.backward(go.double())
    want = dict(out=out.detach(), **{k: v.grad for k, v in leaves.items()})
    for name, ref in want.items():
        # at most seven tensors between the leaves and a result are rounded to bf16 (h0, silu(g), h, the rows' gradient, gh,
        # and in torch's gradient of the activation two more), each by at most half a step of an element, so that in
        # the norm each adds at most half a step; the activation's slope, at most 1.1, and its change with h0, at most
        # 0.5 |u| + 1.1, where h0 has a deviation of one, let h0's count up to twice
        err = (got[name].cpu().double() - ref).norm() / ref.norm()
        assert err <= 9 * X.BF16_HALF, (name, float(err))
