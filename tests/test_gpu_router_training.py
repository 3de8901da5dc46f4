"""A whole training step of a gated layer in the library: the router with its balance losses, layout and dispatch, both
products with the gate between them (its input kept in bf16 or in 8 bits), the routing weights in the combine or at the
gate, and the way back to the logits; against autograd in 64 bits."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X

pytestmark = pytest.mark.gpu

T, H, I, K, E, P, S = 96, 256, 136, 4, 16, 4, 4
BC, ZC = 0.5, 0.05


def step(x, logits, bias, w_up, w_down, grad_out, kept, at_gate, stride, score):
    rs, bal = mg.make_route_shape(T, E, K, score, groups=4, topk_groups=3), mg.make_balance(S, BC, ZC)
    ids, weights = mg.route(rs, logits, bias)
    loss = mg.balance_loss(rs, bal, logits, ids)
    shape = mg.make_shape(T, H, K, E, P)
    rows = P * stride or T * K
    ew = torch.empty(rows, device=X.DEV) if at_gate else None  # the rows' routing weights
    lay, ex, _, _ = mg.layout_dispatch(shape, mg.QUANT_NONE, x, ids, rank_stride=stride, topk_weights=weights,
                                       expand_weights=ew)
    off = lay.expert_offsets
    eu = mg.make_experts_shape(rows, E, H, 2 * I, P, stride)
    ed = mg.make_experts_shape(rows, E, I, H, P, stride)
    h0 = mg.experts_matmul(eu, ex, w_up, off)
    f = mg.swiglu(h0, ew, checkpoint=kept, shape=ed, expert_offsets=off)
    keep = dict(codes=f.codes, scales=f.scales) if kept else dict(h0=h0)
    y = mg.experts_matmul(ed, f.out, w_down, off)
    wc = torch.ones_like(weights) if at_gate else weights
    out = mg.combine(shape, y, ids, wc, lay.dst_row, rows=rows)

    g = mg.combine_grad(shape, grad_out, y, ids, wc, lay.dst_row, rows=rows)
    gh = mg.experts_matmul_dgrad(ed, g.grad_expert_out, w_down, off)
    s = mg.swiglu_grad(gh, **keep, row_weights=ew, shape=ed, expert_offsets=off)
    gw_down = mg.experts_matmul_wgrad(ed, g.grad_expert_out, s.out, off, dtype=torch.float32)
    gw_up = mg.experts_matmul_wgrad(eu, s.grad_h0, ex, off, dtype=torch.float32)
    grad_rows = mg.experts_matmul_dgrad(eu, s.grad_h0, w_up, off)
    gx = mg.combine(shape, grad_rows, ids, torch.ones_like(weights), lay.dst_row, rows=rows)
    gl = mg.route_grad(rs, logits, ids, s.grad_row_weights if at_gate else g.grad_topk_weights, bal, loss,
                       dst_row=lay.dst_row if at_gate else None)
    return dict(out=out, losses=loss.losses, w_down=gw_down, w_up=gw_up, x=gx, logits=gl), ids


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("at_gate", [False, True])
@pytest.mark.parametrize("window", [False, True])
@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
def test_training_step(kept, at_gate, window, score):
    print(f"[step] {kept} {at_gate} {window} {score}", flush=True)
    r = np.random.default_rng(41)
    x, go = X.bf16(r, T, H), X.bf16(r, T, H)
    w_up, w_down = X.bf16(r, E, 2 * I, H, scale=H ** -0.5), X.bf16(r, E, H, I, scale=I ** -0.5)
    logits = torch.from_numpy(r.standard_normal((T, E)).astype(np.float32))
    bias = torch.from_numpy((0.2 * r.standard_normal(E)).astype(np.float32))
    stride = mg.rank_capacity(mg.make_shape(T, H, K, E, P)) if window else 0
    got, ids = step(*(t.to(X.DEV) for t in (x, logits, bias, w_up, w_down, go)), kept, at_gate, stride, score)
    ids = ids.cpu().long()
    assert bool((ids >= 0).all())
    leaves = dict(x=x, logits=logits, w_up=w_up, w_down=w_down)
    leaves = {k: v.double().requires_grad_() for k, v in leaves.items()}
    l = leaves["logits"]
    s = torch.softmax(l, 1) if score == mg.SCORE_SOFTMAX else torch.sigmoid(l)
    w = s.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    p = s / s.sum(1, keepdim=True)
    losses = torch.zeros(2, dtype=torch.float64)
    n = T // S
    balance = 0.0
    for g in range(S):
        c = torch.bincount(ids[g * n:(g + 1) * n].ravel(), minlength=E)
        balance = balance + BC / S * E / (K * n * n) * (c * p[g * n:(g + 1) * n].sum(0)).sum()
    z = float(np.float32(ZC)) / T * torch.logsumexp(l, 1).square().sum()
    losses = torch.stack((balance, z))
    out = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(K):
            h0 = leaves["x"][t] @ leaves["w_up"][ids[t, j]].t()
            h = torch.nn.functional.silu(h0[:I]) * h0[I:]
            out[t] = out[t] + w[t, j] * (h @ leaves["w_down"][ids[t, j]].t())
    ((out * go.double()).sum() + losses.sum()).backward()
    want = dict(out=out.detach(), losses=losses.detach(), **{k: v.grad for k, v in leaves.items()})
    # at most eight tensors between the leaves and a result are rounded to bf16 (dispatch's rows, h0, h, y or the rows'
    # gradient, gh, grad_h0, ..), each by at most half a step of an element, so that in the norm each adds at most half a
    # step; the activation's slope, at most 1.1, and its change with h0, at most 0.5 |u| + 1.1 where h0 has a deviation of
    # one, let h0's count up to twice.  A code is off by at most half of amax / 127 of its 128 elements, in the norm by
    # amax / (127 sqrt(12)); amax of 128 normal values stays below 4.5 of their deviation: 0.0103, counted twice for the same reason
    allowed = 10 * X.BF16_HALF + (2 * 4.5 / (127 * 12 ** 0.5) if kept else 0.0)
    for name, ref in want.items():
        err = (got[name].cpu().double() - ref).norm() / ref.norm()
        assert err <= (1e-5 if name == "losses" else allowed), (name, float(err))
