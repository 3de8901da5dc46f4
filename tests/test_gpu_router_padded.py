"""A training step of a padded batch gives the live tokens what a batch of them alone gives, and the others nothing; also with
special experts among the ids."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X
from tests import _router as R

pytestmark = pytest.mark.gpu

H, I, K, E, P = 256, 136, 4, 16, 4


def step(x, logits, bias, w_up, w_down, grad_out, mask, special, score):
    T, n = logits.shape
    rs, bal = mg.make_route_shape(T, n, K, score), mg.make_balance(1, 0.5, 0.05)
    ids, weights = mg.route(rs, logits, bias, x_active_mask=mask)
    loss = mg.balance_loss(rs, bal, logits, ids, x_active_mask=mask)
    shape = mg.make_shape(T, H, K, E, P, *special)
    lay, ex, _, _ = mg.layout_dispatch(shape, mg.QUANT_NONE, x, ids, x_active_mask=mask)
    off, rows = lay.expert_offsets, T * K
    eu, ed = mg.make_experts_shape(rows, E, H, 2 * I, P), mg.make_experts_shape(rows, E, I, H, P)
    h0 = mg.experts_matmul(eu, ex, w_up, off)
    f = mg.swiglu(h0, checkpoint=True, shape=ed, expert_offsets=off)
    y = mg.experts_matmul(ed, f.out, w_down, off)
    ori = x if sum(special[1:]) else None
    cv = [torch.linspace(-1, 1, H, device=X.DEV).bfloat16().expand(special[2], H).contiguous()] * 3 if special[2] else [None] * 3
    out = mg.combine(shape, y, ids, weights, lay.dst_row, x_active_mask=mask, ori_x=ori, const_alpha1=cv[0], const_alpha2=cv[1],
                     const_v=cv[2], rows=rows)
    g = mg.combine_grad(shape, grad_out, y, ids, weights, lay.dst_row, x_active_mask=mask, ori_x=ori, const_alpha1=cv[0],
                        const_alpha2=cv[1], const_v=cv[2], rows=rows)
    gh = mg.experts_matmul_dgrad(ed, g.grad_expert_out, w_down, off)
    s = mg.swiglu_grad(gh, codes=f.codes, scales=f.scales, shape=ed, expert_offsets=off)
    gw_down = mg.experts_matmul_wgrad(ed, g.grad_expert_out, s.out, off, dtype=torch.float32)
    gw_up = mg.experts_matmul_wgrad(eu, s.grad_h0, ex, off, dtype=torch.float32)
    gl = mg.route_grad(rs, logits, ids, g.grad_topk_weights, bal, loss, x_active_mask=mask)
    return dict(ids=ids, weights=weights, out=out, logits=gl), dict(up=gw_up, down=gw_down, counts=loss.counts, tokens=loss.segment_tokens), loss


@pytest.mark.parametrize("special", [(0, 0, 0), (2, 1, 1)])
@pytest.mark.parametrize("score", [mg.SCORE_SOFTMAX, mg.SCORE_SIGMOID])
def test_padded_batch(score, special):
    print(f"[padded] {score} {special}", flush=True)
    r = np.random.default_rng(7)
    T, live, n = 96, 64, E + sum(special)
    mask = np.zeros(T, np.uint8)
    mask[r.permutation(T)[:live]] = 1
    at = torch.from_numpy(np.flatnonzero(mask)).to(X.DEV)
    x, go = X.bf16(r, T, H).to(X.DEV), X.bf16(r, T, H).to(X.DEV)
    w_up, w_down = X.bf16(r, E, 2 * I, H, scale=H ** -0.5).to(X.DEV), X.bf16(r, E, H, I, scale=I ** -0.5).to(X.DEV)
    logits = torch.from_numpy(r.standard_normal((T, n)).astype(np.float32)).to(X.DEV)
    bias = torch.from_numpy((0.2 * r.standard_normal(n)).astype(np.float32)).to(X.DEV)
    m = torch.from_numpy(mask).to(X.DEV)
    for t in (x, go, logits):  # what padding holds does not matter
        t[m == 0] = float("nan")
    token, whole, loss = step(x, logits, bias, w_up, w_down, go, m, special, score)
    token1, whole1, loss1 = step(x[at], logits[at], bias, w_up, w_down, go[at], None, special, score)
    for k, v in whole.items():
        assert torch.equal(v, whole1[k]), k
    # the losses and their part of the gradient: the same terms, added in an order that the batch's size fixes
    rel = (4 * float(logits[at].abs().max()) + n / 8 + 32 + 64) * R.STEP32
    assert bool(((loss.losses - loss1.losses).abs() <= 2 * rel * loss1.losses.abs()).all())
    for k in ("ids", "weights", "out"):
        assert torch.equal(token[k][at], token1[k]), k
    assert torch.equal(token["logits"][at], token1["logits"])  # counts and numbers of tokens are whole numbers
    off = m == 0
    assert bool((token["ids"][off] == -1).all()) and bool((token["weights"][off] == 0).all()) and bool((token["logits"][off] == 0).all())
