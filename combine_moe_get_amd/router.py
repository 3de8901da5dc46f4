"""ctypes binding of the router of libmoe_get (include/moe_get.h): the choice of each token's experts, the balance
losses and the gradient of the logits.

As in experts.py: argument checks and marshalling only, outputs allocated with PyTorch unless given, every step in the
HIP kernels, no CPU fallback; a call runs on the current stream of its tensors' device, or on the given one.
"""
import ctypes
from collections import namedtuple

import torch

from . import binding as B
from .experts import ExpertsCall, _device_of, _ptr, _result

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1


class RouteShape(ctypes.Structure):
    """moe_route_shape_t."""
    _fields_ = [
        ("num_tokens", ctypes.c_int32),
        ("num_ids", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("topk_groups", ctypes.c_int32),
        ("group_score", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]

    def __repr__(self):
        return "RouteShape(" + ", ".join(f"{f}={getattr(self, f)}" for f, _ in self._fields_) + ")"


class Balance(ctypes.Structure):
    """moe_balance_t."""
    _fields_ = [("segments", ctypes.c_int32), ("balance_coef", ctypes.c_float), ("z_coef", ctypes.c_float)]

    def __repr__(self):
        return "Balance(" + ", ".join(f"{f}={getattr(self, f)}" for f, _ in self._fields_) + ")"


def make_route_shape(T, E, K, score=SCORE_SOFTMAX, renormalize=True, scale=1.0, groups=1, topk_groups=1,
                     group_score=GROUP_MAX):
    """T tokens choose K of E ids (with special experts all of them) from the topk_groups best of `groups` groups."""
    return RouteShape(int(T), int(E), int(K), int(groups), int(topk_groups), int(group_score), int(score),
                      int(bool(renormalize)), float(scale))


def make_balance(segments=1, balance_coef=1.0, z_coef=0.0):
    """Coefficients of the balance loss, of the z loss, and the equal runs of tokens that are balanced each for itself."""
    return Balance(int(segments), float(balance_coef), float(z_coef))


_fns = None


def _lib():
    global _fns
    if _fns is None:
        L = B.lib()
        V, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        SP, BP = ctypes.POINTER(RouteShape), ctypes.POINTER(Balance)
        for name, args, res in (
                ("moe_route_check_shape", [SP], ctypes.c_int),
                ("moe_route", [SP, I32] + [V] * 6, ctypes.c_int),
                ("moe_balance_workspace_size", [SP, BP], SZ),
                ("moe_balance_loss", [SP, BP, I32] + [V] * 8 + [SZ, V], ctypes.c_int),
                ("moe_route_grad", [SP, I32] + [V] * 5 + [BP] + [V] * 5, ctypes.c_int),
                ("moe_route_grad_rows", [SP, I32] + [V] * 3 + [I64] + [V] * 2 + [BP] + [V] * 5, ctypes.c_int)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _fns = L
    return _fns


def check_route_shape(shape):
    """Status of moe_route_check_shape: 0, or a negative MOE_ERR_*."""
    return _lib().moe_route_check_shape(ctypes.byref(shape))


def balance_workspace_size(shape, balance):
    """Bytes of workspace of balance_loss (moe_balance_workspace_size)."""
    return _lib().moe_balance_workspace_size(ctypes.byref(shape), ctypes.byref(balance))


_FP32 = {torch.float32: 1, torch.bfloat16: 0}  # what logits may be


def _logits(shape, logits, what):
    """Device, type flag and address of the logits of a call, whose shape is valid."""
    dev = _device_of(logits, "logits")
    st = _lib().moe_route_check_shape(ctypes.byref(shape))
    if st != B.MOE_OK:
        raise B.MoeGetError(what, st)
    fp32 = _FP32.get(logits.dtype)
    if fp32 is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    numel = shape.num_tokens * shape.num_ids
    if not logits.is_contiguous() or logits.numel() < numel:
        B._ptr(logits, "logits", (logits.dtype,), numel)  # says what is wrong
    return dev, fp32, logits.data_ptr() or None


Route = namedtuple("Route", ["topk_idx", "topk_weights"])


def prepare_route(shape, logits, bias=None, x_active_mask=None, topk_idx=None, topk_weights=None):
    """Checked, marshalled moe_route call; see route()."""
    dev, fp32, logits_p = _logits(shape, logits, "route")
    T, E, K = shape.num_tokens, shape.num_ids, shape.topk
    topk_idx, idx_p = _result(topk_idx, "topk_idx", torch.int32, (T, K), (K, 1), dev)
    topk_weights, w_p = _result(topk_weights, "topk_weights", torch.float32, (T, K), (K, 1), dev)
    args = [
        ctypes.byref(shape), fp32,
        logits_p,
        None if bias is None else _ptr(bias, "bias", B.F32, E, dev),
        None if x_active_mask is None else _ptr(x_active_mask, "x_active_mask", B.U8, T, dev),
        idx_p, w_p, None,
    ]
    return ExpertsCall(_lib().moe_route, args, "route", (shape, logits, bias, x_active_mask),
                       Route(topk_idx, topk_weights), dev)


def route(shape, logits, bias=None, x_active_mask=None, topk_idx=None, topk_weights=None, stream=None):
    """moe_route: the K ids of each token and their weights, as layout() and combine() take them.
      logits  [T, E] float32 or bfloat16
      bias    float32 [E], added to the scores for the choice alone
    Returns Route(topk_idx int32 [T, K], topk_weights float32 [T, K]); -1 and 0 where no id is left."""
    return B.call_on(stream, prepare_route, shape, logits, bias, x_active_mask, topk_idx, topk_weights)


BalanceLoss = namedtuple("BalanceLoss", ["losses", "counts", "prob_sums", "segment_tokens"])


def prepare_balance_loss(shape, balance, logits, topk_idx, x_active_mask=None, workspace=None):
    """Checked, marshalled moe_balance_loss call; see balance_loss()."""
    dev, fp32, logits_p = _logits(shape, logits, "balance_loss")
    T, E, K, S = shape.num_tokens, shape.num_ids, shape.topk, balance.segments
    need = balance_workspace_size(shape, balance)
    if need == 0:
        raise B.MoeGetError("balance_loss", -4 if 4096 < S and T % S == 0 else -2)
    workspace, ws_p = _result(workspace, "workspace", torch.uint8, (need,), (1,), dev)
    losses, losses_p = _result(None, "losses", torch.float32, (2,), (1,), dev)
    counts, counts_p = _result(None, "counts", torch.int32, (S, E), (E, 1), dev)
    sums, sums_p = _result(None, "prob_sums", torch.float32, (S, E), (E, 1), dev)
    tokens, tokens_p = _result(None, "segment_tokens", torch.int32, (S,), (1,), dev)
    args = [
        ctypes.byref(shape), ctypes.byref(balance), fp32,
        logits_p,
        _ptr(topk_idx, "topk_idx", B.I32, T * K, dev),
        None if x_active_mask is None else _ptr(x_active_mask, "x_active_mask", B.U8, T, dev),
        losses_p, counts_p, sums_p, tokens_p, ws_p, workspace.numel(), None,
    ]
    return ExpertsCall(_lib().moe_balance_loss, args, "balance_loss",
                       (shape, balance, logits, topk_idx, x_active_mask, workspace),
                       BalanceLoss(losses, counts, sums, tokens), dev)


def balance_loss(shape, balance, logits, topk_idx, x_active_mask=None, workspace=None, stream=None):
    """moe_balance_loss: the balance and z losses of a batch's routing.
      balance    make_balance(segments, balance_coef, z_coef)
      topk_idx   int32 [T, K], as route() gave it
      workspace  uint8, balance_workspace_size(shape, balance) bytes; made by the call if not given
    Returns a BalanceLoss: losses float32 [2] (balance, z), counts int32 [segments, E], prob_sums float32 [segments, E],
    segment_tokens int32 [segments]."""
    return B.call_on(stream, prepare_balance_loss, shape, balance, logits, topk_idx, x_active_mask, workspace)


def prepare_route_grad(shape, logits, topk_idx, grad_topk_weights=None, balance=None, balance_loss=None, grad_losses=None,
                       x_active_mask=None, dst_row=None, out=None):
    """Checked, marshalled moe_route_grad call; see route_grad()."""
    dev, fp32, logits_p = _logits(shape, logits, "route_grad")
    T, E, K = shape.num_tokens, shape.num_ids, shape.topk
    if (balance is None) != (balance_loss is None):
        raise ValueError("balance and balance_loss go together")
    if balance is None and (grad_topk_weights is None or grad_losses is not None):
        raise ValueError("grad_topk_weights is needed where there are no losses" if grad_topk_weights is None else
                         "grad_losses needs balance and balance_loss")
    if dst_row is not None and grad_topk_weights is None:
        raise ValueError("dst_row needs grad_topk_weights (of receive rows)")
    counts = tokens = None
    S = 0
    if balance is not None:
        S, counts, tokens = balance.segments, balance_loss.counts, balance_loss.segment_tokens
        if counts.numel() != S * E or tokens.numel() != S:
            raise ValueError(f"balance_loss holds counts {tuple(counts.shape)} of {tokens.numel()} segments: not of these "
                             f"{S} segments of {E} ids")
    out, out_p = _result(out, "out", logits.dtype, (T, E), (E, 1), dev)
    args = [
        ctypes.byref(shape), fp32,
        logits_p,
        _ptr(topk_idx, "topk_idx", B.I32, T * K, dev, required=grad_topk_weights is not None),
        _ptr(grad_topk_weights, "grad_topk_weights", B.F32, T * K if dst_row is None else None, dev, required=False),
        *(() if dst_row is None else (grad_topk_weights.numel(),)),
        None if dst_row is None else _ptr(dst_row, "dst_row", B.I32, T * K, dev),
        None if x_active_mask is None else _ptr(x_active_mask, "x_active_mask", B.U8, T, dev),
        ctypes.byref(balance) if balance is not None else None,
        _ptr(counts, "counts", B.I32, S * E, dev, required=False),
        _ptr(tokens, "segment_tokens", B.I32, S, dev, required=False),
        _ptr(grad_losses, "grad_losses", B.F32, 2, dev, required=False),
        out_p, None,
    ]
    return ExpertsCall(_lib().moe_route_grad if dst_row is None else _lib().moe_route_grad_rows, args, "route_grad",
                       (shape, logits, topk_idx, grad_topk_weights, dst_row, x_active_mask, balance, counts, tokens, grad_losses),
                       out, dev)


def route_grad(shape, logits, topk_idx, grad_topk_weights=None, balance=None, balance_loss=None, grad_losses=None,
               x_active_mask=None, dst_row=None, out=None, stream=None):
    """moe_route_grad: the gradient of the logits (of their type) through route()'s weights and balance_loss()'s losses,
    together in one pass.
      grad_topk_weights      float32 [T, K] (combine_grad's); None: the losses alone
      balance, balance_loss  as given to and returned by balance_loss() for this shape; None: the weights alone
      grad_losses            float32 [2]; None: ones
      dst_row                int32 [T, K] of the layout: grad_topk_weights is then float32 [rows], swiglu_grad's
                             grad_row_weights, and each slot takes its receive row's (0 for a row that it does not hold)"""
    return B.call_on(stream, prepare_route_grad, shape, logits, topk_idx, grad_topk_weights, balance, balance_loss,
                     grad_losses, x_active_mask, dst_row, out)
