"""ctypes binding of the expert stage of libmoe_get (include/moe_get.h): products grouped by
expert, their gradients, row quantization, the gate with its gradient and the combine's gradient.

As in binding.py: argument checks and marshalling only, outputs allocated with PyTorch unless
given, every step in the HIP kernels, no CPU fallback.  All tensors of a call must be on one
device; the call runs on that device's current stream (or the given one of that device),
whichever device is current.  With `stream=` arguments and results may be dropped at once (binding.call_on);
a prepare_* call makes its results in the memory of the stream that is current then, keeps its tensors
alive itself, and is to be kept until what it issued on other streams is done.
"""
import ctypes
import math
from collections import namedtuple

import torch

from . import binding as B

ROWS_BF16, ROWS_INT8, ROWS_MXFP4 = 0, 1, 2
ACT_NONE, ACT_SWIGLU = 0, 1
EXPERTS_FORWARD, EXPERTS_DGRAD, EXPERTS_WGRAD = 0, 1, 2

# a device's current stream as a hipStream_t, and the current device: without the objects that torch.cuda makes of them, where
# torch has these names (a build without has torch.cuda's)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())

_TYPE_OF = {torch.bfloat16: ROWS_BF16, torch.int8: ROWS_INT8, torch.uint8: ROWS_MXFP4}
U8 = (torch.uint8,)


class ExpertsShape(ctypes.Structure):
    """moe_experts_shape_t."""
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("rank_stride", ctypes.c_int64),
        ("num_experts", ctypes.c_int32),
        ("num_ranks", ctypes.c_int32),
        ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32),
    ]

    def __repr__(self):
        return "ExpertsShape(" + ", ".join(f"{f}={getattr(self, f)}" for f, _ in self._fields_) + ")"


def make_experts_shape(rows, E, in_features, out_features, P=1, rank_stride=0):
    """rows: rows of the row buffers; E experts on P ranks; rank_stride: window length of a
    fixed-capacity layout (0: compact rows, where P does not matter)."""
    return ExpertsShape(int(rows), int(rank_stride), int(E), int(P), int(in_features), int(out_features))


_fns = None


def _lib():
    global _fns
    if _fns is None:
        L = B.lib()
        V, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        SP = ctypes.POINTER(ExpertsShape)
        for name, args in (
                ("moe_experts_check_shape", [SP, I32]),
                ("moe_experts_tile", [SP, I32, I32, I32, ctypes.POINTER(I32 * 3)]),
                ("moe_experts_matmul", [SP, I32, I32] + [V] * 7),
                ("moe_experts_matmul_dgrad", [SP] + [V] * 5),
                ("moe_experts_matmul_wgrad", [SP, I32] + [V] * 5),
                ("moe_quantize_rows", [I32, I64, I32, V, V, V, SP, V, V]),
                ("moe_swiglu", [I64, I32, V, V, SP, V, V, V, V, V]),
                ("moe_swiglu_grad", [I64, I32, V, V, V, V, V, SP, V, V, V, V, V]),
                ("moe_combine_grad", [ctypes.POINTER(B.Shape)] + [V] * 17)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        _fns = L
    return _fns


def check_experts_shape(shape, row_type):
    """Status of moe_experts_check_shape: 0, or a negative MOE_ERR_*."""
    return _lib().moe_experts_check_shape(ctypes.byref(shape), int(row_type))


def experts_tile(shape, op=EXPERTS_FORWARD, row_type=ROWS_BF16, act=ACT_NONE):
    """(rows, columns, stages in LDS) of the tile that a product of this shape runs on (moe_experts_tile)."""
    tile = (ctypes.c_int32 * 3)()
    st = _lib().moe_experts_tile(ctypes.byref(shape), int(op), int(row_type), int(act), ctypes.byref(tile))
    if st != B.MOE_OK:
        raise B.MoeGetError("experts_tile", st)
    return tuple(tile)


class ExpertsCall(B.PreparedCall):
    """A PreparedCall on the device of its tensors, whichever device is current."""

    __slots__ = ("_device",)

    def __init__(self, fn, args, what, keep, result, device):
        self._fn, self._args, self._what, self._keep, self.result = fn, args, what, keep, result
        self._device = device

    def __call__(self, stream=None):
        device = self._device
        if stream is not None and stream.device != device:
            raise ValueError(f"{self._what}: the stream is on {stream.device}, the tensors on {device}")
        index = device.index
        if _current_device() != index:
            with torch.cuda.device(device):
                return self._run(index, stream)
        return self._run(index, stream)

    def _run(self, index, stream):
        # the current stream's handle alone: an object for it takes 1.8 us, a quarter of a small call
        self._args[-1] = _raw_stream(index) if stream is None else stream.cuda_stream
        st = self._fn(*self._args)
        if st != B.MOE_OK:
            raise B.MoeGetError(self._what, st)
        return self.result


def _ptr(t, name, dtypes, numel, device, required=True):
    """Address of a tensor that is fit for the call, or None for an optional or empty one."""
    if t is None and not required:
        return None
    # everything in order: the case that calls spend their time on
    if (isinstance(t, torch.Tensor) and t.device == device and t.dtype in dtypes and t.is_contiguous()
            and (numel is None or t.numel() >= numel)):
        return t.data_ptr() or None
    B._ptr(t, name, dtypes, numel, required)  # says what is wrong
    raise ValueError(f"{name} is on {t.device}, other tensors of the call on {device}")


def _result(t, name, dtype, size, strides, device):
    """(tensor, address) of a result: the given one if it is fit for the call, else a new one."""
    if t is None:
        t = torch.empty_strided(size, strides, dtype=dtype, device=device)  # 1.1 us; torch.empty 1.7
        return t, t.data_ptr() or None
    return t, _ptr(t, name, (dtype,), math.prod(size), device)


def _checked(shape, row_type, what):
    st = check_experts_shape(shape, row_type)
    if st != B.MOE_OK:
        raise B.MoeGetError(what, st)


def _device_of(t, name):
    if isinstance(t, torch.Tensor) and t.is_cuda:
        return t.device
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device (HIP) tensor, got {t.device}")
    return t.device


def prepare_experts_matmul(shape, x, w, expert_offsets, row_scales=None, w_scales=None, act=ACT_NONE, out=None):
    """Checked, marshalled moe_experts_matmul call; see experts_matmul()."""
    dev = _device_of(x, "x")
    if x.dtype not in _TYPE_OF:
        raise TypeError(f"x must be bfloat16, int8 or uint8 (packed MXFP4), got {x.dtype}")
    ty = _TYPE_OF[x.dtype]
    _checked(shape, ty, "experts_matmul")
    if act not in (ACT_NONE, ACT_SWIGLU):
        raise ValueError(f"act must be ACT_NONE or ACT_SWIGLU, got {act}")
    if ty == ROWS_BF16 and (row_scales is not None or w_scales is not None):
        raise ValueError("bfloat16 rows take no scales")
    rows, E, k, n = shape.rows, shape.num_experts, shape.in_features, shape.out_features
    nw = n * (2 if act == ACT_SWIGLU else 1)
    kx = k // 2 if ty == ROWS_MXFP4 else k
    if out is None:
        out = torch.empty((rows, n), dtype=torch.bfloat16, device=dev)
    sdt = U8 if ty == ROWS_MXFP4 else B.F32
    per = k // 32 if ty == ROWS_MXFP4 else 1
    args = [
        ctypes.byref(shape), ty, int(act),
        _ptr(x, "x", (x.dtype,), rows * kx, dev),
        _ptr(row_scales, "row_scales", sdt, rows * per, dev, required=ty == ROWS_MXFP4),
        _ptr(w, "w", (x.dtype,), E * nw * kx, dev),
        _ptr(w_scales, "w_scales", sdt, E * nw * per, dev, required=ty == ROWS_MXFP4),
        _ptr(expert_offsets, "expert_offsets", B.I32, E + 1, dev),
        _ptr(out, "out", B.BF16, rows * n, dev),
        None,
    ]
    return ExpertsCall(_lib().moe_experts_matmul, args, "experts_matmul",
                       (shape, x, row_scales, w, w_scales, expert_offsets), out, dev)


def experts_matmul(shape, x, w, expert_offsets, row_scales=None, w_scales=None, act=ACT_NONE, out=None, stream=None):
    """moe_experts_matmul: out[r] = act(x[r] w[e]^T) for the rows r of every expert e.
      x          [rows, in] bfloat16; int8 codes; or uint8 [rows, in / 2] packed MXFP4
      w          [E, Nw, in] of the same type, Nw = out_features (twice that with ACT_SWIGLU:
                 out = silu(g) * u, the rows of g first)
      row_scales int8: float32 [rows] (dispatch's dynamic_scales; None: ones); MXFP4: uint8 [rows, in / 32]
      w_scales   int8: float32 [E, Nw] (None: ones); MXFP4: uint8 [E, Nw, in / 32]
      expert_offsets  int32 [E + 1] of the layout
    Returns out [rows, out_features] bfloat16; rows of no expert are left as they were."""
    return B.call_on(stream, prepare_experts_matmul, shape, x, w, expert_offsets, row_scales, w_scales, act, out)


def prepare_experts_matmul_dgrad(shape, grad_out, w, expert_offsets, out=None):
    """Checked, marshalled moe_experts_matmul_dgrad call; see experts_matmul_dgrad()."""
    dev = _device_of(grad_out, "grad_out")
    _checked(shape, ROWS_BF16, "experts_matmul_dgrad")
    rows, E, k, n = shape.rows, shape.num_experts, shape.in_features, shape.out_features
    if out is None:
        out = torch.empty((rows, k), dtype=torch.bfloat16, device=dev)
    args = [
        ctypes.byref(shape),
        _ptr(grad_out, "grad_out", B.BF16, rows * n, dev),
        _ptr(w, "w", B.BF16, E * n * k, dev),
        _ptr(expert_offsets, "expert_offsets", B.I32, E + 1, dev),
        _ptr(out, "out", B.BF16, rows * k, dev),
        None,
    ]
    return ExpertsCall(_lib().moe_experts_matmul_dgrad, args, "experts_matmul_dgrad",
                       (shape, grad_out, w, expert_offsets), out, dev)


def experts_matmul_dgrad(shape, grad_out, w, expert_offsets, out=None, stream=None):
    """moe_experts_matmul_dgrad: the gradient grad_out[r] w[e] [rows, in_features] of the bf16
    product's rows (shape as given to experts_matmul).  Rows of no expert are left as they were."""
    return B.call_on(stream, prepare_experts_matmul_dgrad, shape, grad_out, w, expert_offsets, out)


def prepare_experts_matmul_wgrad(shape, grad_out, x, expert_offsets, dtype=torch.bfloat16, out=None):
    """Checked, marshalled moe_experts_matmul_wgrad call; see experts_matmul_wgrad()."""
    dev = _device_of(expert_offsets, "expert_offsets")
    _checked(shape, ROWS_BF16, "experts_matmul_wgrad")
    rows, E, k, n = shape.rows, shape.num_experts, shape.in_features, shape.out_features
    if out is not None:
        dtype = out.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"the weights' gradient must be bfloat16 or float32, got {dtype}")
    if out is None:
        out = torch.empty((E, n, k), dtype=dtype, device=dev)
    args = [
        ctypes.byref(shape), int(dtype == torch.float32),
        _ptr(grad_out, "grad_out", B.BF16, rows * n, dev),
        _ptr(x, "x", B.BF16, rows * k, dev),
        _ptr(expert_offsets, "expert_offsets", B.I32, E + 1, dev),
        _ptr(out, "out", (dtype,), E * n * k, dev),
        None,
    ]
    return ExpertsCall(_lib().moe_experts_matmul_wgrad, args, "experts_matmul_wgrad",
                       (shape, grad_out, x, expert_offsets), out, dev)


def experts_matmul_wgrad(shape, grad_out, x, expert_offsets, dtype=torch.bfloat16, out=None, stream=None):
    """moe_experts_matmul_wgrad: the gradient grad_out^T x over each expert's rows
    [E, out_features, in_features] of the bf16 product's weights, in dtype (bfloat16 or float32;
    that of out if given).  Zeros for experts without rows."""
    return B.call_on(stream, prepare_experts_matmul_wgrad, shape, grad_out, x, expert_offsets, dtype, out)


def prepare_quantize_rows(x, row_type, codes=None, scales=None, shape=None, expert_offsets=None):
    """Checked, marshalled moe_quantize_rows call; see quantize_rows()."""
    dev = _device_of(x, "x")
    if row_type not in (ROWS_INT8, ROWS_MXFP4):
        raise ValueError(f"row_type must be ROWS_INT8 or ROWS_MXFP4, got {row_type}")
    if x.dim() < 1:
        raise ValueError("x must have rows")
    features = x.shape[-1]
    step = 16 if row_type == ROWS_INT8 else 32
    if features == 0 or features % step:
        raise ValueError(f"the rows of x hold {features} elements: a multiple of {step} is needed")
    rows = x.numel() // features
    lead = tuple(x.shape[:-1])
    if codes is None:
        codes = torch.empty(lead + ((features,) if row_type == ROWS_INT8 else (features // 2,)),
                            dtype=torch.int8 if row_type == ROWS_INT8 else torch.uint8, device=dev)
    if scales is None:
        scales = (torch.empty(lead, dtype=torch.float32, device=dev) if row_type == ROWS_INT8 else
                  torch.empty(lead + (features // 32,), dtype=torch.uint8, device=dev))
    if (shape is None) != (expert_offsets is None):
        raise ValueError("shape and expert_offsets go together")
    mx = row_type == ROWS_MXFP4
    args = [
        int(row_type), rows, features,
        _ptr(x, "x", B.BF16, None, dev),
        _ptr(codes, "codes", U8 if mx else (torch.int8,), rows * (features // 2 if mx else features), dev),
        _ptr(scales, "scales", U8 if mx else B.F32, rows * (features // 32 if mx else 1), dev),
        ctypes.byref(shape) if shape is not None else None,
        _ptr(expert_offsets, "expert_offsets", B.I32, shape.num_experts + 1 if shape is not None else None, dev,
             required=False),
        None,
    ]
    return ExpertsCall(_lib().moe_quantize_rows, args, "quantize_rows", (x, shape, expert_offsets),
                       (codes, scales), dev)


def quantize_rows(x, row_type, codes=None, scales=None, shape=None, expert_offsets=None, stream=None):
    """moe_quantize_rows: bfloat16 x [..., features] to ROWS_INT8 (int8 codes like x, float32 scales
    [...]) or ROWS_MXFP4 (uint8 codes [..., features / 2], uint8 scales [..., features / 32]).  With
    shape and expert_offsets only rows that belong to an expert are touched; without, all (weights).
    Returns (codes, scales)."""
    return B.call_on(stream, prepare_quantize_rows, x, row_type, codes, scales, shape, expert_offsets)


Swiglu = namedtuple("Swiglu", ["out", "codes", "scales"])
SwigluGrad = namedtuple("SwigluGrad", ["grad_h0", "out", "grad_row_weights"])
I8 = (torch.int8,)


def _gate_rows(t, name, halves):
    """(rows, features) of a tensor of rows that hold `halves` times the features."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, {'2 * ' if halves == 2 else ''}features]")
    rows, n = t.shape
    if n == 0 or n % (8 * halves):
        raise ValueError(f"the rows of {name} hold {n} elements: a multiple of {8 * halves} is needed")
    return rows, n // halves


def prepare_swiglu(h0, row_weights=None, checkpoint=False, shape=None, expert_offsets=None, out=None, codes=None,
                   scales=None):
    """Checked, marshalled moe_swiglu call; see swiglu()."""
    dev = _device_of(h0, "h0")
    rows, n = _gate_rows(h0, "h0", 2)
    if (shape is None) != (expert_offsets is None):
        raise ValueError("shape and expert_offsets go together")
    if (codes is not None or scales is not None) and not checkpoint:
        raise ValueError("codes and scales are results of a checkpoint")
    out, out_p = _result(out, "out", torch.bfloat16, (rows, n), (n, 1), dev)
    codes_p = scales_p = None
    if checkpoint:
        codes, codes_p = _result(codes, "codes", torch.int8, (rows, 2 * n), (2 * n, 1), dev)
        nb = (n + 127) // 128
        scales, scales_p = _result(scales, "scales", torch.float32, (rows, 2, nb), (2 * nb, nb, 1), dev)
    args = [
        rows, n,
        _ptr(h0, "h0", B.BF16, None, dev),
        _ptr(row_weights, "row_weights", B.F32, rows, dev, required=False),
        ctypes.byref(shape) if shape is not None else None,
        _ptr(expert_offsets, "expert_offsets", B.I32, shape.num_experts + 1 if shape is not None else None, dev,
             required=False),
        out_p, codes_p, scales_p, None,
    ]
    return ExpertsCall(_lib().moe_swiglu, args, "swiglu", (h0, row_weights, shape, expert_offsets),
                       Swiglu(out, codes, scales), dev)


def swiglu(h0, row_weights=None, checkpoint=False, shape=None, expert_offsets=None, out=None, codes=None, scales=None,
           stream=None):
    """moe_swiglu: out[r] = row_weights[r] silu(g) u of the rows h0[r] = [g | u], bfloat16 [rows, 2 * features].
      row_weights  float32 [rows] (dispatch's expand_weights; None: ones)
      checkpoint   also keep h0 in 8 bits for swiglu_grad: codes int8 [rows, 2 * features] and scales float32
                   [rows, 2, ceil(features / 128)]
      shape, expert_offsets  of the second product (in_features = features): only rows of experts are touched;
                   both None: all rows
    Returns a Swiglu(out [rows, features] bfloat16, codes, scales); the last two None without a checkpoint."""
    return B.call_on(stream, prepare_swiglu, h0, row_weights, checkpoint, shape, expert_offsets, out, codes, scales)


def prepare_swiglu_grad(grad_out, h0=None, codes=None, scales=None, row_weights=None, shape=None, expert_offsets=None,
                        grad_h0=None, out=None, grad_row_weights=None, need_out=True):
    """Checked, marshalled moe_swiglu_grad call; see swiglu_grad()."""
    dev = _device_of(grad_out, "grad_out")
    rows, n = _gate_rows(grad_out, "grad_out", 1)
    if (shape is None) != (expert_offsets is None):
        raise ValueError("shape and expert_offsets go together")
    if (codes is None) != (scales is None) or (h0 is None) == (codes is None):
        raise ValueError("either h0 or codes and scales are needed")
    if out is not None and not need_out:
        raise ValueError("out is given but need_out is not set")
    grad_h0, grad_h0_p = _result(grad_h0, "grad_h0", torch.bfloat16, (rows, 2 * n), (2 * n, 1), dev)
    out_p = grad_w_p = None
    if need_out:
        out, out_p = _result(out, "out", torch.bfloat16, (rows, n), (n, 1), dev)
    if grad_row_weights is not None or row_weights is not None:
        grad_row_weights, grad_w_p = _result(grad_row_weights, "grad_row_weights", torch.float32, (rows,), (1,), dev)
    args = [
        rows, n,
        _ptr(grad_out, "grad_out", B.BF16, None, dev),
        _ptr(h0, "h0", B.BF16, rows * 2 * n, dev, required=False),
        _ptr(codes, "codes", I8, rows * 2 * n, dev, required=False),
        _ptr(scales, "scales", B.F32, rows * 2 * ((n + 127) // 128), dev, required=False),
        _ptr(row_weights, "row_weights", B.F32, rows, dev, required=False),
        ctypes.byref(shape) if shape is not None else None,
        _ptr(expert_offsets, "expert_offsets", B.I32, shape.num_experts + 1 if shape is not None else None, dev,
             required=False),
        grad_h0_p, out_p, grad_w_p, None,
    ]
    return ExpertsCall(_lib().moe_swiglu_grad, args, "swiglu_grad",
                       (grad_out, h0, codes, scales, row_weights, shape, expert_offsets),
                       SwigluGrad(grad_h0, out, grad_row_weights), dev)


def swiglu_grad(grad_out, h0=None, codes=None, scales=None, row_weights=None, shape=None, expert_offsets=None,
                grad_h0=None, out=None, grad_row_weights=None, need_out=True, stream=None):
    """moe_swiglu_grad: the gradients of swiglu() for the gradient grad_out [rows, features] of its result, from h0 or
    from its checkpoint (codes and scales).
    Returns a SwigluGrad: grad_h0 (bfloat16 [rows, 2 * features]), out (the forward's result again, for the second
    product's weight gradient; None with need_out=False), grad_row_weights (float32 [rows]; None without row_weights).
    Rows of no expert are left as they were."""
    return B.call_on(stream, prepare_swiglu_grad, grad_out, h0, codes, scales, row_weights, shape, expert_offsets,
                     grad_h0, out, grad_row_weights, need_out)


CombineGrad = namedtuple("CombineGrad", ["grad_expert_out", "grad_topk_weights", "grad_ori_x", "grad_alpha1",
                                         "grad_alpha2", "grad_v"])


def prepare_combine_grad(shape, grad_out, expert_out, topk_idx, topk_weights, dst_row, x_active_mask=None, ori_x=None,
                         const_alpha1=None, const_alpha2=None, const_v=None, grad_expert_out=None, rows=None):
    """Checked, marshalled moe_combine_grad call; see combine_grad()."""
    st = B.check_shape(shape)
    if st != B.MOE_OK:
        raise B.MoeGetError("combine_grad", st)
    dev = _device_of(grad_out, "grad_out")
    T, H, K, kc = shape.num_tokens, shape.hidden, shape.topk, shape.const_expert_num
    special = shape.copy_expert_num + kc > 0
    rows = T * K if rows is None else int(rows)
    f32 = dict(dtype=torch.float32, device=dev)
    if grad_expert_out is None:
        grad_expert_out = torch.empty((rows, H), dtype=torch.bfloat16, device=dev)
    r = CombineGrad(
        grad_expert_out, torch.empty((T, K), **f32),
        torch.empty((T, H), dtype=torch.bfloat16, device=dev) if special else None,
        *(torch.empty((kc, H), **f32) if kc > 0 else None for _ in range(3)))
    some = T > 0
    args = [
        ctypes.byref(shape),
        _ptr(grad_out, "grad_out", B.BF16, T * H, dev),
        _ptr(expert_out, "expert_out", B.BF16, rows * H, dev, required=some),
        _ptr(topk_idx, "topk_idx", B.I32, T * K, dev),
        _ptr(topk_weights, "topk_weights", B.F32, T * K, dev),
        _ptr(x_active_mask, "x_active_mask", B.U8, T, dev, required=False),
        _ptr(dst_row, "dst_row", B.I32, T * K, dev),
        _ptr(ori_x, "ori_x", B.BF16, T * H, dev, required=special and some),
        _ptr(const_alpha1, "const_alpha1", B.BF16, kc * H, dev, required=kc > 0),
        _ptr(const_alpha2, "const_alpha2", B.BF16, kc * H, dev, required=kc > 0),
        _ptr(const_v, "const_v", B.BF16, kc * H, dev, required=kc > 0),
        _ptr(grad_expert_out, "grad_expert_out", B.BF16, rows * H, dev),
        *(_ptr(t, n, (t.dtype,) if t is not None else (), None, dev, required=False)
          for n, t in zip(CombineGrad._fields[1:], r[1:])),
        None,
    ]
    if not some and kc == 0:  # nothing to write
        return ExpertsCall(lambda *_: B.MOE_OK, [None], "combine_grad", (shape,), r, dev)
    return ExpertsCall(_lib().moe_combine_grad, args, "combine_grad",
                       (shape, grad_out, expert_out, topk_idx, topk_weights, dst_row, x_active_mask, ori_x,
                        const_alpha1, const_alpha2, const_v), r, dev)


def combine_grad(shape, grad_out, expert_out, topk_idx, topk_weights, dst_row, x_active_mask=None, ori_x=None,
                 const_alpha1=None, const_alpha2=None, const_v=None, grad_expert_out=None, rows=None, stream=None):
    """moe_combine_grad: the gradients of combine() for the gradient grad_out [T, H] of its result.
    Returns a CombineGrad: grad_expert_out (bfloat16, rows as expert_out; rows that hold no copy are
    left as they were), grad_topk_weights (float32 [T, K]), grad_ori_x (bfloat16 [T, H]; None without
    copy and constant experts), grad_alpha1 / grad_alpha2 / grad_v (float32 [Kc, H]; None without
    constant experts).  `rows` as for combine().  The gradient of a bf16 dispatch is
    combine(shape, grad_expand_x, topk_idx, ones, dst_row), without special experts in the shape and
    with -1 for their slots in topk_idx."""
    return B.call_on(stream, prepare_combine_grad, shape, grad_out, expert_out, topk_idx, topk_weights, dst_row,
                     x_active_mask, ori_x, const_alpha1, const_alpha2, const_v, grad_expert_out, rows)
