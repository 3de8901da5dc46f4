"""ctypes binding of the expert stage of libmoe_get (include/moe_get.h): products grouped by
expert, their gradients, row quantization and the combine's gradient.

As in binding.py: argument checks and marshalling only, outputs allocated with PyTorch unless
given, every step in the HIP kernels, no CPU fallback.  All tensors of a call must be on one
device; the call runs on that device's current stream (or the given one of that device),
whichever device is current.  With `stream=` arguments and results may be dropped at once (binding.call_on);
a prepare_* call makes its results in the memory of the stream that is current then, keeps its tensors
alive itself, and is to be kept until what it issued on other streams is done.
"""
import ctypes
from collections import namedtuple

import torch

from . import binding as B

ROWS_BF16, ROWS_INT8, ROWS_MXFP4 = 0, 1, 2
ACT_NONE, ACT_SWIGLU = 0, 1
EXPERTS_FORWARD, EXPERTS_DGRAD, EXPERTS_WGRAD = 0, 1, 2

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
        if stream is not None and stream.device != self._device:
            raise ValueError(f"{self._what}: the stream is on {stream.device}, the tensors on {self._device}")
        if torch.cuda.current_device() != self._device.index:
            with torch.cuda.device(self._device):
                return self._run(stream)
        return self._run(stream)

    def _run(self, stream):
        s = torch.cuda.current_stream(self._device) if stream is None else stream
        self._args[-1] = s.cuda_stream
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
