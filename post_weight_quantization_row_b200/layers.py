"""Operators that run a model's layers with the solved weights and judge its
answers: linear, layer norm (both with their gradients), log probabilities of
given tokens, and distillation from a teacher's top logits.

As in the rest of the package every call is a kernel of libmpq.so (the formulas
and limits stand in include/mpq.h); this module checks arguments, allocates
outputs and scratch on the inputs' device and passes the current stream of that
device.  The calls neither synchronise nor keep anything, and can be captured
into CUDA graphs.  Gradients are functions of their own: nothing here takes
part in autograd, and a forward call whose inputs require a gradient outside
torch.no_grad() warns that its results do not carry it.

Tensors of any rank count as rows of their last dimension, which must be
contiguous; the rows must lie at one distance from each other (any slice
`a[..., :n]` of a contiguous tensor does, whatever its alignment).
"""
from __future__ import annotations

import ctypes as C
import math
import warnings
from typing import Optional

import torch

from ._lib import check, lib

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
TOP_MAX = 128
DZ_ROUNDED = 0x100


def _rows(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None):
    """(rows, columns, row stride) of a tensor seen as rows of its last dimension."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}, got {t.device}")
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one dimension")
    shape, stride = t.shape, t.stride()
    n = shape[-1]
    if n > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if len(shape) == 2:
        return shape[0], n, stride[0] if shape[0] > 1 else max(n, 1)
    rows, ld = 1, max(n, 1)
    for size, st in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if size == 1:
            continue
        if rows == 1:
            ld = st
        elif st != ld * rows and rows * size:
            raise ValueError(f"{name}: the rows must lie at one distance from each other")
        rows *= size
    return rows, n, ld


def _param(t: Optional[torch.Tensor], n: int, like: torch.Tensor, name: str):
    """Pointer of a parameter vector of n values in `like`'s type or float32."""
    if t is None:
        return None
    if not t.is_cuda or t.device != like.device:
        raise ValueError(f"{name} must be a CUDA tensor on {like.device}")
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
    if t.dtype != like.dtype and t.dtype != torch.float32:
        raise ValueError(f"{name} must be {like.dtype} or torch.float32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _vector(t: torch.Tensor, dtype, shape, like: torch.Tensor, name: str):
    if not t.is_cuda or t.device != like.device:
        raise ValueError(f"{name} must be a CUDA tensor on {like.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _detached(name: str, *inputs):
    """Warns where autograd would expect a gradient that no result carries."""
    for t in inputs:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            warnings.warn(f"{name} takes no part in autograd: no gradient will reach its inputs by backward().  Use the "
                          "gradients that the package computes, and torch.no_grad() around this call.", stacklevel=3)
            return


def _act(name: str) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"unknown activation {name!r}; one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[name]


# The current stream's handle: torch's direct accessor (0.1 us) where it has
# one, else through a Stream object (3 us, half of a small call's time).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, where: str, device: torch.device, *args):
    """One library call on `device` and its current stream."""
    index = device.index
    if index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    if st:
        check(st, where)


def _scratch(nbytes: int, like: torch.Tensor):
    """Scratch on a 256-byte boundary (from the stream's own allocator)."""
    if nbytes == 0:
        return None, None
    t = like.new_empty(nbytes + 256, dtype=torch.uint8)
    return t, (t.data_ptr() + 255) // 256 * 256


def _half_operand(t: torch.Tensor, name: str):
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype} "
                         "(cast the solved weights once: w_hat.to(torch.bfloat16))")


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
           residual: Optional[torch.Tensor] = None, activation: str = "none", out_dtype=None,
           preact: bool = False):
    """act(x weight^T + bias) + residual.

    x: (..., k), weight: (n, k) as a solve gives it, both bfloat16 or float16;
    bias: (n,); residual: (..., n) of the output's type.  out_dtype: x's type
    (default) or torch.float32, which Gram.accumulate takes.  With preact=True
    the result is (y, z), z = x weight^T + bias in x's type for
    linear_backward.
    """
    act = _act(activation)
    _detached("linear", x, weight, bias, residual)
    _half_operand(x, "x")
    rows, k, ldx = _rows(x, "x")
    if weight.dim() != 2 or weight.dtype != x.dtype:
        raise ValueError(f"weight must be a 2-D tensor of {x.dtype}, got {weight.dim()}-D {weight.dtype}")
    n, kw, ldw = _rows(weight, "weight", x)
    if kw != k or k < 1 or n < 1:
        raise ValueError(f"x has {k} columns, weight is {n} x {kw}")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype != x.dtype and out_dtype != torch.float32:
        raise ValueError(f"out_dtype must be {x.dtype} or torch.float32, got {out_dtype}")
    pb = _param(bias, n, x, "bias")
    shape = (*x.shape[:-1], n)
    pr, ldr = None, 0
    if residual is not None:
        if residual.dtype != out_dtype or residual.shape != shape:
            raise ValueError(f"residual must be {out_dtype} of shape {tuple(shape)}, "
                             f"got {residual.dtype} {tuple(residual.shape)}")
        _, _, ldr = _rows(residual, "residual", x)
        pr = residual.data_ptr()
    y = x.new_empty(shape, dtype=out_dtype)
    z = x.new_empty(shape) if preact else None
    if rows > 0:
        px, pw = x.data_ptr(), weight.data_ptr()
        nbytes = 0  # (as the library says where nothing is unaligned, without asking it)
        if (px | pw) & 15 or (ldx | ldw) & 7 or ldx < k or ldw < k:
            nbytes = lib.mpq_linear_workspace_bytes(px, ldx, pw, ldw, rows, n, k)
        keep, ws = _scratch(nbytes, x)
        _call(lib.mpq_linear, "mpq_linear", x.device, px, ldx, pw, ldw, rows, n, k, DTYPES[x.dtype], pb,
              DTYPES[bias.dtype] if bias is not None else 0, act, pr, ldr,
              z.data_ptr() if preact else None, y.data_ptr(), DTYPES[out_dtype], ws, nbytes)
    return (y, z) if preact else y


def linear_backward(dy: torch.Tensor, x: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                    preact: Optional[torch.Tensor] = None, activation: str = "none", dx: bool = True,
                    dweight: bool = True, dbias: bool = True, bias_dtype=None, round_dz: bool = False) -> dict:
    """Gradients of linear: {"dx", "dweight", "dbias"}, those that are asked for.

    dy: (..., n) and preact: (..., n) as linear returned it (only for an
    activation).  x may be None without dweight (frozen weights), weight
    without dx.  dbias has bias_dtype: dy's type (default) or torch.float32.
    The residual's gradient is dy itself.

    dz = dy act'(z) of gelu, gelu_tanh and silu enters the products in two parts
    of dy's type, to 2^-16 of a value or better; round_dz=True rounds it to that
    type once (as 16-bit training mostly does), for half the products' time.
    """
    act = _act(activation)
    _half_operand(dy, "dy")
    rows, n, ldy = _rows(dy, "dy")
    if n < 1:
        raise ValueError("dy has no columns")
    if (dx and weight is None) or (dweight and x is None):
        raise ValueError("dx needs weight, dweight needs x")
    k, px, ldx, pw, ldw, pz, ldz = 1, None, 0, None, 0, None, 0
    if dx:
        if weight.dim() != 2 or weight.dtype != dy.dtype or weight.shape[0] != n or weight.shape[1] < 1:
            raise ValueError(f"weight must be {dy.dtype} of shape ({n}, k)")
        _, k, ldw = _rows(weight, "weight", dy)
        pw = weight.data_ptr()
    if dweight:
        if x.dtype != dy.dtype or x.dim() < 1 or x.shape[:-1] != dy.shape[:-1] or x.shape[-1] < 1:
            raise ValueError(f"x must be {dy.dtype} of shape {(*dy.shape[:-1], 'k')}, got {x.dtype} {tuple(x.shape)}")
        _, kx, ldx = _rows(x, "x", dy)
        if dx and kx != k:
            raise ValueError(f"x has {kx} columns, weight has {k}")
        k, px = kx, x.data_ptr()
    if act:
        if preact is None:
            raise ValueError("an activation's gradient needs preact")
        if preact.dtype != dy.dtype or preact.shape != dy.shape:
            raise ValueError(f"preact must be {dy.dtype} of shape {tuple(dy.shape)}")
        _, _, ldz = _rows(preact, "preact", dy)
        pz = preact.data_ptr()
    bias_dtype = dy.dtype if bias_dtype is None else bias_dtype
    if bias_dtype != dy.dtype and bias_dtype != torch.float32:
        raise ValueError(f"bias_dtype must be {dy.dtype} or torch.float32, got {bias_dtype}")
    if round_dz:
        act |= DZ_ROUNDED
    out = {}
    if dx:
        out["dx"] = dy.new_empty((*dy.shape[:-1], k))
    if dweight:
        out["dweight"] = dy.new_empty((n, k))
    if dbias:
        out["dbias"] = dy.new_empty((n,), dtype=bias_dtype)
    if out:
        py = dy.data_ptr()
        nbytes = lib.mpq_linear_backward_workspace_bytes(py, ldy, px, ldx, pw, ldw, rows, n, k, act, dx, dweight, dbias)
        keep, ws = _scratch(nbytes, dy)
        _call(lib.mpq_linear_backward, "mpq_linear_backward", dy.device, py, ldy, px, ldx, pw, ldw, pz, ldz,
              rows, n, k, DTYPES[dy.dtype], act, *(out[i].data_ptr() if i in out else None
                                                   for i in ("dx", "dweight", "dbias")),
              DTYPES[bias_dtype], ws, nbytes)
    return out


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, stats: bool = False):
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dimension.

    x: (..., n) float32, bfloat16 or float16; weight, bias: (n,), both of x's
    type or both float32.  With stats=True the result is (y, mean, rstd), the
    statistics in float32 of x's leading shape, for layer_norm_backward.
    """
    if x.dtype not in DTYPES:
        raise ValueError(f"x must be float32, bfloat16 or float16, got {x.dtype}")
    _detached("layer_norm", x, weight, bias)
    rows, n, ldx = _rows(x, "x")
    if n < 1:
        raise ValueError("x has no columns")
    pw, pb = _param(weight, n, x, "weight"), _param(bias, n, x, "bias")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have the same type")
    pt = weight.dtype if weight is not None else bias.dtype if bias is not None else x.dtype
    if not eps > 0.0 or not math.isfinite(eps):
        raise ValueError("eps must be > 0")
    y = x.new_empty(x.shape)
    mean = rstd = None
    if stats:
        mean, rstd = x.new_empty((2, *x.shape[:-1]), dtype=torch.float32).unbind(0)
    if rows > 0:
        _call(lib.mpq_layer_norm, "mpq_layer_norm", x.device, x.data_ptr(), ldx, rows, n, DTYPES[x.dtype], pw, pb,
              DTYPES[pt], eps, y.data_ptr(), mean.data_ptr() if stats else None, rstd.data_ptr() if stats else None)
    return (y, mean, rstd) if stats else y


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, dx: bool = True, dweight: bool = True,
                        dbias: bool = True, param_dtype=None) -> dict:
    """Gradients of layer_norm: {"dx", "dweight", "dbias"}, those asked for.

    mean, rstd: as layer_norm returned them.  dweight and dbias have the
    weight's type (param_dtype where there is no weight, default x's type).
    """
    if x.dtype not in DTYPES:
        raise ValueError(f"x must be float32, bfloat16 or float16, got {x.dtype}")
    rows, n, ldx = _rows(x, "x")
    if n < 1:
        raise ValueError("x has no columns")
    if dy.dtype != x.dtype or dy.shape != x.shape:
        raise ValueError(f"dy must be {x.dtype} of shape {tuple(x.shape)}")
    _, _, ldy = _rows(dy, "dy", x)
    pm = _vector(mean, torch.float32, x.shape[:-1], x, "mean")
    pr = _vector(rstd, torch.float32, x.shape[:-1], x, "rstd")
    pw = _param(weight, n, x, "weight")
    pt = weight.dtype if weight is not None else x.dtype if param_dtype is None else param_dtype
    if (pt != x.dtype and pt != torch.float32) or (param_dtype is not None and pt != param_dtype):
        raise ValueError(f"param_dtype must be the weight's type, or {x.dtype} or torch.float32 without one")
    out = {}
    if dx:
        out["dx"] = x.new_empty(x.shape)
    if dweight:
        out["dweight"] = x.new_empty((n,), dtype=pt)
    if dbias:
        out["dbias"] = x.new_empty((n,), dtype=pt)
    if out:
        nbytes = lib.mpq_layer_norm_backward_workspace_bytes(rows, n, dweight or dbias)
        keep, ws = _scratch(nbytes, x)
        _call(lib.mpq_layer_norm_backward, "mpq_layer_norm_backward", x.device, dy.data_ptr(), ldy, x.data_ptr(),
              ldx, pm, pr, rows, n, DTYPES[x.dtype], pw, DTYPES[pt],
              *(out[i].data_ptr() if i in out else None for i in ("dx", "dweight", "dbias")), ws, nbytes)
    return out


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, top: int = 0,
                   ignore_index: int = -100) -> dict:
    """Log probability of each row's token, entropy, and the top alternatives.

    logits: (..., v) float32, bfloat16 or float16; tokens: int64 of the leading
    shape, or None.  Returns {"logprob" (with tokens), "entropy"} in float32
    and for top > 0 {"top_logprob" (..., top) float32, descending, "top_id"
    int64; equal logits: lowest id first}.  A token equal to ignore_index has
    logprob 0, any other outside [0, v) NaN.
    """
    if logits.dtype not in DTYPES:
        raise ValueError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
    _detached("token_logprobs", logits)
    rows, v, ldl = _rows(logits, "logits")
    if v < 1:
        raise ValueError("logits have no columns")
    if not 0 <= top <= min(v, TOP_MAX):
        raise ValueError(f"top must be in [0, {min(v, TOP_MAX)}], got {top}")
    lead, dev = logits.shape[:-1], logits.device
    out, pt = {}, None
    if tokens is not None:
        pt = _vector(tokens, torch.int64, lead, logits, "tokens")
        out["logprob"] = logits.new_empty(lead, dtype=torch.float32)
    out["entropy"] = logits.new_empty(lead, dtype=torch.float32)
    if top:
        out["top_logprob"] = logits.new_empty((*lead, top), dtype=torch.float32)
        out["top_id"] = logits.new_empty((*lead, top), dtype=torch.int64)
    if rows > 0:
        _call(lib.mpq_token_logprobs, "mpq_token_logprobs", dev, logits.data_ptr(), ldl, rows, v,
              DTYPES[logits.dtype], pt, ignore_index, top,
              out["logprob"].data_ptr() if pt is not None else None, out["entropy"].data_ptr(),
              out["top_logprob"].data_ptr() if top else None, out["top_id"].data_ptr() if top else None)
    return out


def topk_distill(logits: torch.Tensor, top_logits: torch.Tensor, top_ids: torch.Tensor,
                 weight: Optional[torch.Tensor] = None, temperature: float = 1.0, grad: bool = True) -> dict:
    """KL divergence of each row from a teacher's top logits, and its gradient.

    logits: (..., v) of the student, float32, bfloat16 or float16; top_logits
    (float32) and top_ids (int64): (..., top), as token_logprobs gives them for
    the teacher (negative id: padding); weight: float32 of the leading shape.
    Returns {"loss" (float32 per row, unweighted), "dlogits" (with grad): the
    gradient of sum(weight * loss) in the logits' type}.
    """
    if logits.dtype not in DTYPES:
        raise ValueError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
    _detached("topk_distill", logits, top_logits)
    rows, v, ldl = _rows(logits, "logits")
    if v < 1:
        raise ValueError("logits have no columns")
    lead, dev = logits.shape[:-1], logits.device
    top = top_ids.shape[-1] if top_ids.dim() else 0
    if not 1 <= top <= TOP_MAX:
        raise ValueError(f"top_ids must have 1 to {TOP_MAX} entries a row, got {top}")
    pl = _vector(top_logits, torch.float32, (*lead, top), logits, "top_logits")
    pi = _vector(top_ids, torch.int64, (*lead, top), logits, "top_ids")
    pw = None if weight is None else _vector(weight, torch.float32, lead, logits, "weight")
    if not 1e-3 <= temperature <= 1e3:
        raise ValueError(f"temperature must be in [0.001, 1000], got {temperature}")
    out = {"loss": logits.new_empty(lead, dtype=torch.float32)}
    if grad:
        out["dlogits"] = logits.new_empty(logits.shape)
    if rows > 0:
        _call(lib.mpq_topk_distill, "mpq_topk_distill", dev, logits.data_ptr(), ldl, rows, v, DTYPES[logits.dtype],
              pl, pi, top, pw, temperature, out["loss"].data_ptr(), out["dlogits"].data_ptr() if grad else None)
    return out


def ops_status(device=None):
    """Synchronise the current stream; raise MPQError if a kernel of these
    operators ran out of a bounded wait, on any stream of the device, since this
    thread's last call."""
    with torch.cuda.device(device):
        check(lib.mpq_ops_status(torch.cuda.current_stream().cuda_stream), "mpq_ops_status")
