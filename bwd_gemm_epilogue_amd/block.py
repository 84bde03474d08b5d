"""Binding of include/swiglu_block.h: the operators around the SwiGLU MLP step
in a block that trains or serves it.  As in the rest of the package every
function marshals arguments only; the arithmetic runs in the HIP kernels and
there is no CPU path."""
from __future__ import annotations

import torch

from . import _check, _launches, _on_gpu, _stream, _ws, lib

__all__ = [
    "swiglu_layer_norm_fwd", "swiglu_layer_norm_bwd", "swiglu_layer_norm_bwd_workspace",
    "SwiGLULayerNormFunction", "swiglu_layer_norm",
]

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _typed(t, name: str, shape, dtype: torch.dtype) -> int:
    """The address of a contiguous tensor of this shape and type."""
    _on_gpu(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name: str, shape, dtype: torch.dtype):
    """(address, row stride in elements) of a matrix whose rows are dense."""
    _on_gpu(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    M, D = shape
    if D > 1 and M > 0 and t.stride(1) != 1:
        raise ValueError(f"{name} must have dense rows (last stride 1)")
    ld = t.stride(0) if M > 1 else D
    if ld < D:
        raise ValueError(f"{name}'s rows overlap (row stride {ld} < {D})")
    return t.data_ptr(), ld


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------

def _norm_vectors(D, x, **vectors):
    """(type of weight and bias, their addresses or None)."""
    given = [v for v in vectors.values() if v is not None]
    wt = given[0].dtype if given else x.dtype
    if wt not in (x.dtype, torch.float32):
        raise ValueError(f"weight and bias must be {x.dtype} or float32, got {wt}")
    return wt, [None if v is None else _typed(v, n, (D,), wt) for n, v in vectors.items()]


@_launches
def swiglu_layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, y=None, mean=None, rstd=None, stream=None):
    """y = (x - mean) rstd weight + bias over the last dimension of x [M,D]
    (dense rows, any row stride): returns (y, mean, rstd), the statistics
    float32 [M]."""
    if x.dim() != 2:
        raise ValueError(f"x must have two dimensions, got {tuple(x.shape)}")
    M, D = x.shape
    xp, ldx = _rows(x, "x", (M, D), x.dtype)
    code = _dtype(x, "x")
    wt, (wp, bp) = _norm_vectors(D, x, weight=weight, bias=bias)
    y = torch.empty((M, D), dtype=x.dtype, device=x.device) if y is None else y
    stats = None
    if mean is None and rstd is None:
        stats = torch.empty((2, M), dtype=torch.float32, device=x.device)
    mean = (torch.empty(M, dtype=torch.float32, device=x.device) if stats is None else stats[0]) if mean is None else mean
    rstd = (torch.empty(M, dtype=torch.float32, device=x.device) if stats is None else stats[1]) if rstd is None else rstd
    yp, ldy = _rows(y, "y", (M, D), x.dtype)
    _check("swiglu_layer_norm_fwd", lib().swiglu_layer_norm_fwd(
        xp, ldx, wp, bp, yp, ldy, _typed(mean, "mean", (M,), torch.float32),
        _typed(rstd, "rstd", (M,), torch.float32), M, D, eps, code, _DTYPES[wt], _stream(x, stream)))
    return y, mean, rstd


def swiglu_layer_norm_bwd_workspace(M, D) -> int:
    return lib().swiglu_layer_norm_bwd_workspace(M, D)


@_launches
def swiglu_layer_norm_bwd(dy, x, weight, mean, rstd, dres=None, bias_grad=True, dx=None, dweight=None, dbias=None,
                          ws=None, stream=None):
    """Backward of swiglu_layer_norm_fwd: (dx, dweight, dbias).  dres [M,D] is
    added to dx (the gradient that reaches x by a residual branch).  dweight
    is None where weight is; dbias is None unless bias_grad (its type is the
    weight's, or x's where there is none)."""
    if x.dim() != 2:
        raise ValueError(f"x must have two dimensions, got {tuple(x.shape)}")
    M, D = x.shape
    code = _dtype(x, "x")
    dyp, lddy = _rows(dy, "dy", (M, D), x.dtype)
    xp, ldx = _rows(x, "x", (M, D), x.dtype)
    rp, ldr = (None, D) if dres is None else _rows(dres, "dres", (M, D), x.dtype)
    if weight is not None and dweight is None:
        dweight = torch.empty(D, dtype=weight.dtype, device=x.device)
    if bias_grad and dbias is None:
        dbias = torch.empty(D, dtype=x.dtype if weight is None else weight.dtype, device=x.device)
    wt, (wp, dwp, dbp) = _norm_vectors(D, x, weight=weight, dweight=dweight, dbias=dbias)
    dx = torch.empty((M, D), dtype=x.dtype, device=x.device) if dx is None else dx
    dxp, lddx = _rows(dx, "dx", (M, D), x.dtype)
    ws = _ws(swiglu_layer_norm_bwd_workspace(M, D) if dwp or dbp else 0, x, ws)
    _check("swiglu_layer_norm_bwd", lib().swiglu_layer_norm_bwd(
        dyp, lddy, xp, ldx, wp, _typed(mean, "mean", (M,), torch.float32), _typed(rstd, "rstd", (M,), torch.float32),
        rp, ldr, dxp, lddx, dwp, dbp, ws.data_ptr(), ws.numel() * ws.element_size(), M, D, code, _DTYPES[wt],
        _stream(x, stream)))
    return dx, dweight, dbias


def _as_rows(t: torch.Tensor) -> torch.Tensor:
    """t as a matrix of its last dimension with dense, separate rows: a view
    where its layout allows, else a copy."""
    t = t.reshape(-1, t.shape[-1])
    M, D = t.shape
    dense = (D <= 1 or t.stride(1) == 1) and (M <= 1 or t.stride(0) >= D)
    return t if dense else t.contiguous()


class SwiGLULayerNormFunction(torch.autograd.Function):
    """Layer norm over the last dimension; saves {x, weight, mean, rstd}."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x2 = _as_rows(x)
        y, mean, rstd = swiglu_layer_norm_fwd(x2, weight, bias, eps)
        ctx.save_for_backward(x2, weight, mean, rstd)
        ctx.bias_type = None if bias is None else bias.dtype
        ctx.shape = x.shape
        return y.reshape(x.shape)

    @staticmethod
    def backward(ctx, grad_y):
        x2, weight, mean, rstd = ctx.saved_tensors
        _, need_w, need_b, _ = ctx.needs_input_grad
        dbias = torch.empty(x2.shape[1], dtype=ctx.bias_type, device=x2.device) if need_b else None
        dx, dw, db = swiglu_layer_norm_bwd(_as_rows(grad_y), x2, weight, mean, rstd, bias_grad=need_b, dbias=dbias)
        return dx.reshape(ctx.shape), dw if need_w else None, db, None


def swiglu_layer_norm(x, weight=None, bias=None, eps=1e-5):
    return SwiGLULayerNormFunction.apply(x, weight, bias, eps)
