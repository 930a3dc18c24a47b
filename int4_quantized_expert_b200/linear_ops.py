"""bf16 matrix products around and inside the MoE layer, with their gradients:
a projection with bias, activation and residual (``linear``), one product per
expert on rows sorted by expert (``grouped_linear``) and the step between an
expert's two products (``swiglu``).

As in the rest of the package, the functions only check and marshal arguments
into the C ABI (``include/moe_linear.h``).  They run on the device of their
tensors, on ``stream`` or that device's current stream, and allocate what they
return (and nothing else, except ``linear_backward``'s dz) on that stream.
``linear_device_status`` reports what the kernels found wrong.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import DTYPE_BF16, DTYPE_FP32, _check, lib

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = range(4)
_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}


@contextlib.contextmanager
def _on(dev: torch.device, stream):
    """``dev`` current and ``stream`` (or dev's current stream) current on it; yields its handle."""
    if stream is not None and stream.device != dev:
        raise ValueError("the stream belongs to %s, the tensors are on %s" % (stream.device, dev))
    if stream is not None:
        with torch.cuda.stream(stream):   # makes dev current too
            yield stream.cuda_stream
    elif dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            yield torch.cuda.current_stream().cuda_stream
    else:
        yield torch.cuda.current_stream().cuda_stream


def _tensor(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, dev: torch.device) -> Optional[int]:
    """The address of ``t`` after checking it (None for an empty tensor)."""
    if tuple(t.shape) != shape or t.dtype != dtype:
        raise ValueError("%s must be %s %s, not %s %s" % (name, dtype, list(shape), t.dtype, list(t.shape)))
    if t.device != dev:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, dev))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr() or None


def _matrix(name: str, t: torch.Tensor, dims: int = 2) -> tuple:
    if t.dim() != dims:
        raise ValueError("%s must be a %d-D tensor" % (name, dims))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return tuple(t.shape)


def _dtype(dtype: torch.dtype) -> int:
    if dtype not in _DTYPES:
        raise ValueError("the output type must be torch.bfloat16 or torch.float32")
    return _DTYPES[dtype]


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, *, activation: int = ACT_NONE,
           residual: Optional[torch.Tensor] = None, save_preact: bool = False, out: Optional[torch.Tensor] = None,
           stream=None):
    """``y = act(x w^T + bias) + residual`` for bf16 ``x[T, K]``, ``w[N, K]``, ``bias[N]``,
    ``residual[T, N]`` (see ``moe_linear_forward``).  ``out`` may be the residual itself.  With
    ``save_preact`` the result is ``(y, z)``, z the rounded pre-activations ``linear_backward`` takes."""
    (T, K), (N, _) = _matrix("x", x), _matrix("w", w)
    dev, bf = x.device, torch.bfloat16
    px, pw = _tensor("x", x, (T, K), bf, dev), _tensor("w", w, (N, K), bf, dev)
    pb = None if bias is None else _tensor("bias", bias, (N,), bf, dev)
    pr = None if residual is None else _tensor("residual", residual, (T, N), bf, dev)
    with _on(dev, stream) as st:
        if out is None:
            out = torch.empty(T, N, dtype=bf, device=dev)
        z = torch.empty(T, N, dtype=bf, device=dev) if save_preact else None
        _check("moe_linear_forward", lib().moe_linear_forward(
            px, T, K, pw, N, pb, activation, pr, None if z is None else z.data_ptr() or None,
            _tensor("out", out, (T, N), bf, dev), st))
    return (out, z) if save_preact else out


def linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, *, activation: int = ACT_NONE,
                    preact: Optional[torch.Tensor] = None, need_dx: bool = True, need_dw: bool = True,
                    need_dbias: bool = False, grad_dtype: torch.dtype = torch.bfloat16, stream=None):
    """``(dx, dw, dbias)`` of ``linear`` from ``dy[T, N]`` (see ``moe_linear_backward``); None in the
    place of a gradient that is not wanted.  ``preact`` is the z that ``linear(save_preact=True)``
    returned (not needed without an activation); ``grad_dtype`` is the type of dw and dbias.  The
    residual's gradient is ``dy``."""
    (T, K), (N, _) = _matrix("x", x), _matrix("w", w)
    dev, bf, gt = x.device, torch.bfloat16, _dtype(grad_dtype)
    px, pw = _tensor("x", x, (T, K), bf, dev), _tensor("w", w, (N, K), bf, dev)
    pdy = _tensor("dy", dy, (T, N), bf, dev)
    pz = None
    if activation != ACT_NONE:
        if preact is None:
            raise ValueError("an activation's gradient needs preact")
        pz = _tensor("preact", preact, (T, N), bf, dev)
    with _on(dev, stream) as st:
        dz = torch.empty(T, N, dtype=bf, device=dev) if activation != ACT_NONE and (need_dx or need_dw) else None
        dx = torch.empty(T, K, dtype=bf, device=dev) if need_dx else None
        dw = torch.empty(N, K, dtype=grad_dtype, device=dev) if need_dw else None
        db = torch.empty(N, dtype=grad_dtype, device=dev) if need_dbias else None
        _check("moe_linear_backward", lib().moe_linear_backward(
            pdy, px, T, K, pw, N, activation, pz, *(None if t is None else t.data_ptr() or None for t in (dz, dx, dw, db)),
            gt, st))
    return dx, dw, db


def _grouped(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor):
    (n, K), (E, N, _) = _matrix("x", x), _matrix("w", w, 3)
    dev, bf = x.device, torch.bfloat16
    return (n, K, E, N, dev, _tensor("x", x, (n, K), bf, dev), _tensor("w", w, (E, N, K), bf, dev),
            _tensor("offsets", offsets, (E + 1,), torch.int32, dev))


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *,
                   out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """``y[r] = x[r] w[e]^T`` for the rows ``offsets[e] <= r < offsets[e + 1]`` of each expert e: bf16
    ``x[n, K]``, ``w[E, N, K]``, int32 ``offsets[E + 1]`` as ``route`` returns them (see
    ``moe_grouped_linear_forward``).  Rows of no expert are not written."""
    n, K, E, N, dev, px, pw, po = _grouped(x, w, offsets)
    yt = _dtype(out_dtype)
    with _on(dev, stream) as st:
        if out is None:
            out = torch.empty(n, N, dtype=out_dtype, device=dev)
        _check("moe_grouped_linear_forward", lib().moe_grouped_linear_forward(
            px, n, K, pw, E, N, po, _tensor("out", out, (n, N), out_dtype, dev), yt, st))
    return out


def grouped_linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *,
                            need_dx: bool = True, need_dw: bool = True,
                            grad_dtype: torch.dtype = torch.bfloat16, dx: Optional[torch.Tensor] = None, stream=None):
    """``(dx, dw)`` of ``grouped_linear`` from bf16 ``dy[n, N]`` (see ``moe_grouped_linear_backward``);
    None in the place of a gradient that is not wanted.  ``dx`` may be given to be written in place
    (rows of no expert are not written); dw has ``grad_dtype`` and is zero for empty experts."""
    n, K, E, N, dev, px, pw, po = _grouped(x, w, offsets)
    pdy, gt = _tensor("dy", dy, (n, N), torch.bfloat16, dev), _dtype(grad_dtype)
    pdx = None
    with _on(dev, stream) as st:
        if need_dx:
            if dx is None:
                dx = torch.empty(n, K, dtype=torch.bfloat16, device=dev)
            pdx = _tensor("dx", dx, (n, K), torch.bfloat16, dev)
        dw = torch.empty(E, N, K, dtype=grad_dtype, device=dev) if need_dw else None
        _check("moe_grouped_linear_backward", lib().moe_grouped_linear_backward(
            pdy, px, n, K, pw, E, N, po, pdx, None if dw is None else dw.data_ptr(), gt, st))
    return (dx if need_dx else None), dw


def swiglu(gu: torch.Tensor, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``h = silu(g) u`` for bf16 rows ``gu[n, 2F] = [g | u]`` (see ``moe_swiglu_forward``)."""
    n, F2 = _matrix("gu", gu)
    dev, bf = gu.device, torch.bfloat16
    pgu = _tensor("gu", gu, (n, 2 * (F2 // 2)), bf, dev)
    with _on(dev, stream) as st:
        if out is None:
            out = torch.empty(n, F2 // 2, dtype=bf, device=dev)
        _check("moe_swiglu_forward", lib().moe_swiglu_forward(
            pgu, n, F2 // 2, _tensor("out", out, (n, F2 // 2), bf, dev), st))
    return out


def swiglu_backward(dh: torch.Tensor, gu: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """``dgu = [dg | du]`` of ``swiglu`` from bf16 ``dh[n, F]`` (see ``moe_swiglu_backward``)."""
    n, F2 = _matrix("gu", gu)
    dev, bf = gu.device, torch.bfloat16
    pgu = _tensor("gu", gu, (n, 2 * (F2 // 2)), bf, dev)
    pdh = _tensor("dh", dh, (n, F2 // 2), bf, dev)
    with _on(dev, stream) as st:
        if out is None:
            out = torch.empty_like(gu)
        _check("moe_swiglu_backward", lib().moe_swiglu_backward(
            pdh, pgu, n, F2 // 2, _tensor("out", out, (n, F2), bf, dev), st))
    return out


def linear_device_status(stream=None) -> int:
    """Synchronizes the stream; a ``Status`` for all calls of ``linear``, ``grouped_linear`` and their
    backward passes on the current device (or the stream's) since the last query, which this clears."""
    dev = torch.device("cuda", torch.cuda.current_device()) if stream is None else stream.device
    with _on(dev, stream) as st:
        return lib().moe_linear_device_status(st)
