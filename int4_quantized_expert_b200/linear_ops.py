"""bf16 matrix products around and inside the MoE layer, with their gradients:
a projection with bias, activation and residual (``linear``), one product per
expert on rows sorted by expert (``grouped_linear``) and the step between an
expert's two products (``swiglu``).

As in the rest of the package, the functions only check and marshal arguments
into the C ABI (``include/moe_linear.h``).  They run on the device of their
tensors, on ``stream`` or that device's current stream, and allocate what they
return (and nothing else, except ``linear_backward``'s dz) on that stream.
As everywhere in the package, what a call reads has to stay allocated until the
stream is past it, and autograd does not record the calls: the ``*_backward``
functions are the gradients.  ``linear_device_status`` reports what the kernels
found wrong.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import DTYPE_BF16, DTYPE_FP32, MoEError, Status, _check, lib

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = range(4)
_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}


# What the calls of a decode step pay on the host before their kernel starts
# counts as much as the kernel: the checks below read each property of a tensor
# once, and the stream's handle is taken without building a Stream object
# (14.2 -> 8.7 us for a call of linear, of which 3.9 are the library's).  What gives
# it is looked up in a call, whose tensors are on a device already: a torch without
# CUDA does not have it, and the package is imported there too.
_C = torch._C


def _elsewhere(index: int, stream) -> bool:
    """Whether ``stream`` or the device ``index`` of the tensors has to be made current first."""
    return stream is not None or index != _C._cuda_getDevice()


@contextlib.contextmanager
def _on(index: int, stream):
    """The device ``index`` current, and ``stream`` (if any) current on it."""
    if stream is None:
        with torch.cuda.device(index):
            yield
    elif stream.device.index != index:
        raise ValueError("the stream belongs to %s, the tensors are on cuda:%d" % (stream.device, index))
    else:
        with torch.cuda.stream(stream):   # makes its device current too
            yield


def _tensor(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, index: int) -> int:
    """The address of ``t`` after checking it (0, the null pointer, for an empty tensor)."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError("%s must be %s %s, not %s %s" % (name, dtype, list(shape), t.dtype, list(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s is on %s, not on cuda:%d" % (name, t.device, index))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _matrix(name: str, t: torch.Tensor, dims: int = 2) -> torch.Size:
    if t.dim() != dims:
        raise ValueError("%s must be a %d-D tensor" % (name, dims))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.shape


def _too_large(fn: str) -> None:
    """What the C ABI answers to sizes out of its range, for those that its 32-bit arguments cannot hold."""
    raise MoEError(fn, Status.UNSUPPORTED_SHAPE)


def _sizes(fn: str, x: torch.Tensor, w: torch.Tensor) -> tuple:
    """(T, K, N, device index) of ``x[T, K]`` and ``w[N, ...]``."""
    if x.dim() != 2 or w.dim() != 2 or not x.is_cuda:
        _matrix("x", x), _matrix("w", w)   # one of them raises
    T, K = x.shape
    N = w.shape[0]
    if (T | K | N) >> 31:
        _too_large(fn)
    return T, K, N, x.get_device()


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
    T, K, N, at = _sizes("moe_linear_forward", x, w)
    bf = torch.bfloat16
    if _elsewhere(at, stream):
        with _on(at, stream):
            return linear(x, w, bias, activation=activation, residual=residual, save_preact=save_preact, out=out)
    px, pw = _tensor("x", x, (T, K), bf, at), _tensor("w", w, (N, K), bf, at)
    pb = None if bias is None else _tensor("bias", bias, (N,), bf, at)
    pr = None if residual is None else _tensor("residual", residual, (T, N), bf, at)
    if out is None:
        out = x.new_empty((T, N))
        pout = out.data_ptr()
    else:
        pout = _tensor("out", out, (T, N), bf, at)
    z = x.new_empty((T, N)) if save_preact else None
    _check("moe_linear_forward", lib().moe_linear_forward(
        px, T, K, pw, N, pb, activation, pr, None if z is None else z.data_ptr(),
        pout, _C._cuda_getCurrentRawStream(at)))
    return (out, z) if save_preact else out


def linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, *, activation: int = ACT_NONE,
                    preact: Optional[torch.Tensor] = None, need_dx: bool = True, need_dw: bool = True,
                    need_dbias: bool = False, grad_dtype: torch.dtype = torch.bfloat16, stream=None):
    """``(dx, dw, dbias)`` of ``linear`` from ``dy[T, N]`` (see ``moe_linear_backward``); None in the
    place of a gradient that is not wanted.  ``preact`` is the z that ``linear(save_preact=True)``
    returned (not needed without an activation); ``grad_dtype`` is the type of dw and dbias.  The
    residual's gradient is ``dy``."""
    T, K, N, at = _sizes("moe_linear_backward", x, w)
    bf, gt = torch.bfloat16, _dtype(grad_dtype)
    if _elsewhere(at, stream):
        with _on(at, stream):
            return linear_backward(dy, x, w, activation=activation, preact=preact, need_dx=need_dx, need_dw=need_dw,
                                   need_dbias=need_dbias, grad_dtype=grad_dtype)
    px, pw = _tensor("x", x, (T, K), bf, at), _tensor("w", w, (N, K), bf, at)
    pdy = _tensor("dy", dy, (T, N), bf, at)
    pz = None
    if activation != ACT_NONE:
        if preact is None:
            raise ValueError("an activation's gradient needs preact")
        pz = _tensor("preact", preact, (T, N), bf, at)
    dz = x.new_empty((T, N)) if activation != ACT_NONE and (need_dx or need_dw) else None
    dx = x.new_empty((T, K)) if need_dx else None
    dw = x.new_empty((N, K), dtype=grad_dtype) if need_dw else None
    db = x.new_empty((N,), dtype=grad_dtype) if need_dbias else None
    _check("moe_linear_backward", lib().moe_linear_backward(
        pdy, px, T, K, pw, N, activation, pz, *(None if t is None else t.data_ptr() for t in (dz, dx, dw, db)), gt,
        _C._cuda_getCurrentRawStream(at)))
    return dx, dw, db


def _grouped(fn: str, x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, at: int):
    (n, K), (E, N, _) = x.shape, w.shape
    if (n | K | E | N) >> 31:
        _too_large(fn)
    return (n, K, E, N, _tensor("x", x, (n, K), torch.bfloat16, at), _tensor("w", w, (E, N, K), torch.bfloat16, at),
            _tensor("offsets", offsets, (E + 1,), torch.int32, at))


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *,
                   out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """``y[r] = x[r] w[e]^T`` for the rows ``offsets[e] <= r < offsets[e + 1]`` of each expert e: bf16
    ``x[n, K]``, ``w[E, N, K]``, int32 ``offsets[E + 1]`` as ``route`` returns them (see
    ``moe_grouped_linear_forward``).  Rows of no expert are not written."""
    _matrix("x", x), _matrix("w", w, 3)
    at, yt = x.get_device(), _dtype(out_dtype)
    if _elsewhere(at, stream):
        with _on(at, stream):
            return grouped_linear(x, w, offsets, out_dtype=out_dtype, out=out)
    n, K, E, N, px, pw, po = _grouped("moe_grouped_linear_forward", x, w, offsets, at)
    if out is None:
        out = x.new_empty((n, N), dtype=out_dtype)
        pout = out.data_ptr()
    else:
        pout = _tensor("out", out, (n, N), out_dtype, at)
    _check("moe_grouped_linear_forward", lib().moe_grouped_linear_forward(
        px, n, K, pw, E, N, po, pout, yt, _C._cuda_getCurrentRawStream(at)))
    return out


def grouped_linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *,
                            need_dx: bool = True, need_dw: bool = True,
                            grad_dtype: torch.dtype = torch.bfloat16, dx: Optional[torch.Tensor] = None, stream=None):
    """``(dx, dw)`` of ``grouped_linear`` from bf16 ``dy[n, N]`` (see ``moe_grouped_linear_backward``);
    None in the place of a gradient that is not wanted.  ``dx`` may be given to be written in place
    (rows of no expert are not written); dw has ``grad_dtype`` and is zero for empty experts."""
    _matrix("x", x), _matrix("w", w, 3)
    at, gt = x.get_device(), _dtype(grad_dtype)
    if _elsewhere(at, stream):
        with _on(at, stream):
            return grouped_linear_backward(dy, x, w, offsets, need_dx=need_dx, need_dw=need_dw, grad_dtype=grad_dtype,
                                           dx=dx)
    n, K, E, N, px, pw, po = _grouped("moe_grouped_linear_backward", x, w, offsets, at)
    pdy, pdx = _tensor("dy", dy, (n, N), torch.bfloat16, at), None
    if need_dx:
        if dx is None:
            dx = x.new_empty((n, K))
        pdx = _tensor("dx", dx, (n, K), torch.bfloat16, at)
    dw = x.new_empty((E, N, K), dtype=grad_dtype) if need_dw else None
    _check("moe_grouped_linear_backward", lib().moe_grouped_linear_backward(
        pdy, px, n, K, pw, E, N, po, pdx, None if dw is None else dw.data_ptr(), gt, _C._cuda_getCurrentRawStream(at)))
    return (dx if need_dx else None), dw


def swiglu(gu: torch.Tensor, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``h = silu(g) u`` for bf16 rows ``gu[n, 2F] = [g | u]`` (see ``moe_swiglu_forward``)."""
    n, F2 = _matrix("gu", gu)
    at, bf, F = gu.get_device(), torch.bfloat16, F2 // 2
    if (n | F) >> 31:
        _too_large("moe_swiglu_forward")
    if _elsewhere(at, stream):
        with _on(at, stream):
            return swiglu(gu, out=out)
    pgu = _tensor("gu", gu, (n, 2 * F), bf, at)
    if out is None:
        out = gu.new_empty((n, F))
        pout = out.data_ptr()
    else:
        pout = _tensor("out", out, (n, F), bf, at)
    _check("moe_swiglu_forward", lib().moe_swiglu_forward(
        pgu, n, F, pout, _C._cuda_getCurrentRawStream(at)))
    return out


def swiglu_backward(dh: torch.Tensor, gu: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """``dgu = [dg | du]`` of ``swiglu`` from bf16 ``dh[n, F]`` (see ``moe_swiglu_backward``)."""
    n, F2 = _matrix("gu", gu)
    at, bf, F = gu.get_device(), torch.bfloat16, F2 // 2
    if (n | F) >> 31:
        _too_large("moe_swiglu_backward")
    if _elsewhere(at, stream):
        with _on(at, stream):
            return swiglu_backward(dh, gu, out=out)
    pgu, pdh = _tensor("gu", gu, (n, 2 * F), bf, at), _tensor("dh", dh, (n, F), bf, at)
    if out is None:
        out = gu.new_empty((n, F2))
        pout = out.data_ptr()
    else:
        pout = _tensor("out", out, (n, F2), bf, at)
    _check("moe_swiglu_backward", lib().moe_swiglu_backward(
        pdh, pgu, n, F, pout, _C._cuda_getCurrentRawStream(at)))
    return out


def linear_device_status(stream=None) -> int:
    """Synchronizes the stream; a ``Status`` for all calls of ``linear``, ``grouped_linear`` and their
    backward passes on the current device (or the stream's) since the last query, which this clears."""
    if stream is None:
        return lib().moe_linear_device_status(torch.cuda.current_stream().cuda_stream)
    with torch.cuda.device(stream.device):
        return lib().moe_linear_device_status(stream.cuda_stream)
