"""Refusals of the linear, grouped linear and SwiGLU entry points: what the C
ABI and the Python functions reject before touching a device."""
import os
import re
import subprocess
import sys

import pytest
import torch

import int4_quantized_expert_b200 as moe
from tests import test_build_resources as resources

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
S = moe.Status
A = [(1 << 24) * (i + 1) for i in range(12)]   # aligned addresses far apart, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from int4_quantized_expert_b200 import build
        build.build()
    return moe.lib()


def test_exports_every_declared_symbol(lib):
    src = open(os.path.join(ROOT, "include", "moe_linear.h")).read()
    names = re.findall(r"MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", src)
    assert len(names) == 7
    for n in names:
        assert hasattr(lib, n), n


def fwd(lib, **kw):
    a = dict(x=A[0], T=4, K=16, w=A[1], N=24, bias=A[2], act=0, residual=A[3], preact=A[4], y=A[5])
    a.update(kw)
    return lib.moe_linear_forward(*a.values(), None)


def test_linear_forward_refusals(lib):
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(K=0), dict(K=12), dict(K=65544), dict(N=4), dict(N=-8)):
        assert fwd(lib, **kw) == S.UNSUPPORTED_SHAPE, kw
    for kw in (dict(act=-1), dict(act=4), dict(x=None), dict(w=None), dict(y=None), dict(x=A[0] + 8), dict(bias=A[2] + 2),
               dict(preact=A[4] + 4), dict(y=A[0]), dict(y=A[3] + 16), dict(preact=A[5]), dict(preact=A[2]),
               dict(y=A[1] + 16)):
        assert fwd(lib, **kw) == S.INVALID_ARG, kw
    assert fwd(lib, T=0, x=None, w=None, y=None, bias=None, residual=None, preact=None) == S.OK


def bwd(lib, **kw):
    a = dict(dy=A[0], x=A[1], T=4, K=16, w=A[2], N=24, act=3, z=A[3], dz=A[4], dx=A[5], dw=A[6], db=A[7], dt=0)
    a.update(kw)
    return lib.moe_linear_backward(*a.values(), None)


def test_linear_backward_refusals(lib):
    for kw in (dict(T=-1), dict(K=20), dict(N=0)):
        assert bwd(lib, **kw) == S.UNSUPPORTED_SHAPE, kw
    for kw in (dict(act=9), dict(dt=2), dict(dy=None), dict(x=None), dict(w=None), dict(z=None), dict(dz=None),
               dict(dx=A[0]), dict(dw=A[5]), dict(dz=A[0]), dict(db=A[6] + 32), dict(dw=A[6] + 8)):
        assert bwd(lib, **kw) == S.INVALID_ARG, kw
    # nothing wanted: nothing needed
    assert bwd(lib, T=0, act=0, dy=None, x=None, w=None, z=None, dz=None, dx=None, dw=None, db=None) == S.OK


def test_grouped_refusals(lib):
    def f(**kw):
        a = dict(x=A[0], n=4, K=16, w=A[1], E=3, N=24, off=A[2], y=A[3], dt=0)
        a.update(kw)
        return lib.moe_grouped_linear_forward(*a.values(), None)

    def b(**kw):
        a = dict(dy=A[0], x=A[1], n=4, K=16, w=A[2], E=3, N=24, off=A[3], dx=A[4], dw=A[5], dt=0)
        a.update(kw)
        return lib.moe_grouped_linear_backward(*a.values(), None)

    for g in (f, b):
        for kw in (dict(n=-1), dict(E=0), dict(E=257), dict(K=9), dict(N=65544)):
            assert g(**kw) == S.UNSUPPORTED_SHAPE, kw
        for kw in (dict(dt=3), dict(off=None), dict(x=None), dict(w=None), dict(off=A[3] + 4)):
            assert g(**kw) == S.INVALID_ARG, kw
    for kw in (dict(y=None), dict(y=A[0]), dict(y=A[2])):
        assert f(**kw) == S.INVALID_ARG, kw
    for kw in (dict(dy=None), dict(dx=A[0]), dict(dw=A[2]), dict(dx=A[5])):
        assert b(**kw) == S.INVALID_ARG, kw
    assert f(n=0, x=None, w=None, y=None) == S.OK
    assert b(n=0, dy=None, x=None, w=None, dx=None, dw=None) == S.OK


def test_swiglu_refusals(lib):
    assert lib.moe_swiglu_forward(A[0], -1, 16, A[1], None) == S.UNSUPPORTED_SHAPE
    assert lib.moe_swiglu_forward(A[0], 4, 12, A[1], None) == S.UNSUPPORTED_SHAPE
    assert lib.moe_swiglu_forward(None, 4, 16, A[1], None) == S.INVALID_ARG
    assert lib.moe_swiglu_forward(A[0], 4, 16, A[0], None) == S.INVALID_ARG
    assert lib.moe_swiglu_forward(None, 0, 16, None, None) == S.OK
    assert lib.moe_swiglu_backward(A[0], A[1], 4, 16, A[0], None) == S.INVALID_ARG
    assert lib.moe_swiglu_backward(A[0], A[1] + 2, 4, 16, A[2], None) == S.INVALID_ARG
    assert lib.moe_swiglu_backward(A[0], A[1], 4, 7, A[2], None) == S.UNSUPPORTED_SHAPE
    assert lib.moe_swiglu_backward(None, None, 0, 8, None, None) == S.OK


def test_python_refuses_what_it_cannot_marshal():
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(24, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.linear(x, w)
    with pytest.raises(ValueError, match="2-D"):
        moe.linear(x[0], w)
    with pytest.raises(ValueError, match="CUDA"):
        moe.linear_backward(x, x, w)
    with pytest.raises(ValueError, match="3-D"):
        moe.grouped_linear(_FakeCuda(x), w, None)
    with pytest.raises(ValueError, match="CUDA"):
        moe.swiglu(x)


class _FakeCuda:
    """A 2-D tensor that says it is on a device: the next check is reached."""

    def __init__(self, t):
        self._t = t
        self.is_cuda = True
        self.shape = t.shape

    def dim(self):
        return self._t.dim()


@pytest.mark.parametrize("src,kernels", [("linear.cu", ["linear_kernel", "act_grad_kernel"]), ("swiglu.cu", ["swiglu_kernel"])])
def test_kernels_do_not_spill(src, kernels, tmp_path, monkeypatch):
    monkeypatch.setitem(resources.HOT, src, kernels)
    resources.test_hot_kernels_do_not_spill(src, tmp_path)


def test_imports_without_cuda_bindings():
    """A torch built without CUDA lacks the functions that give the current device and stream."""
    code = """
import torch
del torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
import int4_quantized_expert_b200 as moe
try:
    moe.linear(torch.zeros(4, 16).bfloat16(), torch.zeros(24, 16).bfloat16())
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError("not refused")
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300, cwd=ROOT)


class _Huge:
    """What the functions ask of a CUDA tensor, with any shape and no memory behind it."""

    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16, index=0, contiguous=True):
        self.shape, self.dtype, self.device, self.contiguous = torch.Size(shape), dtype, torch.device("cuda", index), contiguous

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return A[0]

    def new_empty(self, shape, dtype=None):
        return _Huge(*shape, dtype=dtype or self.dtype)


def test_sizes_that_do_not_fit_the_abi(lib, monkeypatch):
    """Rows or widths of 2^31 and more are refused, not taken modulo 2^32: 2^32 + 5 rows are not five."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0)
    W = 1 << 32
    off = _Huge(3, dtype=torch.int32)
    calls = []
    for t, k, n in ((W + 5, 16, 24), (5, W + 16, 24), (5, 16, W + 24), (1 << 31, 16, 24)):
        x, w, dy = _Huge(t, k), _Huge(n, k), _Huge(t, n)
        xs, ws = _Huge(t, k), _Huge(2, n, k)
        calls += [lambda x=x, w=w: moe.linear(x, w), lambda x=x, w=w, dy=dy: moe.linear_backward(dy, x, w),
                  lambda xs=xs, ws=ws: moe.grouped_linear(xs, ws, off),
                  lambda xs=xs, ws=ws, dy=dy: moe.grouped_linear_backward(dy, xs, ws, off)]
    calls += [lambda: moe.grouped_linear(_Huge(5, 16), _Huge(W + 2, 24, 16), _Huge(W + 3, dtype=torch.int32))]
    for n, f in ((W + 5, 16), (5, W + 16)):
        calls += [lambda n=n, f=f: moe.swiglu(_Huge(n, 2 * f)),
                  lambda n=n, f=f: moe.swiglu_backward(_Huge(n, f), _Huge(n, 2 * f))]
    for call in calls:
        with pytest.raises(moe.MoEError) as e:
            call()
        assert e.value.status == S.UNSUPPORTED_SHAPE


def test_python_refuses_tensors_that_do_not_fit(lib, monkeypatch):
    """Every argument of every function: a wrong shape, type, device or layout, before the library is called."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(moe.linear_ops, "lib", lambda: pytest.fail("the library was called"))
    T, K, N, E, bf = 4, 16, 24, 3, torch.bfloat16
    good = {
        moe.linear: dict(x=(T, K), w=(N, K), bias=(N,), residual=(T, N), out=(T, N)),
        moe.linear_backward: dict(dy=(T, N), x=(T, K), w=(N, K), preact=(T, N)),
        moe.grouped_linear: dict(x=(T, K), w=(E, N, K), offsets=(E + 1,), out=(T, N)),
        moe.grouped_linear_backward: dict(dy=(T, N), x=(T, K), w=(E, N, K), offsets=(E + 1,), dx=(T, K)),
        moe.swiglu: dict(gu=(T, 2 * K), out=(T, K)),
        moe.swiglu_backward: dict(dh=(T, K), gu=(T, 2 * K), out=(T, 2 * K)),
    }
    for fn, shapes in good.items():
        more = dict(activation=moe.ACT_SILU) if fn is moe.linear_backward else {}
        for name, shape in shapes.items():
            dtype = torch.int32 if name == "offsets" else bf
            longer = (shape[0],) * (len(shape) == 2) + (shape[-1] + 8,) if name != "gu" else (shape[0], shape[1] + 1)
            for bad in (_Huge(*longer, dtype=dtype), _Huge(*shape, dtype=torch.float16), _Huge(*shape, 1, dtype=dtype),
                        _Huge(*shape, dtype=torch.int64 if name == "offsets" else torch.float32),
                        _Huge(*shape, dtype=dtype, contiguous=False)):
                args = {k: _Huge(*v, dtype=torch.int32 if k == "offsets" else bf) for k, v in shapes.items()}
                args[name] = bad
                with pytest.raises(ValueError):
                    fn(**args, **more)
            if name != next(iter(shapes)) and not (name in ("x", "gu") and "dy" in shapes or "dh" in shapes):
                args = {k: _Huge(*v, dtype=torch.int32 if k == "offsets" else bf) for k, v in shapes.items()}
                args[name] = _Huge(*shape, dtype=dtype, index=1)
                with pytest.raises(ValueError, match="cuda:1"):
                    fn(**args, **more)


def test_python_refuses_other_arguments(lib, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    x, w, dy, off = _Huge(4, 16), _Huge(24, 16), _Huge(4, 24), _Huge(2, dtype=torch.int32)
    we = _Huge(1, 24, 16)
    with pytest.raises(ValueError, match="preact"):
        moe.linear_backward(dy, x, w, activation=moe.ACT_GELU)
    for call in (lambda t: moe.linear_backward(dy, x, w, grad_dtype=t), lambda t: moe.grouped_linear(x, we, off, out_dtype=t),
                 lambda t: moe.grouped_linear_backward(dy, x, we, off, grad_dtype=t)):
        with pytest.raises(ValueError, match="output type"):
            call(torch.float16)

    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    for call in (lambda: moe.linear(x, w, stream=Stream()), lambda: moe.linear_backward(dy, x, w, stream=Stream()),
                 lambda: moe.grouped_linear(x, we, off, stream=Stream()), lambda: moe.swiglu(x, stream=Stream()),
                 lambda: moe.grouped_linear_backward(dy, x, we, off, stream=Stream()),
                 lambda: moe.swiglu_backward(_Huge(4, 8), x, stream=Stream())):
        with pytest.raises(ValueError, match="the stream belongs to cuda:1"):
            call()
    for bad in (-1, 4):
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0)
        with pytest.raises(moe.MoEError) as e:
            moe.linear(x, w, activation=bad)
        assert e.value.status == S.INVALID_ARG
