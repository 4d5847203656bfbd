"""The training-step operators of libgc.so (include/gc_train.h): 8-bit activation
checkpoints, the MLP activation, layer norm and the weight gradient of a linear layer.

Marshalling only, as in the package's other calls: each function checks its tensors,
allocates the outputs and the workspace that the caller does not pass, and forwards device
pointers and the HIP stream to the C ABI.

Matrices are 2-D tensors with consecutive columns (``stride(1) == 1``) and any row stride.
A checkpoint is a pair of tensors ``(codes, exps)``: int8 [rows, 32 * ceil(cols / 32)] and
uint8 [rows, ceil(cols / 32)], both contiguous.  Outputs that a caller passes may not overlap the inputs or
each other (no call works in place); one that does raises GCError.

``stream``: the torch stream to enqueue on, by default the current one.  With another
stream, what a call allocates belongs to that stream's pool and the tensors passed in are
recorded on it, so that torch does not hand their memory out again while the work is
pending; ordering the streams themselves is the caller's part, as with any torch operation.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import GCError, GC_OK, _lib

__all__ = ["ckpt_pack", "ckpt_unpack", "act_forward", "act_backward", "layernorm_forward", "layernorm_backward",
           "linear_wgrad"]

_p, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_SIGS = {
    "gc_ckpt_pack": [_i32, _p, _i64, _i64, _i64, _p, _p, _p],
    "gc_ckpt_unpack": [_i32, _p, _p, _i64, _i64, _p, _i64, _p],
    "gc_act_forward": [_i32, _i32, _p, _i64, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p],
    "gc_act_backward": [_i32, _i32, _p, _i64, _p, _i64, _p, _p, _i64, _i64, _p, _i64, _p],
    "gc_layernorm_forward": [_i32, _p, _i64, _i64, _i64, _i32, _p, _p, _f32, _p, _i64, _p, _p, _p, _p, _p, _p, _p],
    "gc_layernorm_backward_workspace": [_i64, _i64, ctypes.POINTER(_sz)],
    "gc_layernorm_backward": [_i32, _p, _i64, _p, _i64, _p, _p, _i64, _i64, _i32, _p, _p, _p, _p, _i64, _p, _p, _i32,
                              _p, _sz, _p],
    "gc_linear_wgrad_workspace": [_i32, _i64, _i64, _i64, ctypes.POINTER(_sz)],
    "gc_linear_wgrad": [_i32, _p, _i64, _p, _p, _i64, _i64, _i64, _p, _i64, _p, _i32, _p, _sz, _p],
}
_FN = {}
for _name, _args in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _i32
    _FN[_name] = _fn

_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_KIND = {"gelu": 0, "gelu_tanh": 1, "silu": 2}


def _call(name, *args):
    status = _FN[name](*args)
    if status != GC_OK:
        raise GCError(status, name)


def _kind(kind):
    if kind not in _KIND:
        raise ValueError(f"kind must be one of {', '.join(_KIND)}, got {kind!r}")
    return _KIND[kind]


def _matrix(t, name, dtype=None, shape=None):
    """(pointer, row stride) of a 2-D tensor with consecutive columns."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dtype is None:
        if t.dtype not in _DTYPE:
            raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    elif t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {t.dim()}")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        raise ValueError(f"{name} must have consecutive columns (stride 1), got {s1}")
    if rows <= 1:            # one row: its stride means nothing
        return t.data_ptr(), cols
    if s0 < cols:
        raise ValueError(f"{name}: rows overlap (stride {s0} for {cols} columns)")
    return t.data_ptr(), s0


def _vector(t, name, dtype, n, device):
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {device}")
    return t.data_ptr()


def _on_device(t, name, device):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _ckpt(ckpt, rows, cols, device):
    """Pointers of a checkpoint of a rows x cols matrix."""
    codes, exps = ckpt
    groups = (cols + 31) // 32
    if codes.dtype != torch.int8 or tuple(codes.shape) != (rows, groups * 32) or not codes.is_contiguous():
        raise ValueError(f"codes must be a contiguous int8 tensor {(rows, groups * 32)}, got {codes.dtype} {tuple(codes.shape)}")
    if exps.dtype != torch.uint8 or tuple(exps.shape) != (rows, groups) or not exps.is_contiguous():
        raise ValueError(f"exps must be a contiguous uint8 tensor {(rows, groups)}, got {exps.dtype} {tuple(exps.shape)}")
    _on_device(codes, "codes", device)
    _on_device(exps, "exps", device)
    return codes.data_ptr(), exps.data_ptr()


def _new_ckpt(rows, cols, device):
    groups = (cols + 31) // 32
    return (torch.empty((rows, groups * 32), dtype=torch.int8, device=device),
            torch.empty((rows, groups), dtype=torch.uint8, device=device))


def _pack_into(wanted, rows, cols, device):
    """(checkpoint or None, its pointers) of an optional checkpoint output."""
    if not wanted:
        return None, (None, None)
    ckpt = _new_ckpt(rows, cols, device)
    return ckpt, (ckpt[0].data_ptr(), ckpt[1].data_ptr())


def _out(t, name, dtype, rows, cols, device):
    """(tensor, pointer, row stride) of an output matrix: the given one, checked, or a new one."""
    if t is None:
        t = torch.empty((rows, cols), dtype=dtype, device=device)
        return t, t.data_ptr(), cols
    p, ld = _matrix(t, name, dtype, (rows, cols))
    _on_device(t, name, device)
    return t, p, ld


def _out_vector(t, name, n, device):
    if t is None:
        t = torch.empty(n, dtype=torch.float32, device=device)
        return t, t.data_ptr()
    return t, _vector(t, name, torch.float32, n, device)


@contextlib.contextmanager
def _other_stream(stream, inputs):
    with torch.cuda.stream(stream):
        yield
        for t in inputs:
            if t is not None:
                t.record_stream(stream)


@contextlib.contextmanager
def _other_device(device):
    with torch.cuda.device(device):
        yield


_HERE = contextlib.nullcontext()


def _where(stream, device, *inputs):
    """The context in which a call allocates and launches."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
        if stream != torch.cuda.current_stream(device):
            return _other_stream(stream, inputs)
    if device.index != torch._C._cuda_getDevice():
        return _other_device(device)
    return _HERE


def _handle(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def ckpt_pack(x, *, codes=None, exps=None, stream=None):
    """The 8-bit checkpoint of ``x`` [rows, cols]: ``(codes, exps)``."""
    px, ldx = _matrix(x, "x")
    rows, cols = x.shape
    dev = x.device
    if (codes is None) != (exps is None):
        raise ValueError("pass both codes and exps, or neither")
    with _where(stream, dev, x, codes, exps):
        if codes is None:
            (codes, exps), (pc, pe) = _pack_into(True, rows, cols, dev)
        else:
            pc, pe = _ckpt((codes, exps), rows, cols, dev)
        _call("gc_ckpt_pack", _DTYPE[x.dtype], px, ldx, rows, cols, pc, pe, _handle(dev))
    return codes, exps


def ckpt_unpack(codes, exps, cols, dtype, *, out=None, stream=None):
    """The values of a checkpoint of a [rows, cols] matrix, as ``dtype``."""
    if dtype not in _DTYPE:
        raise ValueError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    if not codes.is_cuda:
        raise ValueError("codes must be a GPU tensor")
    rows = codes.shape[0]
    dev = codes.device
    pc, pe = _ckpt((codes, exps), rows, cols, dev)
    with _where(stream, dev, codes, exps, out):
        out, po, ldo = _out(out, "out", dtype, rows, cols, dev)
        _call("gc_ckpt_unpack", _DTYPE[dtype], pc, pe, rows, cols, po, ldo, _handle(dev))
    return out


def act_forward(x, kind="gelu", *, pack_x=False, pack_y=False, y=None, stream=None):
    """``y = f(x)`` for kind "gelu", "gelu_tanh" or "silu"; returns ``(y, x_ckpt, y_ckpt)``, the
    checkpoints (of x, and of y as stored) made in the same pass when asked for, else None."""
    k = _kind(kind)
    px, ldx = _matrix(x, "x")
    rows, cols = x.shape
    dt, dev = x.dtype, x.device
    with _where(stream, dev, x, y):
        y, py, ldy = _out(y, "y", dt, rows, cols, dev)
        xc, pxc = _pack_into(pack_x, rows, cols, dev)
        yc, pyc = _pack_into(pack_y, rows, cols, dev)
        _call("gc_act_forward", _DTYPE[dt], k, px, ldx, rows, cols, py, ldy, *pxc, *pyc, _handle(dev))
    return y, xc, yc


def _kept(x, ckpt, dtype, rows, cols, device):
    """(pointer, stride, codes, exps) of the input kept for a backward pass: in full, or as its checkpoint."""
    if ckpt is not None:
        return (None, 0, *_ckpt(ckpt, rows, cols, device))
    px, ldx = _matrix(x, "x", dtype, (rows, cols))
    _on_device(x, "x", device)
    return px, ldx, None, None


def act_backward(dy, kind="gelu", *, x=None, ckpt=None, dx=None, stream=None):
    """``dx = dy * f'(x)`` from ``x`` itself or from its checkpoint (exactly one of the two)."""
    k = _kind(kind)
    if (x is None) == (ckpt is None):
        raise ValueError("pass exactly one of x and ckpt")
    pdy, lddy = _matrix(dy, "dy")
    rows, cols = dy.shape
    dt, dev = dy.dtype, dy.device
    kept = _kept(x, ckpt, dt, rows, cols, dev)
    with _where(stream, dev, dy, x, dx, *(ckpt or ())):
        dx, pdx, lddx = _out(dx, "dx", dt, rows, cols, dev)
        _call("gc_act_backward", _DTYPE[dt], k, pdy, lddy, *kept, rows, cols, pdx, lddx, _handle(dev))
    return dx


def _weights(dtype, cols, device, weight, bias=None):
    """(type, pointers) of optional weight vectors that share the input's type or float32."""
    wdt = weight.dtype if weight is not None else bias.dtype if bias is not None else dtype
    if wdt is not dtype and wdt is not torch.float32:
        raise ValueError(f"weight and bias must be {dtype} or float32, got {wdt}")
    return (_DTYPE[wdt], None if weight is None else _vector(weight, "weight", wdt, cols, device),
            None if bias is None else _vector(bias, "bias", wdt, cols, device))


def layernorm_forward(x, weight=None, bias=None, eps=1e-5, *, pack_x=False, pack_y=False, y=None, stream=None):
    """Layer norm over the columns; returns ``(y, mean, rstd, x_ckpt, y_ckpt)`` with float32
    statistics, and the checkpoints as in :func:`act_forward`.  ``weight`` and ``bias`` are of x's type or
    float32."""
    px, ldx = _matrix(x, "x")
    rows, cols = x.shape
    dev = x.device
    wdt, pw, pb = _weights(x.dtype, cols, dev, weight, bias)
    dt = x.dtype
    with _where(stream, dev, x, weight, bias, y):
        y, py, ldy = _out(y, "y", dt, rows, cols, dev)
        mean = torch.empty(rows, dtype=torch.float32, device=dev)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        xc, pxc = _pack_into(pack_x, rows, cols, dev)
        yc, pyc = _pack_into(pack_y, rows, cols, dev)
        _call("gc_layernorm_forward", _DTYPE[dt], px, ldx, rows, cols, wdt, pw, pb, eps, py, ldy, mean.data_ptr(),
              rstd.data_ptr(), *pxc, *pyc, _handle(dev))
    return y, mean, rstd, xc, yc


def _workspace(name, args, device, workspace):
    need = ctypes.c_size_t(0)
    _call(name, *args, ctypes.byref(need))
    if need.value == 0:
        return None, 0, None
    if workspace is None:
        workspace = torch.empty(need.value, dtype=torch.uint8, device=device)
    elif workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace.data_ptr(), workspace.numel(), workspace


def layernorm_backward(dy, mean, rstd, weight=None, *, x=None, ckpt=None, dx=None, dw=None, db=None, accumulate=False,
                       workspace=None, stream=None):
    """Gradients of :func:`layernorm_forward` from ``x`` itself or from its checkpoint (exactly one
    of the two); returns ``(dx, dw, db)``.  dw and db are float32; with ``accumulate`` they are
    added to the tensors passed in."""
    if (x is None) == (ckpt is None):
        raise ValueError("pass exactly one of x and ckpt")
    if accumulate and (dw is None or db is None):
        raise ValueError("accumulate needs dw and db")
    pdy, lddy = _matrix(dy, "dy")
    rows, cols = dy.shape
    dt, dev = dy.dtype, dy.device
    wdt, pw, _ = _weights(dt, cols, dev, weight)
    pm = _vector(mean, "mean", torch.float32, rows, dev)
    pr = _vector(rstd, "rstd", torch.float32, rows, dev)
    kept = _kept(x, ckpt, dt, rows, cols, dev)
    with _where(stream, dev, dy, mean, rstd, weight, x, dx, dw, db, workspace, *(ckpt or ())):
        dx, pdx, lddx = _out(dx, "dx", dt, rows, cols, dev)
        dw, pdw = _out_vector(dw, "dw", cols, dev)
        db, pdb = _out_vector(db, "db", cols, dev)
        pws, nws, keep = _workspace("gc_layernorm_backward_workspace", (rows, cols), dev, workspace)
        _call("gc_layernorm_backward", _DTYPE[dt], pdy, lddy, *kept, rows, cols, wdt, pw, pm, pr, pdx, lddx, pdw, pdb,
              1 if accumulate else 0, pws, nws, _handle(dev))
    return dx, dw, db


def linear_wgrad(dy, codes, exps, in_features, *, dw=None, db=None, bias=True, accumulate=False, workspace=None,
                 stream=None):
    """Weight and bias gradient of ``y = x W^T + b`` from the checkpoint of x [rows, in_features] and
    dy [rows, out_features]; returns float32 ``(dw [out_features, in_features], db [out_features])``,
    db None with ``bias=False``.  ``dw`` may be a view into a gradient bucket; with ``accumulate`` the
    gradients are added to the tensors passed in."""
    if accumulate and (dw is None or (bias and db is None)):
        raise ValueError("accumulate needs dw (and db)")
    pdy, lddy = _matrix(dy, "dy")
    rows, outs = dy.shape
    dev = dy.device
    pc, pe = _ckpt((codes, exps), rows, in_features, dev)
    with _where(stream, dev, dy, codes, exps, dw, db, workspace):
        dw, pdw, lddw = _out(dw, "dw", torch.float32, outs, in_features, dev)
        pdb = None
        if bias:
            db, pdb = _out_vector(db, "db", outs, dev)
        dt = _DTYPE[dy.dtype]
        pws, nws, keep = _workspace("gc_linear_wgrad_workspace", (dt, rows, in_features, outs), dev, workspace)
        _call("gc_linear_wgrad", dt, pdy, lddy, pc, pe, rows, in_features, outs, pdw, lddw, pdb, 1 if accumulate else 0,
              pws, nws, _handle(dev))
    return dw, (db if bias else None)
