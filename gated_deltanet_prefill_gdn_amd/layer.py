"""Binding of the layer operators of include/gdn.h: the short causal convolution in front of the
recurrence, the gated norm behind it, and the selective state space scan.

As in the package's other calls the names are those of the C ABI, tensors are checked here and
outputs and workspaces allocated with torch where the caller passes none; every step of the
computation runs in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (GDN_DTYPE_BF16, GDN_DTYPE_F32, GDN_OK, GdnError, GdnProblem, _need, load_library)

GDN_CONV_SILU = 1
GDN_NORM_RMS = 1
GDN_NORM_GATE_FIRST = 2

_Three = ctypes.c_int32 * 3
_CODES = {torch.bfloat16: GDN_DTYPE_BF16, torch.float32: GDN_DTYPE_F32}
_F32, _I64 = torch.float32, torch.int64


class GdnConvProblem(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64),
        ("batch", ctypes.c_int64),
        ("pool_size", ctypes.c_int64),
        ("x_stride", ctypes.c_int64),
        ("dx_stride", ctypes.c_int64),
        ("channels", _Three),
        ("width", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("dout_dtype", ctypes.c_int32),
        ("flags", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class GdnNormProblem(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64),
        ("x_stride", ctypes.c_int64),
        ("z_stride", ctypes.c_int64),
        ("dz_stride", ctypes.c_int64),
        ("heads", ctypes.c_int32),
        ("dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("flags", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("reserved", ctypes.c_int32),
    ]


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _shape(t, name, shape, dtype, like):
    """t: a dense tensor of this shape and dtype on the device of `like`."""
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != like.get_device()
            or not t.is_contiguous()):
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        _need(t, name, dtype=dtype, device=like.device)


def _rows(t, name, inner, like):
    """Token stride of t, whose tokens are dense rows of `inner` shape some stride apart, of the
    dtype and on the device of `like`."""
    if t.shape[1:] != inner:
        raise ValueError(f"{name} must be [N, {', '.join(map(str, inner))}], got {list(t.shape)}")
    if t.dtype is not like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    size = math.prod(inner)
    if t.is_contiguous():
        return size
    dense = 1
    for d, st in zip(reversed(inner), reversed(t.stride()[1:])):
        if st != dense and d != 1:
            raise ValueError(f"{name}: the entries of a token must be dense")
        dense *= d
    if t.shape[0] <= 1:
        return size
    if t.stride(0) < size:
        raise ValueError(f"{name}: tokens overlap (stride {t.stride(0)} for rows of {size})")
    return t.stride(0)


def _p(t):
    return t.data_ptr() if t is not None else None


def _new(stream, shape, dtype, device):
    """Memory for an output or a workspace. It belongs to the stream that the call runs on, so
    that its reuse is ordered with the kernels that write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _like(stream, t):
    """Dense memory of t's shape and dtype (empty_like costs half of what empty does)."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    return _new(stream, t.shape, t.dtype, t.device)


def _call(what, device, stream, fn, *args):
    """The library launches on the current device, so it is made that of the tensors."""
    if device.type != "cuda":
        raise ValueError(f"{what} runs on a HIP device; tensors are on {device}")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device.index)  # 1.7 us less than current_stream()
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    else:
        raw = stream.cuda_stream
    if device.index == torch.cuda.current_device():
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, raw)
    if rc != GDN_OK:
        raise GdnError(rc, what)


def _workspace(workspace, need, device, stream):
    if workspace is None:
        return _new(stream, max(need, 1), torch.uint8, device)
    _need(workspace, "workspace", dtype=torch.uint8, ndim=1, device=device)
    return workspace


def _index(t, name, like):
    if (t.dtype is not _I64 or t.dim() != 1 or t.get_device() != like.get_device()
            or not t.is_contiguous()):
        _need(t, name, dtype=_I64, ndim=1, device=like.device)
    return t.shape[0]


def _slots(pool):
    return pool.shape[0] if pool.dim() else 0


def _requests(cache_indices, cu_seqlens, like):
    """B; cache_indices may be None (a convolution without a state pool)."""
    n = None if cache_indices is None else _index(cache_indices, "cache_indices", like)
    if cu_seqlens is None:
        return n
    b = _index(cu_seqlens, "cu_seqlens", like) - 1
    if b < 0 or (n is not None and n != b):
        raise ValueError("cu_seqlens must have B + 1 entries")
    return b


# ---- short causal convolution

def conv_problem(x, width, dims, batch, pool_size=0, silu=True, dout_dtype=GDN_DTYPE_F32,
                 dx_stride=None) -> GdnConvProblem:
    """Descriptor of a convolution of x [N, sum(dims)] (see gdn_conv_problem_t)."""
    if not 1 <= len(dims) <= 3:
        raise ValueError("one to three outputs")
    ch = sum(dims)
    dense = x.is_contiguous() and x.dim() == 2 and x.shape[1] == ch
    stride = ch if dense else _rows(x, "x", (ch,), x)
    return GdnConvProblem(x.shape[0], batch, pool_size, stride,
                          ch if dx_stride is None else dx_stride,
                          _Three(*dims), width, _code(x, "x"),
                          dout_dtype, GDN_CONV_SILU if silu else 0, 0)


def _conv_check(x, weight, bias, state_pool, cache_indices, cu_seqlens, dims, silu, **kw):
    dev = x.device
    if x.dim() != 2:
        raise ValueError(f"x must be [N, channels], got {list(x.shape)}")
    ch = x.shape[1]
    dims = (ch,) if dims is None else tuple(dims)
    if sum(dims) != ch:
        raise ValueError(f"dims {dims} do not add up to the {ch} channels of x")
    if weight.dim() != 2 or weight.shape[0] != ch:
        raise ValueError(f"weight must be [{ch}, W], got {list(weight.shape)}")
    w = weight.shape[1]
    _shape(weight, "weight", (ch, w), _F32, x)
    if bias is not None:
        _shape(bias, "bias", (ch,), _F32, x)
    if state_pool is None and cu_seqlens is None:
        raise ValueError("state_pool is required")
    if state_pool is not None:
        if cache_indices is None:
            raise ValueError("cache_indices are required with a state_pool")
        _shape(state_pool, "state_pool", (_slots(state_pool), w - 1, ch), x.dtype, x)
    batch = _requests(cache_indices if state_pool is not None else None, cu_seqlens, x)
    prob = conv_problem(x, w, dims, batch, 0 if state_pool is None else state_pool.shape[0], silu,
                        **kw)
    return dev, dims, prob


def _conv_outs(outs, x, dims, stream):
    n = x.shape[0]
    if outs is None:
        if len(dims) == 1:
            return (_like(stream, x),)
        if stream is not None:
            return tuple([_new(stream, (n, d), x.dtype, x.device) for d in dims])
        made = [x.new_empty((n, dims[0]))]
        for d, before in zip(dims[1:], dims):
            made.append(torch.empty_like(made[-1]) if d == before else x.new_empty((n, d)))
        return tuple(made)
    if len(outs) != len(dims):
        raise ValueError(f"{len(dims)} outputs are wanted, got {len(outs)}")
    for i, (o, d) in enumerate(zip(outs, dims)):
        _shape(o, f"outs[{i}]", (n, d), x.dtype, x)
    return tuple(outs)


def _three(ts):
    return [_p(t) if t.shape[1] else None for t in ts] + [None] * (3 - len(ts))


def gdn_conv_fwd(x, weight, bias, state_pool, cache_indices, cu_seqlens, dims=None,
                 silu: bool = True, outs=None, stream=None):
    """Short causal convolution over every request's tokens; returns a tuple of dense tensors
    [N, dims[i]] in x's dtype (``.view(N, heads, d)`` makes them q, k, v of gdn_prefill_fwd).

    x [N, channels] bf16/fp32, rows any stride apart (a slice of a projection's row); weight
    [channels, W] fp32, W = 2 .. 4; bias [channels] fp32 or None; state_pool [pool, W - 1,
    channels] in x's dtype, the last inputs of each slot, oldest first, updated in place (None:
    zero history, none kept; cache_indices is then not used); cache_indices [B] and cu_seqlens
    [B + 1] int64. ``dims``: channels of the one to three outputs (default: one output). Rows
    behind cu_seqlens[B], and requests whose cache index is outside the pool, are padding: their
    outputs are not written."""
    dev, dims, prob = _conv_check(x, weight, bias, state_pool, cache_indices, cu_seqlens, dims,
                                  silu)
    outs = _conv_outs(outs, x, dims, stream)
    _call("gdn_conv_fwd", dev, stream, load_library().gdn_conv_fwd, _p(x), _p(weight), _p(bias),
          _p(state_pool), _p(cache_indices), _p(cu_seqlens), *_three(outs), ctypes.byref(prob))
    return outs


def gdn_conv_decode_fwd(x, weight, bias, state_pool, cache_indices, dims=None, silu: bool = True,
                        outs=None, stream=None):
    """gdn_conv_fwd for one new token per request: x [B, channels], row b with request b."""
    dev, dims, prob = _conv_check(x, weight, bias, state_pool, cache_indices, None, dims, silu)
    outs = _conv_outs(outs, x, dims, stream)
    _call("gdn_conv_decode_fwd", dev, stream, load_library().gdn_conv_decode_fwd, _p(x),
          _p(weight), _p(bias), _p(state_pool), _p(cache_indices), *_three(outs),
          ctypes.byref(prob))
    return outs


def gdn_conv_bwd_workspace_size(prob: GdnConvProblem) -> int:
    return int(load_library().gdn_conv_bwd_workspace_size(ctypes.byref(prob)))


def gdn_conv_bwd(x, weight, bias, state_pool, cache_indices, cu_seqlens, douts, dstate=None,
                 silu: bool = True, dx=None, workspace=None, stream=None):
    """Gradients of gdn_conv_fwd. state_pool: the pool as it was BEFORE the forward call (or
    None); douts: the outputs' gradients, dense [N, dims[i]], all bf16 or all fp32 (those of
    gdn_prefill_bwd, say); dstate [B, W - 1, channels] fp32, the final states' gradient, or None.
    Returns a dict: dx [N, channels] in x's dtype (``dx``: rows any stride apart), dweight fp32,
    dbias fp32 (with a bias), dstate0 [B, W - 1, channels] fp32 (with a state_pool)."""
    douts = tuple(douts)
    if not douts or any(d.dim() != 2 for d in douts):
        raise ValueError("douts are one to three tensors [N, dims[i]]")
    dims = tuple(d.shape[1] for d in douts)
    n, dev = x.shape[0], x.device
    for i, d in enumerate(douts):
        _shape(d, f"douts[{i}]", (n, dims[i]), douts[0].dtype, x)
    ch = x.shape[1] if x.dim() == 2 else 0
    if dx is None:
        dx = _like(stream, x)
    dev, dims, prob = _conv_check(x, weight, bias, state_pool, cache_indices, cu_seqlens, dims,
                                  silu, dout_dtype=_code(douts[0], "douts"),
                                  dx_stride=_rows(dx, "dx", (ch,), x))
    if dx.shape[0] != n:
        raise ValueError("dx must have N rows")
    b, w = prob.batch, prob.width
    if dstate is not None:
        _shape(dstate, "dstate", (b, w - 1, ch), _F32, x)
    g = {"dx": dx, "dweight": _like(stream, weight)}
    if bias is not None:
        g["dbias"] = _like(stream, bias)
    if state_pool is not None:
        g["dstate0"] = _new(stream, (b, w - 1, ch), _F32, dev)
    ws = _workspace(workspace, gdn_conv_bwd_workspace_size(prob), dev, stream)
    _call("gdn_conv_bwd", dev, stream, load_library().gdn_conv_bwd, _p(x), _p(weight), _p(bias),
          _p(state_pool), _p(cache_indices), _p(cu_seqlens), *_three(douts), _p(dstate), _p(dx),
          _p(g["dweight"]), _p(g.get("dbias")), _p(g.get("dstate0")), ctypes.byref(prob), _p(ws),
          ws.numel())
    return g


# ---- selective state space scan

def gdn_ssm_workspace_size(prob: GdnProblem) -> int:
    return int(load_library().gdn_ssm_workspace_size(ctypes.byref(prob)))


def _ssm_check(C, B, x, dt, A_log, dt_bias, D, state_pool, cache_indices, cu_seqlens, out,
               stream):
    dev = x.device
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [N, HV, dv] and B [N, H, dk]")
    n, hv, dv = x.shape
    _, h, dk = B.shape
    code = _code(x, "x")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    _shape(B, "B", (n, h, dk), x.dtype, x)
    _shape(C, "C", (n, h, dk), x.dtype, x)
    _shape(dt, "dt", (n, hv), _F32, x)
    _shape(A_log, "A_log", (hv,), _F32, x)
    _shape(dt_bias, "dt_bias", (hv,), _F32, x)
    if D is not None:
        _shape(D, "D", (hv,), _F32, x)
    _shape(state_pool, "state_pool", (_slots(state_pool), hv, dv, dk), _F32, x)
    batch = _requests(cache_indices, cu_seqlens, x)
    if cu_seqlens is None and batch != n:
        raise ValueError("cache_indices must have one entry per row of x")
    if out is None:
        out = _like(stream, x)
    else:
        _shape(out, "out", (n, hv, dv), x.dtype, x)
    return dev, out, GdnProblem(n, batch, h, hv, dk, dv, state_pool.shape[0], code, 0)


def gdn_ssm_prefill_fwd(C, B, x, dt, A_log, dt_bias, D, state_pool, cache_indices, cu_seqlens,
                        out=None, workspace=None, stream=None):
    """Selective state space scan over every request's tokens; returns ``out`` [N, HV, dv] in x's
    dtype. S <- exp(-exp(A_log) d) S + d x B^T, out = S C + D x, d = softplus(dt + dt_bias).

    C, B [N, H, dk] and x [N, HV, dv] bf16/fp32; dt [N, HV] fp32; A_log, dt_bias [HV] fp32; D
    [HV] fp32 or None; state_pool [pool, HV, dv, dk] fp32 (updated in place); cache_indices [B]
    and cu_seqlens [B + 1] int64. ``workspace``: an optional uint8 device tensor of at least
    gdn_ssm_workspace_size bytes. Rows behind cu_seqlens[B], and requests whose cache index is
    outside the pool, are padding: their outputs are not written."""
    dev, out, prob = _ssm_check(C, B, x, dt, A_log, dt_bias, D, state_pool, cache_indices,
                                cu_seqlens, out, stream)
    ws = _workspace(workspace, gdn_ssm_workspace_size(prob), dev, stream)
    _call("gdn_ssm_prefill_fwd", dev, stream, load_library().gdn_ssm_prefill_fwd, _p(C), _p(B),
          _p(x), _p(dt), _p(A_log), _p(dt_bias), _p(D), _p(state_pool), _p(cache_indices),
          _p(cu_seqlens), _p(out), ctypes.byref(prob), _p(ws), ws.numel())
    return out


def gdn_ssm_decode_fwd(C, B, x, dt, A_log, dt_bias, D, state_pool, cache_indices, out=None,
                       stream=None):
    """One step of the scan, one token per request: row b of every input with request b."""
    dev, out, prob = _ssm_check(C, B, x, dt, A_log, dt_bias, D, state_pool, cache_indices, None,
                                out, stream)
    _call("gdn_ssm_decode_fwd", dev, stream, load_library().gdn_ssm_decode_fwd, _p(C), _p(B),
          _p(x), _p(dt), _p(A_log), _p(dt_bias), _p(D), _p(state_pool), _p(cache_indices),
          _p(out), ctypes.byref(prob))
    return out


# ---- gated norm

def norm_problem(x, z=None, eps=1e-6, rms=True, gate_first=False, dz=None) -> GdnNormProblem:
    """Descriptor of a norm of x [N, heads, dim] (see gdn_norm_problem_t)."""
    inner = x.shape[1:]
    xs = inner.numel() if x.is_contiguous() else _rows(x, "x", inner, x)
    zs = 0 if z is None else _rows(z, "z", inner, x)
    dzs = zs if dz is None else _rows(dz, "dz", inner, x)
    return GdnNormProblem(x.shape[0], xs, zs, dzs, inner[0], inner[1], _code(x, "x"),
                          (GDN_NORM_RMS if rms else 0) | (GDN_NORM_GATE_FIRST if gate_first else 0),
                          eps, 0)


def _norm_check(x, weight, bias, z, eps, rms, gate_first, dz=None):
    dev = x.device
    if x.dim() != 3:
        raise ValueError(f"x must be [N, heads, dim], got {list(x.shape)}")
    dim = x.shape[2]
    _shape(weight, "weight", (dim,), _F32, x)
    if bias is not None:
        _shape(bias, "bias", (dim,), _F32, x)
    for t, name in ((z, "z"), (dz, "dz")):
        if t is not None and t.shape != x.shape:
            raise ValueError(f"{name} must have x's shape {list(x.shape)}, got {list(t.shape)}")
    if gate_first and z is None:
        raise ValueError("gate_first needs a gate z")
    return dev, norm_problem(x, z, eps, rms, gate_first, dz)


def gdn_norm_fwd(x, weight, bias=None, z=None, eps: float = 1e-6, rms: bool = True,
                 gate_first: bool = False, out=None, stream=None):
    """RMS norm (``rms=False``: layer norm) of every row x[t, h], with an optional gate silu(z)
    on the result, or on the input with ``gate_first``; returns ``out`` [N, heads, dim].

    x and z [N, heads, dim] bf16/fp32, tokens any stride apart; weight [dim] and bias [dim] or
    None fp32, shared by the heads; 1 <= dim <= 16384."""
    dev, prob = _norm_check(x, weight, bias, z, eps, rms, gate_first)
    if out is None:
        out = _like(stream, x)
    else:
        _shape(out, "out", x.shape, x.dtype, x)
    _call("gdn_norm_fwd", dev, stream, load_library().gdn_norm_fwd, _p(x), _p(weight), _p(bias),
          _p(z), _p(out), ctypes.byref(prob))
    return out


def gdn_norm_bwd_workspace_size(prob: GdnNormProblem) -> int:
    return int(load_library().gdn_norm_bwd_workspace_size(ctypes.byref(prob)))


def gdn_norm_bwd(x, weight, bias, z, dout, eps: float = 1e-6, rms: bool = True,
                 gate_first: bool = False, dz=None, workspace=None, stream=None):
    """Gradients of gdn_norm_fwd: a dict of dx (dense) and, with a gate, dz (``dz``: tokens any
    stride apart) in x's dtype, dweight and, with a bias, dbias, fp32. dout: dense, x's dtype."""
    if z is not None and dz is None:
        dz = _like(stream, z)
    elif z is None and dz is not None:
        raise ValueError("dz without a gate z")
    dev, prob = _norm_check(x, weight, bias, z, eps, rms, gate_first, dz)
    _shape(dout, "dout", x.shape, x.dtype, x)
    g = {"dx": _like(stream, x), "dweight": _like(stream, weight)}
    if z is not None:
        g["dz"] = dz
    if bias is not None:
        g["dbias"] = _like(stream, weight)
    ws = _workspace(workspace, gdn_norm_bwd_workspace_size(prob), dev, stream)
    _call("gdn_norm_bwd", dev, stream, load_library().gdn_norm_bwd, _p(x), _p(weight), _p(bias),
          _p(z), _p(dout), _p(g["dx"]), _p(dz), _p(g["dweight"]), _p(g.get("dbias")),
          ctypes.byref(prob), _p(ws), ws.numel())
    return g


def declare(L):
    """C signatures of the layer operators."""
    P, S, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    for name, n, prob, tail in (
            ("gdn_conv_fwd", 9, GdnConvProblem, [P]),
            ("gdn_conv_decode_fwd", 8, GdnConvProblem, [P]),
            ("gdn_conv_bwd", 14, GdnConvProblem, [P, S, P]),
            ("gdn_ssm_prefill_fwd", 11, GdnProblem, [P, S, P]),
            ("gdn_ssm_decode_fwd", 10, GdnProblem, [P]),
            ("gdn_norm_fwd", 5, GdnNormProblem, [P]),
            ("gdn_norm_bwd", 9, GdnNormProblem, [P, S, P])):
        fn = getattr(L, name)
        fn.restype = I
        fn.argtypes = [P] * n + [ctypes.POINTER(prob)] + tail
    for name, prob in (("gdn_conv_bwd_workspace_size", GdnConvProblem),
                       ("gdn_ssm_workspace_size", GdnProblem),
                       ("gdn_norm_bwd_workspace_size", GdnNormProblem)):
        fn = getattr(L, name)
        fn.restype = S
        fn.argtypes = [ctypes.POINTER(prob)]
