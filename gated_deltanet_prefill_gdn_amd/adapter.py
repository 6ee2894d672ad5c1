"""Binding of the low-rank adapters beside a shared projection (include/gdn.h). Conventions as in
layer.py."""
from __future__ import annotations

import ctypes

from . import GdnAdapterProblem, load_library
from .layer import _F32, _call, _code, _like, _new, _requests, _rows, _shape, _workspace


def _stride(t, name, width, like):
    """Row stride of t [N, width]: as layer._rows, quick where the rows are plainly fine."""
    s0, s1 = t.stride()
    if s1 == 1 and t.dtype is like.dtype and t.get_device() == like.get_device():
        if t.shape[0] <= 1:
            return width
        if s0 >= width:
            return s0
    return _rows(t, name, (width,), like)


def adapter_problem(x, base, A, batch, out=None) -> GdnAdapterProblem:
    """Descriptor of adapters A [adapters, R, K] on x [N, K] beside base [N, M] (see
    gdn_adapter_problem_t); ``out`` is dense where none is given."""
    n, k = x.shape
    m = base.shape[1]
    na, r, _ = A.shape
    return GdnAdapterProblem(n, batch, _stride(x, "x", k, x), _stride(base, "base", m, x),
                             m if out is None else _stride(out, "out", m, x), k, m, r, na,
                             _code(x, "x"), 0)


def gdn_adapter_workspace_size(prob: GdnAdapterProblem) -> int:
    return int(load_library().gdn_adapter_workspace_size(ctypes.byref(prob)))


def _run(what, x, base, A, B, scaling, adapter_indices, cu_seqlens, out, workspace, stream):
    if x.dim() != 2 or base.dim() != 2:
        raise ValueError(f"x must be [N, K] and base [N, M], got {list(x.shape)} and "
                         f"{list(base.shape)}")
    if A.dim() != 3:
        raise ValueError(f"A must be [adapters, R, K], got {list(A.shape)}")
    n, k = x.shape
    rows, m = base.shape
    na, r, _ = A.shape
    if rows != n:
        raise ValueError(f"base must have {n} rows, got {rows}")
    _shape(A, "A", (na, r, k), x.dtype, x)
    _shape(B, "B", (na, m, r), x.dtype, x)
    _shape(scaling, "scaling", (na,), _F32, x)
    batch = _requests(adapter_indices, cu_seqlens, x)
    if cu_seqlens is None and batch != n:
        raise ValueError("adapter_indices must have one entry per row of x")
    dense = out is None
    if dense:
        out = _like(stream, base) if base.is_contiguous() else _new(stream, (n, m), x.dtype, x.device)
    elif out.shape != base.shape:
        raise ValueError(f"out must be {list(base.shape)}, got {list(out.shape)}")
    prob = adapter_problem(x, base, A, batch, None if dense else out)
    ref = ctypes.byref(prob)
    lib = load_library()
    device = x.device
    ws = _workspace(workspace, lib.gdn_adapter_workspace_size(ref), device, stream)
    cu = () if cu_seqlens is None else (cu_seqlens.data_ptr(),)
    _call(what, device, stream, getattr(lib, what), x.data_ptr(), base.data_ptr(), A.data_ptr(),
          B.data_ptr(), scaling.data_ptr(), adapter_indices.data_ptr(), *cu, out.data_ptr(), ref,
          ws.data_ptr(), ws.numel())
    return out


def gdn_adapter_fwd(x, base, A, B, scaling, adapter_indices, cu_seqlens, out=None, workspace=None,
                    stream=None):
    """Low-rank adapters of a batch's requests beside a projection that they share; returns
    ``out`` [N, M] = base + scaling[a] (x A[a]^T) B[a]^T, a = adapter_indices of the row's request.

    x [N, K] and base [N, M] bf16/fp32, rows any stride apart; A [adapters, R, K] and B [adapters,
    M, R] in x's dtype, R <= 128; scaling [adapters] fp32; adapter_indices [B] (outside the bank:
    no adapter, out = base) and cu_seqlens [B + 1] int64. ``out``: rows any stride apart, or base
    itself (dense by default). Rows behind cu_seqlens[B] are not written."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _run("gdn_adapter_fwd", x, base, A, B, scaling, adapter_indices, cu_seqlens, out,
                workspace, stream)


def gdn_adapter_decode_fwd(x, base, A, B, scaling, adapter_indices, out=None, workspace=None,
                           stream=None):
    """gdn_adapter_fwd for one new token per request: row b of x and base with request b."""
    return _run("gdn_adapter_decode_fwd", x, base, A, B, scaling, adapter_indices, None, out,
                workspace, stream)


def declare(L):
    """C signatures of the adapters."""
    P, S, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    prob = ctypes.POINTER(GdnAdapterProblem)
    for name, n in (("gdn_adapter_fwd", 8), ("gdn_adapter_decode_fwd", 7)):
        fn = getattr(L, name)
        fn.restype = I
        fn.argtypes = [P] * n + [prob, P, S, P]
    L.gdn_adapter_workspace_size.restype = S
    L.gdn_adapter_workspace_size.argtypes = [prob]
