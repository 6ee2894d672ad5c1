"""Binding of the low-rank adapters beside a shared projection (include/gdn.h). Conventions as in
layer.py."""
from __future__ import annotations

import ctypes

from . import GdnAdapterProblem, load_library
from .layer import _F32, _call, _code, _new, _p, _requests, _rows, _shape, _workspace


def adapter_problem(x, base, A, batch, out=None) -> GdnAdapterProblem:
    """Descriptor of adapters A [adapters, R, K] on x [N, K] beside base [N, M] (see
    gdn_adapter_problem_t); ``out`` is dense where none is given."""
    k, m = x.shape[1], base.shape[1]
    return GdnAdapterProblem(x.shape[0], batch, _rows(x, "x", (k,), x),
                             _rows(base, "base", (m,), x),
                             m if out is None else _rows(out, "out", (m,), x), k, m, A.shape[1],
                             A.shape[0], _code(x, "x"), 0)


def gdn_adapter_workspace_size(prob: GdnAdapterProblem) -> int:
    return int(load_library().gdn_adapter_workspace_size(ctypes.byref(prob)))


def _run(what, x, base, A, B, scaling, adapter_indices, cu_seqlens, out, workspace, stream):
    if x.dim() != 2 or base.dim() != 2 or x.shape[0] != base.shape[0]:
        raise ValueError(f"x must be [N, K] and base [N, M], got {list(x.shape)} and "
                         f"{list(base.shape)}")
    if A.dim() != 3:
        raise ValueError(f"A must be [adapters, R, K], got {list(A.shape)}")
    (n, k), m = x.shape, base.shape[1]
    na, r = A.shape[:2]
    _shape(A, "A", (na, r, k), x.dtype, x)
    _shape(B, "B", (na, m, r), x.dtype, x)
    _shape(scaling, "scaling", (na,), _F32, x)
    batch = _requests(adapter_indices, cu_seqlens, x)
    if cu_seqlens is None and batch != n:
        raise ValueError("adapter_indices must have one entry per row of x")
    if out is None:
        out = _new(stream, (n, m), x.dtype, x.device)
    elif out.shape != base.shape:
        raise ValueError(f"out must be {list(base.shape)}, got {list(out.shape)}")
    prob = adapter_problem(x, base, A, batch, out)
    ws = _workspace(workspace, gdn_adapter_workspace_size(prob), x.device, stream)
    fn = getattr(load_library(), what)
    cu = () if cu_seqlens is None else (_p(cu_seqlens),)
    _call(what, x.device, stream, fn, _p(x), _p(base), _p(A), _p(B), _p(scaling),
          _p(adapter_indices), *cu, _p(out), ctypes.byref(prob), _p(ws), ws.numel())
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
