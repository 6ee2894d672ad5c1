"""Binding of linear attention with a fixed decay for each head (include/gdn.h): prompts, single
tokens, gradients. Conventions as in layer.py."""
from __future__ import annotations

import ctypes

from . import GdnLinearProblem, load_library
from .layer import _F32, _call, _code, _like, _new, _p, _requests, _rows, _shape, _slots, _workspace


def _stride(t, name, heads, dim, like):
    """Token stride of t [N, heads, dim]: as layer._rows, quick where the rows are plainly fine."""
    s0, s1, s2 = t.stride()
    if s2 == 1 and s1 == dim and t.dtype is like.dtype and t.get_device() == like.get_device():
        if t.shape[0] <= 1:
            return heads * dim
        if s0 >= heads * dim:
            return s0
    return _rows(t, name, (heads, dim), like)


def linear_problem(q, k, v, batch, pool_size=0, scale=None) -> GdnLinearProblem:
    """Descriptor of a call on q, k [N, H, dk] and v [N, HV, dv] (see gdn_linear_problem_t)."""
    n, h, dk = q.shape
    _, hv, dv = v.shape
    return GdnLinearProblem(n, batch, pool_size, _stride(q, "q", h, dk, v),
                            _stride(k, "k", h, dk, v), _stride(v, "v", hv, dv, v), h, hv, dk, dv,
                            _code(v, "v"), dk ** -0.5 if scale is None else scale, 0, 0)


def _check(q, k, v, log_decay, state_pool, cache_indices, cu_seqlens, scale):
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q and k must be [N, H, dk] and v [N, HV, dv]")
    n, hv, dv = v.shape
    if q.shape[0] != n or k.shape != q.shape:
        raise ValueError(f"q and k must be [{n}, H, dk], got {list(q.shape)} and {list(k.shape)}")
    _shape(log_decay, "log_decay", (hv,), _F32, v)
    if state_pool is None:
        if cu_seqlens is None:
            raise ValueError("state_pool is required")
        batch = _requests(None, cu_seqlens, v)
    else:
        if cache_indices is None:
            raise ValueError("cache_indices are required with a state_pool")
        _shape(state_pool, "state_pool", (_slots(state_pool), hv, dv, q.shape[2]), _F32, v)
        batch = _requests(cache_indices, cu_seqlens, v)
        if cu_seqlens is None and batch != n:
            raise ValueError("cache_indices must have one entry per row of v")
    return linear_problem(q, k, v, batch, 0 if state_pool is None else state_pool.shape[0], scale)


def _out(out, v, stream):
    if out is None:
        return _like(stream, v)
    _shape(out, "out", v.shape, v.dtype, v)
    return out


def gdn_linear_workspace_size(prob: GdnLinearProblem) -> int:
    return int(load_library().gdn_linear_workspace_size(ctypes.byref(prob)))


def gdn_linear_prefill_fwd(q, k, v, log_decay, state_pool, cache_indices, cu_seqlens, scale=None,
                           out=None, workspace=None, stream=None):
    """Linear attention over every request's tokens; returns ``out`` [N, HV, dv], dense, in v's
    dtype. S <- exp(log_decay) S + v k^T, out = scale S q.

    q, k [N, H, dk] and v [N, HV, dv] bf16/fp32, tokens any multiple of 16 bytes apart (slices of
    a projection's row); log_decay [HV] fp32, not above 0; state_pool [pool, HV, dv, dk] fp32,
    updated in place (None: zero start states, none kept; cache_indices is then not used);
    cache_indices [B] and cu_seqlens [B + 1] int64. ``scale``: default dk ** -0.5. ``workspace``:
    an optional uint8 device tensor of at least gdn_linear_workspace_size bytes. Rows behind
    cu_seqlens[B], and requests whose cache index is outside the pool, are padding: their outputs
    are not written."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    prob = _check(q, k, v, log_decay, state_pool, cache_indices, cu_seqlens, scale)
    out = _out(out, v, stream)
    lib, ref, device = load_library(), ctypes.byref(prob), v.device
    ws = _workspace(workspace, lib.gdn_linear_workspace_size(ref), device, stream)
    _call("gdn_linear_prefill_fwd", device, stream, lib.gdn_linear_prefill_fwd, q.data_ptr(),
          k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _p(state_pool), _p(cache_indices),
          cu_seqlens.data_ptr(), out.data_ptr(), ref, ws.data_ptr(), ws.numel())
    return out


def gdn_linear_decode_fwd(q, k, v, log_decay, state_pool, cache_indices, scale=None, out=None,
                          stream=None):
    """One step of linear attention, one token per request: row b of every input with request b."""
    prob = _check(q, k, v, log_decay, state_pool, cache_indices, None, scale)
    out = _out(out, v, stream)
    _call("gdn_linear_decode_fwd", v.device, stream, load_library().gdn_linear_decode_fwd,
          q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), state_pool.data_ptr(),
          cache_indices.data_ptr(), out.data_ptr(), ctypes.byref(prob))
    return out


def gdn_linear_bwd_workspace_size(prob: GdnLinearProblem) -> int:
    return int(load_library().gdn_linear_bwd_workspace_size(ctypes.byref(prob)))


def gdn_linear_bwd(q, k, v, log_decay, state_pool, cache_indices, cu_seqlens, dout, dstate=None,
                   scale=None, workspace=None, stream=None):
    """Gradients of gdn_linear_prefill_fwd. state_pool: the pool as it was BEFORE the forward call
    (or None); dout [N, HV, dv] dense in v's dtype; dstate [B, HV, dv, dk] fp32, the final states'
    gradient, or None. Returns a dict of dense dq, dk [N, H, dk] and dv [N, HV, dv] in the inputs'
    dtype and, with a state_pool, dstate0 [B, HV, dv, dk] fp32. The decays are constants: they have
    no gradient."""
    prob = _check(q, k, v, log_decay, state_pool, cache_indices, cu_seqlens, scale)
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    _shape(dout, "dout", v.shape, v.dtype, v)
    states = (prob.batch, prob.num_v_heads, prob.head_v, prob.head_k)
    if dstate is not None:
        _shape(dstate, "dstate", states, _F32, v)
    g = {"dq": _like(stream, q), "dk": _like(stream, k), "dv": _like(stream, v)}
    if state_pool is not None:
        g["dstate0"] = _new(stream, states, _F32, v.device)
    ws = _workspace(workspace, gdn_linear_bwd_workspace_size(prob), v.device, stream)
    _call("gdn_linear_bwd", v.device, stream, load_library().gdn_linear_bwd, _p(q), _p(k), _p(v),
          _p(log_decay), _p(state_pool), _p(cache_indices), _p(cu_seqlens), _p(dout), _p(dstate),
          _p(g["dq"]), _p(g["dk"]), _p(g["dv"]), _p(g.get("dstate0")), ctypes.byref(prob), _p(ws),
          ws.numel())
    return g


def declare(L):
    """C signatures of linear attention."""
    P, S, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    prob = ctypes.POINTER(GdnLinearProblem)
    for name, n, tail in (("gdn_linear_prefill_fwd", 8, [P, S, P]),
                          ("gdn_linear_decode_fwd", 7, [P]), ("gdn_linear_bwd", 13, [P, S, P])):
        fn = getattr(L, name)
        fn.restype = I
        fn.argtypes = [P] * n + [prob] + tail
    for name in ("gdn_linear_workspace_size", "gdn_linear_bwd_workspace_size"):
        fn = getattr(L, name)
        fn.restype = S
        fn.argtypes = [prob]
