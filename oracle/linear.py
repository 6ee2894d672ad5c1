"""Linear attention with a decay per head, and low-rank adapters, in fp64 -- TEST INFRASTRUCTURE
ONLY.

Only ``tests/`` and ``smoke()`` import this module. It shares no code with the HIP library. The
recurrence and its gradients token by token, the adapters request by request, each from its
definition. Beside a result stands its *magnitude*: the same sums over absolute values, which bounds
the rounding error of any evaluation of the sum. Pinned by tests/test_oracle_linear.py (central
differences, closed forms).
"""
from __future__ import annotations

import numpy as np


def _requests(pool, idx, cu, n):
    """(request, slot, tokens) of the live requests; slot None without a pool."""
    for b in range(len(cu) - 1):
        if pool is None:
            yield b, None, range(cu[b], cu[b + 1])
        elif 0 <= idx[b] < len(pool):
            yield b, idx[b], range(cu[b], cu[b + 1])


def _heads(t, hv):
    t = np.asarray(t, np.float64)
    return np.repeat(t, hv // t.shape[1], 1)


def linear_fwd(q, k, v, log_decay, scale, pool, idx, cu):
    """(out, new pool, magnitude of out, magnitude of the states, written rows)."""
    v = np.asarray(v, np.float64)
    n, hv, dv = v.shape
    q, k = _heads(q, hv), _heads(k, hv)
    dk = q.shape[2]
    a = np.exp(np.minimum(np.asarray(log_decay, np.float64), 0))[:, None, None]
    new = None if pool is None else np.array(pool, np.float64)
    mags = None if pool is None else np.abs(new)
    out, mag, written = np.zeros((n, hv, dv)), np.zeros((n, hv, dv)), np.zeros(n, bool)
    for b, slot, tokens in _requests(pool, idx, cu, n):
        s = np.zeros((hv, dv, dk)) if slot is None else new[slot]
        m = np.zeros((hv, dv, dk)) if slot is None else mags[slot]
        for t in tokens:
            u = v[t][:, :, None] * k[t][:, None, :]
            s[:] = a * s + u
            m[:] = a * m + np.abs(u)
            out[t] = scale * np.matmul(s, q[t][:, :, None])[..., 0]
            mag[t] = abs(scale) * np.matmul(m, np.abs(q[t])[:, :, None])[..., 0]
            written[t] = True
    return out, new, mag, mags, written


def linear_bwd(q, k, v, log_decay, scale, pool, idx, cu, dout, dstate):
    """dict of dq, dk, dv, dstate0 and of their magnitudes (key + "_mag")."""
    v, dout = np.asarray(v, np.float64), np.asarray(dout, np.float64)
    n, hv, dv = v.shape
    h = q.shape[1]
    q, k = _heads(q, hv), _heads(k, hv)
    dk = q.shape[2]
    a = np.exp(np.minimum(np.asarray(log_decay, np.float64), 0))[:, None, None]
    g = {}
    for name, shape in (("dq", (n, hv, dk)), ("dk", (n, hv, dk)), ("dv", (n, hv, dv)),
                        ("dstate0", (len(cu) - 1, hv, dv, dk))):
        g[name], g[name + "_mag"] = np.zeros(shape), np.zeros(shape)
    for suffix, f in (("", lambda x: x), ("_mag", np.abs)):
        Q, K, V, O = (f(x) for x in (q, k, v, dout))
        c = f(np.float64(scale))
        for b, slot, tokens in _requests(pool, idx, cu, n):
            s = np.zeros((hv, dv, dk)) if slot is None else f(np.array(pool[slot], np.float64))
            for t in tokens:
                s = a * s + V[t][:, :, None] * K[t][:, None, :]
                g["dq" + suffix][t] = c * np.matmul(O[t][:, None, :], s)[:, 0]
            d = np.zeros((hv, dv, dk)) if dstate is None else f(np.array(dstate[b], np.float64))
            for t in reversed(tokens):
                d = d + c * O[t][:, :, None] * Q[t][:, None, :]
                g["dv" + suffix][t] = np.matmul(d, K[t][:, :, None])[..., 0]
                g["dk" + suffix][t] = np.matmul(V[t][:, None, :], d)[:, 0]
                d = a * d
            g["dstate0" + suffix][b] = d
    for name in ("dq", "dk", "dq_mag", "dk_mag"):
        g[name] = g[name].reshape(n, h, hv // h, dk).sum(2)
    return g


def adapter(x, base, A, B, scaling, idx, cu):
    """(out, magnitude, written rows)."""
    x, out = np.asarray(x, np.float64), np.array(base, np.float64)
    mag, written = np.abs(out), np.zeros(len(x), bool)
    for b in range(len(cu) - 1):
        rows = slice(cu[b], cu[b + 1])
        written[rows] = True
        if 0 <= idx[b] < len(A):
            a, bb = np.asarray(A[idx[b]], np.float64), np.asarray(B[idx[b]], np.float64)
            out[rows] += scaling[idx[b]] * (x[rows] @ a.T) @ bb.T
            mag[rows] += abs(scaling[idx[b]]) * (np.abs(x[rows]) @ np.abs(a).T) @ np.abs(bb).T
    return out, mag, written
