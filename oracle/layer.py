"""Layer operators in fp64 -- TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module. It shares no code with the HIP library.

The short causal convolution (forward, state, gradients), the selective state space scan token by
token, and the gated layer / RMS norm (forward, gradients), each from its definition with plain
numpy loops over requests. Beside a result stands its *magnitude*: the same sums over absolute
values, which bounds the rounding error of any evaluation of the sum, so that tests can state
tolerances in units of rounding steps. Pinned by tests/test_oracle_layer.py (central differences,
closed forms).
"""
from __future__ import annotations

import numpy as np


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def silu(x):
    return x * sigmoid(x)


def dsilu(x):
    s = sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


# ---- short causal convolution

def _live(slot, pool):
    return 0 <= slot < pool


def conv_fwd(x, weight, bias, pool, idx, cu, act):
    """(out, new pool, magnitude of pre, written rows) in fp64; pool None: zero history."""
    x = np.asarray(x, np.float64)
    n, ch = x.shape
    w = weight.shape[1]
    out, mag = np.zeros((n, ch)), np.zeros((n, ch))
    written = np.zeros(n, bool)
    new = None if pool is None else np.array(pool, np.float64)
    for b in range(len(cu) - 1):
        if pool is not None and not _live(idx[b], len(pool)):
            continue
        hist = np.zeros((w - 1, ch)) if pool is None else np.asarray(pool[idx[b]], np.float64)
        u = np.concatenate([hist, x[cu[b]:cu[b + 1]]])
        for p in range(cu[b + 1] - cu[b]):
            out[cu[b] + p] = (weight.T * u[p:p + w]).sum(0)
            mag[cu[b] + p] = np.abs(weight.T * u[p:p + w]).sum(0)
        written[cu[b]:cu[b + 1]] = True
        if new is not None:
            new[idx[b]] = u[len(u) - (w - 1):]
    if bias is not None:
        out, mag = out + bias, mag + np.abs(bias)
    return (silu(out) if act else out), new, mag, written


def conv_bwd(x, weight, bias, pool, idx, cu, dout, dstate, act):
    """dict of dx, dweight, dbias, dstate0 and of their magnitudes (key + "_mag")."""
    x, dout = np.asarray(x, np.float64), np.asarray(dout, np.float64)
    n, ch = x.shape
    w = weight.shape[1]
    nb = len(cu) - 1
    g = {k: np.zeros(s) for k, s in (("dx", (n, ch)), ("dweight", (ch, w)), ("dbias", (ch,)),
                                     ("dstate0", (nb, w - 1, ch)))}
    g.update({k + "_mag": np.zeros_like(v) for k, v in list(g.items())})
    for b in range(nb):
        if pool is not None and not _live(idx[b], len(pool)):
            continue
        hist = np.zeros((w - 1, ch)) if pool is None else np.asarray(pool[idx[b]], np.float64)
        u = np.concatenate([hist, x[cu[b]:cu[b + 1]]])
        du, dm = np.zeros_like(u), np.zeros_like(u)
        for p in range(cu[b + 1] - cu[b]):
            win = u[p:p + w]
            pre = (weight.T * win).sum(0) + (0 if bias is None else bias)
            gm = np.abs(dout[cu[b] + p]) * (
                1.1 + 0.5 * (np.abs(weight.T * win).sum(0) + (0 if bias is None else np.abs(bias))))
            gp = dout[cu[b] + p] * (dsilu(pre) if act else 1.0)
            g["dweight"] += (gp * win).T
            g["dweight_mag"] += (gm * np.abs(win)).T
            g["dbias"] += gp
            g["dbias_mag"] += gm
            du[p:p + w] += weight.T * gp
            dm[p:p + w] += np.abs(weight.T) * gm
        if dstate is not None:
            du[len(u) - (w - 1):] += dstate[b]
            dm[len(u) - (w - 1):] += np.abs(dstate[b])
        g["dstate0"][b], g["dx"][cu[b]:cu[b + 1]] = du[:w - 1], du[w - 1:]
        g["dstate0_mag"][b], g["dx_mag"][cu[b]:cu[b + 1]] = dm[:w - 1], dm[w - 1:]
    return g


# ---- selective state space scan

def ssm(C, B, x, dt, A_log, dt_bias, D, pool, idx, cu):
    """(out, new pool, magnitude of out, magnitude of the states, written rows): the magnitudes
    are the same recurrence over absolute values."""
    C, B, x = (np.asarray(t, np.float64) for t in (C, B, x))
    n, hv, dv = x.shape
    h, dk = B.shape[1:]
    rep = hv // h
    C, B = np.repeat(C, rep, 1), np.repeat(B, rep, 1)
    xg = np.asarray(dt, np.float64) + np.asarray(dt_bias, np.float64)
    step = np.maximum(xg, 0) + np.log1p(np.exp(-np.abs(xg)))
    a = np.exp(-np.exp(np.asarray(A_log, np.float64)) * step)
    new = np.array(pool, np.float64)
    mags = np.abs(new)
    out, mag = np.zeros((n, hv, dv)), np.zeros((n, hv, dv))
    written = np.zeros(n, bool)
    for b in range(len(cu) - 1):
        if not _live(idx[b], len(pool)):
            continue
        s, m = new[idx[b]], mags[idx[b]]
        for t in range(cu[b], cu[b + 1]):
            u = step[t][:, None] * x[t]
            s[:] = a[t][:, None, None] * s + u[:, :, None] * B[t][:, None, :]
            m[:] = a[t][:, None, None] * m + np.abs(u[:, :, None] * B[t][:, None, :])
            out[t] = np.matmul(s, C[t][:, :, None])[..., 0]
            mag[t] = np.matmul(m, np.abs(C[t])[:, :, None])[..., 0]
        written[cu[b]:cu[b + 1]] = True
    if D is not None:
        out += np.asarray(D, np.float64)[None, :, None] * x
        mag += np.abs(np.asarray(D, np.float64)[None, :, None] * x)
    return out, new, mag, mags, written


# ---- gated norm

def _norm(x, z, eps, rms, gate):
    x = np.asarray(x, np.float64)
    sz = None if z is None else silu(np.asarray(z, np.float64))
    u = x * sz if gate == "first" else x
    c = u if rms else u - u.mean(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    return x, u, sz, c * rstd, rstd


def norm_fwd(x, weight, bias, z, eps, rms, gate):
    """(out, magnitude); gate: "none", "last" or "first"."""
    x, u, sz, hat, rstd = _norm(x, z, eps, rms, gate)
    y = hat * weight
    mag = np.abs(weight) * (rstd * (np.abs(u) + np.abs(u).mean(-1, keepdims=True)) + np.abs(hat))
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    if gate == "last":
        y, mag = y * sz, mag * np.abs(sz) + np.abs(y * sz) * (1 + np.abs(z))
    if gate == "first":
        mag = mag * (1 + np.abs(z).max(-1, keepdims=True))
    return y, mag


def norm_bwd(x, weight, bias, z, dout, eps, rms, gate):
    """dict of dx, dz, dweight, dbias."""
    x, u, sz, hat, rstd = _norm(x, z, eps, rms, gate)
    dout = np.asarray(dout, np.float64)
    y = hat * weight + (0 if bias is None else bias)
    dy = dout * sz if gate == "last" else dout
    axes = tuple(range(x.ndim - 1))
    g = {"dweight": (dy * hat).sum(axes), "dbias": dy.sum(axes)}
    g["dweight_mag"] = np.abs(dy * (np.abs(hat) + rstd * np.abs(u).mean(-1, keepdims=True))).sum(axes)
    g["dbias_mag"] = np.abs(dy).sum(axes)
    dhat = dy * weight
    m1 = (dhat * hat).mean(-1, keepdims=True)
    m0 = 0.0 if rms else dhat.mean(-1, keepdims=True)
    du = rstd * (dhat - m0 - hat * m1)
    # rounding of hat (relative to |u| rstd) moves every term that holds it
    lever = 1 + rstd * np.abs(u).max(-1, keepdims=True)
    g["dx_mag"] = rstd * lever ** 2 * (np.abs(dhat) + np.abs(dhat).mean(-1, keepdims=True)
                                       + np.abs(hat) * np.abs(dhat * hat).mean(-1, keepdims=True))
    if gate == "first":
        g["dx"], g["dz"] = du * sz, du * x * dsilu(np.asarray(z, np.float64))
        g["dz_mag"] = g["dx_mag"] * np.abs(x) * (1.1 + np.abs(z))
        g["dx_mag"] = g["dx_mag"] * np.abs(sz) * (1 + np.abs(z)) * (1 + np.abs(z).max(-1, keepdims=True))
        g["dz_mag"] = g["dz_mag"] * (1 + np.abs(z).max(-1, keepdims=True))
    else:
        g["dx"] = du
        if gate == "last":
            g["dz"] = dout * y * dsilu(np.asarray(z, np.float64))
            g["dz_mag"] = np.abs(dout) * (1.1 + np.abs(z)) * (
                np.abs(weight) * (np.abs(hat) + rstd * np.abs(u).mean(-1, keepdims=True))
                + (0 if bias is None else np.abs(bias)))
            g["dx_mag"] = g["dx_mag"] * (1 + np.abs(z).max(-1, keepdims=True))
    return g
