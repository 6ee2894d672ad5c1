"""Pins of the layer operators' oracle: gradients against central differences of its own
forward, the convolution against numpy's, the scan against its closed forms, the norm against
the moments it sets."""
import numpy as np
import pytest

from oracle import layer as L

CU = [0, 0, 1, 3, 9]
IDX = [2, 0, 4, 1]


def _conv_case(w, seed=0):
    r = np.random.default_rng(seed)
    ch = 5
    return dict(x=r.standard_normal((9, ch)), weight=r.standard_normal((ch, w)),
                bias=r.standard_normal(ch), pool=r.standard_normal((5, w - 1, ch)))


@pytest.mark.parametrize("w", [2, 3, 4])
def test_conv_forward_and_state(w):
    c = _conv_case(w)
    out, new, _, written = L.conv_fwd(c["x"], c["weight"], c["bias"], c["pool"], IDX, CU, False)
    assert written.all()
    for b in range(4):
        u = np.concatenate([c["pool"][IDX[b]], c["x"][CU[b]:CU[b + 1]]])
        np.testing.assert_array_equal(new[IDX[b]], u[len(u) - w + 1:])
        for k in range(5):
            ref = np.convolve(u[:, k], c["weight"][k, ::-1], "valid") + c["bias"][k]
            np.testing.assert_allclose(out[CU[b]:CU[b + 1], k], ref[:CU[b + 1] - CU[b]], atol=1e-13)
    np.testing.assert_array_equal(new[3], c["pool"][3])
    # a slot outside the pool: a padding request
    out, new, _, written = L.conv_fwd(c["x"], c["weight"], None, c["pool"], [2, 0, -1, 5], CU, True)
    assert list(written) == [True] + [False] * 8
    np.testing.assert_array_equal(new[[1, 3, 4]], c["pool"][[1, 3, 4]])


def _check_gradient(f, values, grads, seed, eps=1e-6):
    """Directional central differences of f at every tensor of `values`."""
    r = np.random.default_rng(seed)
    for k, g in grads.items():
        d = r.standard_normal(values[k].shape)
        hi, lo = (f(**{**values, k: values[k] + s * eps * d}) for s in (1, -1))
        np.testing.assert_allclose((hi - lo) / (2 * eps), (g * d).sum(), rtol=2e-7, atol=2e-7)


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("w", [2, 3, 4])
def test_conv_gradient_is_that_of_the_forward(w, act):
    c = _conv_case(w, 3)
    r = np.random.default_rng(4)
    dout, dstate = r.standard_normal((9, 5)), r.standard_normal((4, w - 1, 5))

    def loss(x, weight, bias, pool):
        out, new, _, _ = L.conv_fwd(x, weight, bias, pool, IDX, CU, act)
        return (out * dout).sum() + (new[IDX] * dstate).sum()

    g = L.conv_bwd(c["x"], c["weight"], c["bias"], c["pool"], IDX, CU, dout, dstate, act)
    dpool = np.zeros_like(c["pool"])
    dpool[IDX] = g["dstate0"]
    _check_gradient(loss, c, dict(x=g["dx"], weight=g["dweight"], bias=g["dbias"], pool=dpool), 5)


def test_scan_closed_forms():
    r = np.random.default_rng(6)
    n, hv, dv, dk = 7, 2, 3, 4
    C, B, x = r.standard_normal((n, 1, dk)), r.standard_normal((n, 1, dk)), r.standard_normal((n, hv, dv))
    dt, bias, D = r.standard_normal((n, hv)), r.standard_normal(hv), r.standard_normal(hv)
    pool = r.standard_normal((3, hv, dv, dk))
    step = np.log1p(np.exp(dt + bias))
    # no decay: a plain sum of outer products
    out, new, mag, mags, _ = L.ssm(C, B, x, dt, np.full(hv, -np.inf), bias, D, pool, [1], [0, n])
    ref = pool[1] + np.einsum("th,thi,tj->hij", step, x, B[:, 0])
    np.testing.assert_allclose(new[1], ref, rtol=1e-12)
    np.testing.assert_array_equal(new[[0, 2]], pool[[0, 2]])
    # the last token's output reads the final state
    np.testing.assert_allclose(out[-1], ref @ C[-1, 0] + D[:, None] * x[-1], rtol=1e-11)
    assert (mags[1] >= np.abs(new[1]) - 1e-12).all() and (mag >= np.abs(out) - 1e-12).all()
    # decayed attention over the tokens
    A = r.uniform(0, 1, hv)
    out, _, _, _, _ = L.ssm(C, B, x, dt, A, bias, None, 0 * pool, [1], [0, n])
    g = np.cumsum(-np.exp(A) * step, 0)
    w = np.exp(np.minimum(g[:, None] - g[None], 0)) * np.tril(np.ones((n, n)))[:, :, None]
    ref = np.einsum("ij,ijh,jh,jhd->ihd", C[:, 0] @ B[:, 0].T, w, step, x)
    np.testing.assert_allclose(out, ref, rtol=1e-10, atol=1e-12)
    # strong decay and large steps leave the last token alone; a step of zero leaves the state
    out, new, _, _, _ = L.ssm(C, B, x, dt + 60, np.full(hv, 3.0), bias, None, pool, [0], [0, n])
    np.testing.assert_allclose(new[0], ((dt[-1] + 60 + bias)[:, None] * x[-1])[..., None] * B[-1], rtol=1e-12)
    _, new, _, _, _ = L.ssm(C, B, x, dt - 1e4, A, bias, None, pool, [2], [0, n])
    np.testing.assert_array_equal(new, pool)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_moments(rms):
    r = np.random.default_rng(7)
    x = 3 + 2 * r.standard_normal((4, 2, 50))
    y, _ = L.norm_fwd(x, np.ones(50), None, None, 0.0, rms, "none")
    np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-12)
    if not rms:
        np.testing.assert_allclose(y.mean(-1), 0, atol=1e-13)


@pytest.mark.parametrize("gate", ["none", "last", "first"])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradient_is_that_of_the_forward(rms, gate):
    r = np.random.default_rng(8)
    v = dict(x=r.standard_normal((4, 2, 9)) + 0.5, weight=r.standard_normal(9),
             bias=r.standard_normal(9), z=r.standard_normal((4, 2, 9)))
    dout = r.standard_normal((4, 2, 9))

    def loss(x, weight, bias, z):
        return (L.norm_fwd(x, weight, bias, z if gate != "none" else None, 1e-2, rms, gate)[0]
                * dout).sum()

    g = L.norm_bwd(v["x"], v["weight"], v["bias"], v["z"] if gate != "none" else None, dout, 1e-2,
                   rms, gate)
    _check_gradient(loss, v, {k[1:]: g[k] for k in ("dx", "dweight", "dbias", "dz") if k in g}, 9)
