"""Pins of the fp64 oracle of linear attention and of the adapters: closed forms and central
differences."""
import numpy as np
import pytest

from oracle import linear as L


def make(seed, lengths, h=1, hv=2, dk=3, dv=4, pool=True):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(int)
    n, b = int(cu[-1]), len(lengths)
    return dict(q=r.standard_normal((n, h, dk)), k=r.standard_normal((n, h, dk)),
                v=r.standard_normal((n, hv, dv)), log_decay=-r.uniform(0.01, 1, hv), scale=0.7,
                pool=r.standard_normal((b + 1, hv, dv, dk)) if pool else None,
                idx=r.permutation(b + 1)[:b], cu=cu)


def test_forward_is_the_sum_over_earlier_tokens():
    c = make(1, [5, 0, 3], h=2, hv=4)
    out, new, mag, mags, written = L.linear_fwd(**c)
    assert written.all() and (np.abs(out) <= mag + 1e-12).all() and (np.abs(new) <= mags + 1e-12).all()
    for b in range(3):
        lo, hi = c["cu"][b], c["cu"][b + 1]
        for hv in range(4):
            lam, s0 = np.exp(c["log_decay"][hv]), c["pool"][c["idx"][b], hv]
            for t in range(lo, hi):
                want = lam ** (t - lo + 1) * s0 @ c["q"][t, hv // 2]
                for j in range(lo, t + 1):
                    want = want + lam ** (t - j) * (c["q"][t, hv // 2] @ c["k"][j, hv // 2]) * c["v"][j, hv]
                np.testing.assert_allclose(out[t, hv], 0.7 * want, rtol=1e-12, atol=1e-12)
    untouched = (set(range(4)) - set(c["idx"])).pop()
    np.testing.assert_array_equal(new[untouched], c["pool"][untouched])


def test_decays_of_zero_and_above_one():
    c = make(2, [4])
    c["log_decay"] = np.array([-np.inf, 3.0])
    out, new, *_ = L.linear_fwd(**c)
    for t in range(4):  # nothing is kept, everything is kept
        np.testing.assert_allclose(out[t, 0], 0.7 * (c["q"][t, 0] @ c["k"][t, 0]) * c["v"][t, 0])
    np.testing.assert_allclose(new[c["idx"][0], 1], c["pool"][c["idx"][0], 1]
                               + np.einsum("ti,tj->ij", c["v"][:, 1], c["k"][:, 0]))


@pytest.mark.parametrize("pool", [True, False])
def test_gradients_by_differences(pool):
    c = make(3, [4, 0, 3], h=1, hv=2, pool=pool)
    r = np.random.default_rng(4)
    dout = r.standard_normal(c["v"].shape)
    dstate = r.standard_normal((3, 2, 4, 3)) if pool else None

    def loss(c):
        out, new, *_ = L.linear_fwd(**c)
        return (dout * out).sum() + (0 if new is None else (dstate * new[c["idx"]]).sum())

    g = L.linear_bwd(**c, dout=dout, dstate=dstate)
    for name in ("q", "k", "v"):
        d = r.standard_normal(c[name].shape)
        up, down = ({**c, name: c[name] + s * 1e-4 * d} for s in (1, -1))
        np.testing.assert_allclose((loss(up) - loss(down)) / 2e-4, (g["d" + name] * d).sum(), rtol=1e-8)
        assert (np.abs(g["d" + name]) <= g["d" + name + "_mag"] + 1e-12).all()
    if pool:
        d = np.zeros_like(c["pool"])
        d[c["idx"]] = r.standard_normal((3, 2, 4, 3))
        up, down = ({**c, "pool": c["pool"] + s * 1e-4 * d} for s in (1, -1))
        np.testing.assert_allclose((loss(up) - loss(down)) / 2e-4, (g["dstate0"] * d[c["idx"]]).sum(), rtol=1e-8)


def test_padding_requests_are_left_alone():
    c = make(5, [3, 2])
    c["idx"] = np.array([7, 0])
    out, new, _, _, written = L.linear_fwd(**c)
    assert list(written) == [False] * 3 + [True] * 2 and (out[:3] == 0).all()
    g = L.linear_bwd(**c, dout=np.ones_like(c["v"]), dstate=np.ones((2, 2, 4, 3)))
    assert (g["dstate0"][0] == 0).all() and (g["dq"][:3] == 0).all() and (g["dstate0"][1] != 0).any()


def test_adapters_are_a_change_of_the_weight():
    r = np.random.default_rng(6)
    x, w = r.standard_normal((6, 5)), r.standard_normal((7, 5))
    A, B, s = r.standard_normal((2, 3, 5)), r.standard_normal((2, 7, 3)), np.array([0.5, -2.0])
    out, mag, written = L.adapter(x, x @ w.T, A, B, s, [1, -1, 0], [0, 2, 3, 5])
    np.testing.assert_allclose(out[:2], x[:2] @ (w - 2 * B[1] @ A[1]).T)
    np.testing.assert_allclose(out[2], x[2] @ w.T)
    np.testing.assert_allclose(out[3:5], x[3:5] @ (w + 0.5 * B[0] @ A[0]).T)
    assert list(written) == [True] * 5 + [False] and (np.abs(out) <= mag + 1e-12).all()
