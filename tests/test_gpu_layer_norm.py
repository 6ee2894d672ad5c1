"""The gated layer / RMS norm and its gradients against the fp64 oracle.

Tolerances, derived: u = 2^-24. Every sum over a row runs through at most 16 additions per thread
and 10 levels across threads (mean, variance, and in the backward two more), so mean, rstd and
the two means of the gradient carry at most 26 u of their terms' magnitudes, twice that where one
enters the other; products, the square root and the gate's sigmoid (8 + 2 |z| steps) stay below
the rest of 80 u. The oracle's magnitudes hold those sums. One rounding to the output type.
dweight and dbias add one u per addition of the longest chain: the rows of a workgroup's loop,
its row groups, and the workgroups' partial rows."""
import numpy as np
import pytest

from layer_util import DEV, HALF, U32, f32, rounded, strided, within
from oracle import layer as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

K = 80 * U32
DIMS = [1, 2, 7, 8, 24, 64, 100, 128, 129, 256, 511, 512, 520, 1000, 1024, 2047, 2048, 2056, 4096,
        4097, 8192, 16384]
MODES = [(True, "last", False), (False, "none", True), (True, "none", False), (False, "last", True),
         (True, "first", True), (False, "first", False)]


def make(seed, n, heads, dim, dtype, bias, gate, pad=0, offset=0, scale=1.5, mean=0.3):
    r = np.random.default_rng(seed)
    c = {}
    c["x"], c["x64"] = rounded(scale * r.standard_normal((n, heads, dim)) + mean, dtype)
    c["z"], c["z64"] = rounded(2 * r.standard_normal((n, heads, dim)), dtype) if gate != "none" else (None, None)
    if pad or offset:
        c["x"] = strided(c["x"], pad, offset)
        c["z"] = None if c["z"] is None else strided(c["z"], pad + 16, offset)
    c["weight"], c["weight64"] = f32(1 + 0.3 * r.standard_normal(dim))
    c["bias"], c["bias64"] = f32(0.3 * r.standard_normal(dim)) if bias else (None, None)
    return c


def check(c, dtype, rms, gate, what, eps=1e-5, backward=True):
    import gated_deltanet_prefill_gdn_amd as gdn
    kw = dict(eps=eps, rms=rms, gate_first=gate == "first")
    n, heads, dim = c["x"].shape
    out = gdn.gdn_norm_fwd(c["x"], c["weight"], c["bias"], c["z"], **kw)
    torch.cuda.synchronize()
    e32 = float(np.float32(eps))
    ref, mag = L.norm_fwd(c["x64"], c["weight64"], c["bias64"], c["z64"], e32, rms, gate)
    h = HALF[dtype]
    within(out, ref, h * np.abs(ref) + (1 + h) * K * mag + 1e-38, what)
    if not backward:
        return out
    r = np.random.default_rng(5)
    dout, dout64 = rounded(r.standard_normal((n, heads, dim)), dtype)
    g = gdn.gdn_norm_bwd(c["x"], c["weight"], c["bias"], c["z"], dout, **kw)
    torch.cuda.synchronize()
    ref = L.norm_bwd(c["x64"], c["weight64"], c["bias64"], c["z64"], dout64, e32, rms, gate)
    assert set(g) == ({"dx", "dweight"} | ({"dz"} if gate != "none" else set())
                      | ({"dbias"} if c["bias"] is not None else set()))
    for k in ("dx", "dz"):
        if k in g:
            within(g[k], ref[k], h * np.abs(ref[k]) + (1 + h) * K * ref[k + "_mag"] + 1e-38, f"{what} {k}")
    # rows of a workgroup's loop, at most 32 row groups, partial rows added 16 chains wide
    chain = 80 + n * heads / 256 + 32 + 1024 / 16
    zmax = 1.0 if gate == "none" else 1 + float(np.abs(c["z64"]).max())
    for k in ("dweight", "dbias"):
        if k in g:
            within(g[k], ref[k], U32 * (chain + 10 * zmax) * zmax * ref[k + "_mag"] + 1e-38, f"{what} {k}")
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", DIMS)
def test_norm_row_lengths(dtype, dim):
    rms, gate, bias = MODES[dim % len(MODES)]
    heads = 3 if dim <= 512 else 1
    c = make(dim, 19, heads, dim, dtype, bias, gate)
    check(c, dtype, rms, gate, f"norm {dtype} d={dim} rms={rms} gate={gate}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", range(len(MODES)))
@pytest.mark.parametrize("n,heads,dim", [(1, 1, 128), (41, 32, 128), (700, 4, 64), (5, 1, 3000), (130, 1, 1023)])
def test_norm_modes(dtype, mode, n, heads, dim):
    rms, gate, bias = MODES[mode]
    check(make(7 + mode, n, heads, dim, dtype, bias, gate), dtype, rms, gate,
          f"norm {dtype} {n}x{heads}x{dim} rms={rms} gate={gate}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 8), (32, 0), (5, 0), (8, 3)])
def test_norm_strides(dtype, pad, offset):
    check(make(3, 21, 4, 128, dtype, False, "last", pad, offset), dtype, True, "last",
          f"norm strided {dtype} +{pad} @{offset}")


def test_norm_gate_gradient_into_a_wider_row():
    import gated_deltanet_prefill_gdn_amd as gdn
    c = make(4, 9, 2, 64, "bf16", False, "last")
    dout = torch.randn(9, 2, 64, device=DEV).bfloat16()
    wide = torch.full((9, 200), 7.5, dtype=torch.bfloat16, device=DEV)
    g = gdn.gdn_norm_bwd(c["x"], c["weight"], None, c["z"], dout, dz=wide[:, 8:136].unflatten(1, (2, 64)))
    h = gdn.gdn_norm_bwd(c["x"], c["weight"], None, c["z"], dout)
    torch.cuda.synchronize()
    assert torch.equal(g["dz"], h["dz"]) and (wide[:, :8] == 7.5).all() and (wide[:, 136:] == 7.5).all()


def test_norm_far_from_zero_and_constant_rows():
    """A mean a thousand deviations away costs a layer norm digits only as its magnitude says; a
    constant row gives the bias."""
    check(make(6, 10, 1, 777, "f32", True, "none", mean=1000.0, scale=1.0), "f32", False, "none",
          "norm far mean", backward=False)
    c = make(6, 3, 1, 96, "f32", True, "none")
    c["x"].fill_(4.0)
    import gated_deltanet_prefill_gdn_amd as gdn
    out = gdn.gdn_norm_fwd(c["x"], c["weight"], c["bias"], rms=False)
    assert torch.equal(out, c["bias"].expand_as(out))


def test_norm_bad_rows_stay_alone():
    import gated_deltanet_prefill_gdn_amd as gdn
    c = make(8, 50, 2, 64, "f32", False, "last")
    ref = gdn.gdn_norm_fwd(c["x"], c["weight"], None, c["z"])
    c["x"][3, 1, 5], c["x"][20, 0, 0], c["z"][30, 1, 2] = float("nan"), float("inf"), float("nan")
    out = gdn.gdn_norm_fwd(c["x"], c["weight"], None, c["z"])
    keep = torch.ones(50, 2, dtype=torch.bool, device=DEV)
    keep[3, 1] = keep[20, 0] = keep[30, 1] = False
    assert torch.equal(out[keep], ref[keep])
    assert torch.isnan(out[3, 1]).all() and torch.isnan(out[30, 1]).sum() == 1


def test_norm_backward_without_rows_and_twice():
    import gated_deltanet_prefill_gdn_amd as gdn
    e = torch.empty(0, 2, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    g = gdn.gdn_norm_bwd(e, w, w, None, e)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
    c = make(9, 3000, 4, 128, "bf16", True, "last")
    dout = torch.randn(3000, 4, 128, device=DEV).bfloat16()
    a, b = (gdn.gdn_norm_bwd(c["x"], c["weight"], c["bias"], c["z"], dout) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)
