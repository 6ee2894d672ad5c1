"""Finite values beyond the largest bf16 (3.39e38): the scan takes fp32 values as sums of bf16, and
none of the parts may overflow. Bounds as in test_gpu_layer_ssm, relative to the recurrence over
absolute values."""
import numpy as np
import pytest

from layer_util import f32, rounded
from test_gpu_layer_ssm import call, check, make

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TOP = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("lengths", [[70, 1], [1300, 20]], ids=["whole", "cut"])
@pytest.mark.parametrize("hv,dk,dv", [(2, 128, 64), (1, 64, 128), (1, 256, 256)])
def test_large_inputs(lengths, hv, dk, dv):
    """fp32 x up to the largest float; B and C so small that states and outputs are far below it."""
    c = make(31, lengths, 1, hv, dk, dv, "f32", D=False)
    x = c["x64"].copy()
    x[::7] = np.sign(x[::7]) * TOP
    c["x"], c["x64"] = f32(x)
    c["B"], c["B64"] = f32(c["B64"] * 2.0 ** -70)
    c["C"], c["C64"] = f32(c["C64"] * 2.0 ** -20)
    out, pool = call(c)
    check(c, "f32", out, pool, f"ssm large x {lengths} HV={hv} dk={dk} dv={dv}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[70, 1], [1300, 20]], ids=["whole", "cut"])
@pytest.mark.parametrize("hv,dk,dv", [(2, 128, 64), (1, 64, 128), (1, 256, 256)])
def test_large_states(dtype, lengths, hv, dk, dv):
    """Start states up to the largest float under decays next to one, read by small C."""
    c = make(32, lengths, 1, hv, dk, dv, dtype, D=False, dt_mean=-20.0, a_hi=1.5)
    pool = c["pool64"].copy()
    pool[..., ::5] = np.sign(pool[..., ::5]) * TOP
    c["pool"], c["pool64"] = f32(pool)
    c["C"], c["C64"] = rounded(c["C64"] * 2.0 ** -40, dtype)
    out, new = call(c)
    check(c, dtype, out, new, f"ssm large states {dtype} {lengths} HV={hv} dk={dk} dv={dv}")


@pytest.mark.parametrize("hv,dk,dv", [(2, 64, 64), (2, 128, 64), (1, 128, 128), (1, 256, 256)])
def test_f32_products_do_not_lean_to_one_side(hv, dk, dv):
    """Start states read by C, all positive, under decays next to one: the mean error of the outputs
    is at most the half step of fp32, 2^-25, that one kind of rounding can lean by. Products of
    second and third parts, which are left out, are at most 2^-8 2^-17 of a product and of either
    sign where parts are rounded; were they cut off, up to 2^-7 2^-15 and all of one sign."""
    from oracle import layer as L
    c = make(33, [150, 70], 1, hv, dk, dv, "f32", D=False, dt_mean=-30.0, a_hi=1.5)
    r = np.random.default_rng(34)
    for k, shape in (("pool", c["pool"].shape), ("C", c["C"].shape)):
        c[k], c[k + "64"] = f32(r.uniform(1, 2, shape))
    out, pool = call(c)
    check(c, "f32", out, pool, f"ssm positive HV={hv} dk={dk} dv={dv}")
    ref = L.ssm(c["C64"], c["B64"], c["x64"], c["dt64"], c["A_log64"], c["dt_bias64"], None,
                c["pool64"], c["idx"], c["cu"])[0]
    lean = float(((out.double().cpu().numpy() - ref) / ref).mean())
    print(f"[layer] mean error {lean:.2e}", flush=True)
    assert abs(lean) <= 2.0 ** -25
