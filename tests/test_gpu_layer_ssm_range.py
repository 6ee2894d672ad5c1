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
