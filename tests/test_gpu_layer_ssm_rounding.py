"""bf16 outputs of the scan carry one rounding to bf16, whole and cut requests alike, at every state
size (requests of more than 512 tokens are cut in all of these shapes).

Tolerance, derived, with M the recurrence over absolute values. Inputs enter the products as they
are. Decayed scores, the state that S C reads and the decayed x of a piece's state are sums of two
bf16: what two leave off is at most 2^-16 of a value, and a term meets two of them at most (the
decayed x, then the state), 2^-15 M. Gates and fp32 sums take 2^-16 M, as in the states. Then the
output's own rounding, 2^-8 of the value."""
import numpy as np
import pytest

from layer_util import HALF, np64, within
from oracle import layer as L
from test_gpu_layer_ssm import call, check, make

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

INNER = 1.5 * 2.0 ** -15


def check_rounding(c, out, what):
    ref, _, mag, _, written = L.ssm(c["C64"], c["B64"], c["x64"], c["dt64"], c["A_log64"],
                                    c["dt_bias64"], c["D64"], c["pool64"], c["idx"], c["cu"])
    h = HALF["bf16"]
    within(np64(out)[written], ref[written], (h * np.abs(ref) + (1 + h) * INNER * mag + 1e-38)[written],
           what + ", one rounding")


SHAPES = [(1, 2, 128, 64), (2, 2, 64, 64), (1, 3, 64, 64), (2, 4, 128, 128), (1, 1, 64, 256),
          (1, 2, 256, 64), (1, 1, 256, 256)]


@pytest.mark.parametrize("h,hv,dk,dv", SHAPES)
@pytest.mark.parametrize("lengths", [[150, 1, 70], [1300, 20, 700]], ids=["whole", "cut"])
@pytest.mark.parametrize("dt_mean,a_hi", [(-3.0, 16.0), (-6.0, 2.0)], ids=["fast", "slow"])
def test_bf16_outputs_are_rounded_once(h, hv, dk, dv, lengths, dt_mean, a_hi):
    c = make(21 + dk + dv, lengths, h, hv, dk, dv, "bf16", D=False, dt_mean=dt_mean, a_hi=a_hi)
    out, pool = call(c)
    what = f"ssm {lengths} H={h} HV={hv} dk={dk} dv={dv}"
    check(c, "bf16", out, pool, what)
    check_rounding(c, out, what)
