"""Decays that differ by orders of magnitude between a chunk's tokens, and decays beyond the range of
fp32, whose sums must not overflow into differences of infinities. Bounds as in
test_gpu_layer_ssm_rounding and test_gpu_layer_ssm."""
import numpy as np
import pytest

from layer_util import f32
from test_gpu_layer_ssm import call, check, make
from test_gpu_layer_ssm_rounding import check_rounding

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("high", [3.0, 40.0])
@pytest.mark.parametrize("hv,dk,dv", [(2, 128, 64), (1, 64, 128), (1, 256, 256)])
@pytest.mark.parametrize("lengths", [[200, 1, 65], [1300, 20]], ids=["whole", "cut"])
def test_tokens_that_erase_among_tokens_that_keep(dtype, high, hv, dk, dv, lengths):
    """Every third token erases the state and writes, the ones between hardly change it: sums of
    logs run into the thousands while the differences that matter stay below one."""
    c = make(41, lengths, 1, hv, dk, dv, dtype, D=False)
    n = sum(lengths)
    dt = np.where(np.arange(n)[:, None] % 3 == 0, high, -6.0) + 0.1 * c["dt64"]
    c["dt"], c["dt64"] = f32(dt)
    c["dt_bias"], c["dt_bias64"] = f32(np.zeros(hv))
    c["A_log"], c["A_log64"] = f32(np.log(np.linspace(16, 12, hv)))
    out, pool = call(c)
    what = f"ssm {dtype} erasing tokens {high} {lengths} HV={hv} dk={dk} dv={dv}"
    check(c, dtype, out, pool, what)
    if dtype == "bf16":
        check_rounding(c, out, what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("a_log", [80.0, 87.0, 95.0])
@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 128), (256, 256)])
@pytest.mark.parametrize("lengths", [[200, 1, 65], [1300, 20]], ids=["whole", "cut"])
def test_decays_beyond_the_range_of_fp32(dtype, a_log, dk, dv, lengths):
    """exp(A_log) next to the largest float, and infinite: every token erases the state before it."""
    c = make(42, lengths, 1, 2, dk, dv, dtype, D=False, dt_mean=1.0)
    c["A_log"], c["A_log64"] = f32([a_log, 1.0])
    out, pool = call(c)
    check(c, dtype, out, pool, f"ssm {dtype} A_log {a_log} {lengths} dk={dk} dv={dv}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decode", [False, True])
def test_steps_of_zero_under_infinite_rates(dtype, decode):
    """exp(A_log) above the largest float, and steps that underflow: such a token keeps the state."""
    lengths = [1] * 6 if decode else [70, 3]
    c = make(43, lengths, 1, 2, 64, 64, dtype, D=False)
    dt = np.where(np.arange(sum(lengths))[:, None] % 2 == 1, -200.0, c["dt64"])
    c["dt"], c["dt64"] = f32(dt)
    c["A_log"], c["A_log64"] = f32([95.0, 2.0])
    out, pool = call(c, decode=decode)
    check(c, dtype, out, pool, f"ssm {dtype} zero steps decode={decode}")
