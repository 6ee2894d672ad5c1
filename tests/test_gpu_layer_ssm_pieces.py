"""Requests that are cut into pieces, at the state sizes whose kernels are compiled apart: states of
pieces, their join, and outputs from a start state, with pieces in one part and in four."""
import numpy as np
import pytest

from layer_util import DEV, DT, np64
from test_gpu_layer_ssm import call, check, make
from test_gpu_layer_ssm_rounding import check_rounding

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,hv,dv", [(1, 2, 64), (2, 2, 256)])
@pytest.mark.parametrize("dt_mean,a_hi", [(-7.0, 1.5), (0.5, 16.0)], ids=["slow", "fast"])
def test_pieces_at_a_state_size_of_256(dtype, h, hv, dv, dt_mean, a_hi):
    """Pieces whose states all reach the request's end, and pieces of which none does."""
    c = make(22, [1300, 20, 700], h, hv, 256, dv, dtype, dt_mean=dt_mean, a_hi=a_hi)
    out, pool = call(c)
    check(c, dtype, out, pool, f"ssm {dtype} pieces dk=256 dv={dv}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv,hv", [(256, 64, 256), (128, 64, 256), (128, 256, 64)])
def test_four_parts_of_a_piece_at_large_state_sizes(dtype, dk, dv, hv):
    """Pieces of more than 4096 tokens, whose states are formed in four parts, beside a request
    that is not cut. Heads do not mix, so the recurrence of a few of them is enough."""
    g = torch.Generator(device=DEV).manual_seed(dk + dv)
    rn = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    lengths, heads = [40, 15999], [0, 1, hv - 1] if dv == 64 else [0, hv - 1]
    n = sum(lengths)
    a_log = torch.full((hv,), 4.0, device=DEV)
    a_log[heads] = torch.tensor([-4.0, 2.0, 4.6][:len(heads)], device=DEV)
    c = dict(C=(0.6 * rn(n, 1, dk)).to(DT[dtype]), B=(0.6 * rn(n, 1, dk)).to(DT[dtype]),
             x=(0.8 * rn(n, hv, dv)).to(DT[dtype]), dt=rn(n, hv), A_log=a_log,
             dt_bias=rn(hv) - 3, D=None, pool=0.3 * rn(2, hv, dv, dk), idx=np.array([1, 0]),
             cu=np.concatenate([[0], np.cumsum(lengths)]).astype(int))
    out, pool = call(c)
    few = {k: c[k][:, heads] for k in ("x", "dt", "pool")}
    few.update({k: c[k][heads] for k in ("A_log", "dt_bias")}, C=c["C"], B=c["B"])
    for k, v in few.items():
        c[k], c[k + "64"] = v, np64(v)
    c["D64"] = None
    what = f"ssm {dtype} {lengths} HV={hv} dk={dk} dv={dv}"
    check(c, dtype, out[:, heads], pool[:, heads], what)
    if dtype == "bf16":
        check_rounding(c, out[:, heads], what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[1, 0, 700, 3] + [1] * 150, [1] * 150 + [300]], ids=["chunks", "tokens"])
def test_one_prompt_beside_many_single_tokens(dtype, lengths):
    """So many requests that none is cut: the single tokens in chunks, or, where the mean length says
    so, token by token."""
    c = make(23, lengths, 8, 64, 64, 64, dtype)
    out, pool = call(c)
    what = f"ssm {dtype} {max(lengths)} tokens beside single ones"
    check(c, dtype, out, pool, what)
    if dtype == "bf16":
        check_rounding(c, out, what)
