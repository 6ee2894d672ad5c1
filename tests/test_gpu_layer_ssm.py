"""The selective state space scan and its single-token form against the fp64 recurrence.

Tolerances, derived. Let M be the same recurrence over absolute values (the oracle's magnitudes):
any evaluation that rounds the factors of its products by a relative r is off by at most about
r M. States are fp32 and every factor of their sums is split into three bf16, 2^-24 off: 2^-16 M
leaves room for the gates (steps of 2^-24, exponents below 128 steps, so 2^-17) and the fp32 sums.
Outputs: for bf16 inputs the decayed scores and the start state enter the matrix products
as bf16 (2^-8 each, and their own factors below that), so 2^-8 M + 2^-9 M; for fp32 inputs
2^-15 M. Then one rounding to the output type."""
import numpy as np
import pytest

from layer_util import DEV, HALF, f32, i64, np64, rounded, within
from oracle import layer as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

OUT = {"bf16": 1.5 * 2.0 ** -8, "f32": 2.0 ** -15}
STATE = 2.0 ** -16


def make(seed, lengths, h, hv, dk, dv, dtype, D=True, extra=2, dead=(), dt_mean=-3.0, a_hi=16.0, s0=0.3):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(int)
    n, b = int(cu[-1]), len(lengths)
    c = dict(cu=cu)
    for k, shape, s in (("C", (n, h, dk), 0.6), ("B", (n, h, dk), 0.6), ("x", (n, hv, dv), 0.8)):
        c[k], c[k + "64"] = rounded(s * r.standard_normal(shape) + 0.1, dtype)
    c["dt"], c["dt64"] = f32(r.standard_normal((n, hv)))
    c["A_log"], c["A_log64"] = f32(np.log(r.uniform(1, a_hi, hv)))
    c["dt_bias"], c["dt_bias64"] = f32(dt_mean + r.standard_normal(hv))
    c["D"], c["D64"] = f32(1 + 0.2 * r.standard_normal(hv)) if D else (None, None)
    c["pool"], c["pool64"] = f32(s0 * r.standard_normal((b + extra, hv, dv, dk)))
    c["idx"] = r.permutation(b + extra)[:b]
    for k, v in dead:
        c["idx"][k] = v
    return c


def call(c, decode=False, **kw):
    import gated_deltanet_prefill_gdn_amd as gdn
    pool = c["pool"].clone()
    out = torch.full(c["x"].shape, 7.5, dtype=c["x"].dtype, device=DEV)
    args = (c["C"], c["B"], c["x"], c["dt"], c["A_log"], c["dt_bias"], c["D"], pool, i64(c["idx"]))
    if decode:
        gdn.gdn_ssm_decode_fwd(*args, out=out, **kw)
    else:
        gdn.gdn_ssm_prefill_fwd(*args, i64(c["cu"]), out=out, **kw)
    torch.cuda.synchronize()
    return out, pool


def check(c, dtype, out, pool, what):
    ref, new, mag, mags, written = L.ssm(c["C64"], c["B64"], c["x64"], c["dt64"], c["A_log64"],
                                         c["dt_bias64"], c["D64"], c["pool64"], c["idx"], c["cu"])
    got, h = np64(out), HALF[dtype]
    assert (got[~written] == 7.5).all(), "a padding row was written"
    within(got[written], ref[written], (h * np.abs(ref) + (1 + h) * OUT[dtype] * mag + 1e-38)[written], what)
    within(pool, new, STATE * mags + 1e-38, what + " state")
    touched = [s for s, n in zip(c["idx"], np.diff(c["cu"])) if n and 0 <= s < len(new)]
    for s in set(range(len(new))) - set(touched):
        np.testing.assert_array_equal(pool[s].cpu().numpy(), c["pool"][s].cpu().numpy())


LENGTHS = {
    "one": [1], "chunk": [64], "edges": [63, 65, 1, 0, 128, 127, 2], "ragged": [200, 0, 31, 333, 17],
    "long": [1500, 700], "zero": [0, 0, 5, 0],
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("h,hv,dk,dv", [(1, 2, 128, 64), (2, 2, 64, 64), (1, 3, 64, 128), (2, 4, 128, 128)])
def test_ssm_prefill(dtype, lengths, h, hv, dk, dv):
    c = make(len(lengths) + hv, LENGTHS[lengths], h, hv, dk, dv, dtype, D=hv != 3)
    out, pool = call(c)
    check(c, dtype, out, pool, f"ssm {dtype} {lengths} H={h} HV={hv} dk={dk} dv={dv}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(256, 64), (64, 256), (256, 128), (128, 256), (256, 256)])
def test_ssm_wide_heads(dtype, dk, dv):
    c = make(dk + dv, [150, 1, 70], 1, 2, dk, dv, dtype)
    out, pool = call(c)
    check(c, dtype, out, pool, f"ssm {dtype} dk={dk} dv={dv}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,hv", [(1, 64), (3, 15), (8, 8)])
def test_ssm_many_heads_and_requests(dtype, h, hv):
    r = np.random.default_rng(3)
    c = make(5, list(r.integers(0, 90, 24)), h, hv, 64, 64, dtype)
    out, pool = call(c)
    check(c, dtype, out, pool, f"ssm {dtype} 24 requests H={h} HV={hv}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_one_long_request(dtype):
    """One request on few heads: long enough to be cut into pieces that are joined again, with
    states that live over thousands of tokens."""
    c = make(8, [5003], 1, 2, 128, 64, dtype, dt_mean=-6.0, a_hi=2.0)
    out, pool = call(c)
    check(c, dtype, out, pool, f"ssm {dtype} 5003 tokens, slow decay")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,hv,dv", [([8960, 40], 256, 64), ([40, 15999], 64, 256)])
def test_ssm_long_pieces(dtype, lengths, hv, dv):
    """Pieces of thousands of tokens, whose states are formed in parts: heads that forget within a
    few tokens beside heads that never do, in one workgroup where heads are narrow. Heads do not
    mix, so the recurrence of a few of them is enough."""
    from layer_util import DT
    g = torch.Generator(device=DEV).manual_seed(len(lengths) + hv)
    rn = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    n, dk, heads = sum(lengths), 64, [0, 1, hv // 2, hv - 1]
    a_log = torch.full((hv,), 4.0, device=DEV)
    a_log[heads] = torch.tensor([-4.0, 4.6, 0.0, 2.0], device=DEV)
    c = dict(C=(0.6 * rn(n, 1, dk)).to(DT[dtype]), B=(0.6 * rn(n, 1, dk)).to(DT[dtype]),
             x=(0.8 * rn(n, hv, dv)).to(DT[dtype]), dt=rn(n, hv), A_log=a_log,
             dt_bias=rn(hv) - 3, D=rn(hv), pool=0.3 * rn(2, hv, dv, dk), idx=np.array([1, 0]),
             cu=np.concatenate([[0], np.cumsum(lengths)]).astype(int))
    out, pool = call(c)
    few = {k: c[k][:, heads] for k in ("x", "dt", "pool")}
    few.update({k: c[k][heads] for k in ("A_log", "dt_bias", "D")}, C=c["C"], B=c["B"])
    for k, v in few.items():
        c[k], c[k + "64"] = v, np64(v)
    check(c, dtype, out[:, heads], pool[:, heads], f"ssm {dtype} {lengths} HV={hv} dv={dv}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dt_mean,a_hi", [(3.0, 16.0), (30.0, 2.0), (-90.0, 16.0), (-12.0, 1.0)])
def test_ssm_gates_at_their_ends(dtype, dt_mean, a_hi):
    """Decays that erase the state in one token, steps that vanish, decays next to one."""
    c = make(9, [130, 70], 1, 2, 64, 64, dtype, dt_mean=dt_mean, a_hi=a_hi + 0.01)
    out, pool = call(c)
    check(c, dtype, out, pool, f"ssm {dtype} dt {dt_mean}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_padding_requests_rows_and_nan(dtype):
    """Requests without a slot and rows behind the last request hold NaN and infinities: nobody
    reads or writes them, though they share chunks and tiles with live ones."""
    c = make(10, [70, 33, 50, 1, 90], 1, 2, 128, 64, dtype, dead=((1, -1), (3, 7), (4, 1 << 40)))
    bad = float("nan")
    for k in ("x", "B", "C", "dt"):
        c[k][70:103], c[k][153:] = bad, float("inf")
        c[k] = torch.cat([c[k], torch.full((200,) + c[k].shape[1:], bad, dtype=c[k].dtype, device=DEV)])
        c[k + "64"] = np.concatenate([c[k + "64"], np.zeros((200,) + c[k + "64"].shape[1:])])
    out, pool = call(c)
    check(c, dtype, out, pool, f"ssm {dtype} padding")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_nan_stays_in_its_request(dtype):
    """Besides the tokens after it, a bad x reaches at most the 31 before it in its request (they
    share a step of a matrix product, where its weight is zero); a bad B or C no token before."""
    bad = float("nan")
    c = make(11, [100, 100, 100], 1, 1, 64, 64, dtype)
    good, gpool = call(c)
    c["x"][150, 0, 5] = float("nan")
    out, pool = call(c)
    keep = torch.ones(300, 64, dtype=torch.bool, device=DEV)
    keep[119:200, 5] = False
    assert torch.equal(out[:, 0][keep], good[:, 0][keep])
    assert torch.isnan(out[150:200, 0, 5]).all()
    s = c["idx"][1]
    assert torch.isnan(pool[s, 0, 5]).all()
    pool[s, 0, 5] = gpool[s, 0, 5]
    assert torch.equal(pool, gpool)
    c["x"][150, 0, 5], c["B"][150, 0, 3], c["C"][30, 0, 1] = 0.0, bad, bad
    c2 = dict(c, B=c["B"].clone(), C=c["C"].clone())
    c2["B"][150, 0, 3], c2["C"][30, 0, 1] = 0.0, 0.0
    (out, _), (good, _) = call(c), call(c2)
    keep[:] = True
    keep[30], keep[150:200] = False, False
    assert torch.equal(out[:, 0][keep], good[:, 0][keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b", [1, 3, 65])
@pytest.mark.parametrize("h,hv,dk,dv", [(1, 4, 128, 64), (2, 2, 64, 128), (1, 2, 256, 256), (3, 3, 64, 64)])
def test_ssm_decode(dtype, b, h, hv, dk, dv):
    c = make(12, [1] * b, h, hv, dk, dv, dtype, dead=((1, -2),) if b > 3 else ())
    out, pool = call(c, decode=True)
    check(c, dtype, out, pool, f"ssm decode {dtype} B={b} H={h} HV={hv} dk={dk} dv={dv}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_prompt_in_pieces(dtype):
    """A prompt in two calls and then token by token stays within the bounds of one recurrence."""
    import gated_deltanet_prefill_gdn_amd as gdn
    c = make(13, [140], 1, 2, 128, 64, dtype)
    pool, idx, got = c["pool"].clone(), i64(c["idx"]), []
    for lo, hi in ((0, 50), (50, 136)):
        got.append(gdn.gdn_ssm_prefill_fwd(
            *(c[k][lo:hi].contiguous() for k in ("C", "B", "x", "dt")), c["A_log"], c["dt_bias"], c["D"],
            pool, idx, i64([0, hi - lo])))
    for t in range(136, 140):
        got.append(gdn.gdn_ssm_decode_fwd(*(c[k][t:t + 1].contiguous() for k in ("C", "B", "x", "dt")),
                                          c["A_log"], c["dt_bias"], c["D"], pool, idx))
    torch.cuda.synchronize()
    check(c, dtype, torch.cat(got), pool, f"ssm {dtype} in pieces")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_short_requests_beside_a_long_one(dtype):
    """Enough short requests that they run token by token, among them empty and longer ones."""
    lengths = [1, 2, 3, 4, 0, 5, 1, 1] * 16 + [70]
    c = make(16, lengths, 1, 16, 64, 64, dtype, dead=((9, -1),))
    out, pool = call(c)
    check(c, dtype, out, pool, f"ssm {dtype} short requests")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_pieces_of_several_requests(dtype):
    """Long requests cut into pieces between short and empty ones, decays slow enough that every
    piece reaches the request's end, and fast enough that none does."""
    for dt_mean, a_hi in ((-7.0, 1.5), (0.5, 16.0)):
        c = make(17, [0, 2200, 31, 0, 1537, 600, 64], 2, 4, 64, 64, dtype, dt_mean=dt_mean, a_hi=a_hi)
        out, pool = call(c)
        check(c, dtype, out, pool, f"ssm {dtype} pieces, dt {dt_mean}")


@pytest.mark.parametrize("seed", range(10))
def test_ssm_random_shapes(seed):
    r = np.random.default_rng(100 + seed)
    dtype = ("bf16", "f32")[seed % 2]
    h = int(r.integers(1, 4))
    hv, dk, dv = h * int(r.integers(1, 4)), int(r.choice([64, 128])), int(r.choice([64, 128]))
    lengths = [int(x) for x in r.integers(0, 300, int(r.integers(1, 7)))]
    c = make(200 + seed, lengths, h, hv, dk, dv, dtype, dt_mean=float(r.uniform(-6, 0)))
    out, pool = call(c)
    check(c, dtype, out, pool, f"ssm {dtype} {lengths} H={h} HV={hv} dk={dk} dv={dv}")


def test_ssm_repeats_bit_for_bit():
    c = make(14, [900, 20, 1300], 2, 8, 128, 64, "bf16")
    (a, p), (b, q) = call(c), call(c)
    assert torch.equal(a, b) and torch.equal(p, q)
