"""Linear attention with a decay per head (prompts, single tokens, gradients) against the fp64
recurrence.

Tolerances, derived. Let M be the same sums over absolute values (the oracle's magnitudes): any
evaluation that rounds the factors of its products by a relative r is off by at most about r M.
States and the outputs of fp32 inputs: factors keep 24 bits, powers of the decay are a few steps of
2^-24 off, and a sum over n tokens, of which a chain of n / 64 + 64 additions touches each term, is
below 150 steps off for 5000 tokens: 2^-16 M. Outputs of bf16 inputs: scores, states read and the
decayed values behind them keep 16 bits each, the last cut off (2^-16 each, three of them): 2^-14 M,
then one rounding to bf16."""
import numpy as np
import pytest

from layer_util import DEV, DT, HALF, f32, i64, np64, rounded, strided, within
from oracle import linear as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

OUT = {"bf16": 2.0 ** -14, "f32": 2.0 ** -16}
STATE = 2.0 ** -16


def decays(r, hv):
    """A mixture: heads that forget within a few tokens, within hundreds, hardly ever."""
    return -np.exp2(-r.uniform(-2, 12, hv))


def make(seed, lengths, h, hv, dk, dv, dtype, extra=2, dead=(), pad=0, tail=0, log_decay=None):
    """`tail` padding rows behind the last request; `pad` elements between tokens."""
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(int)
    n, b = int(cu[-1]) + tail, len(lengths)
    c = dict(cu=cu, scale=float(np.float32(dk ** -0.5)), dtype=dtype)
    for k, shape in (("q", (n, h, dk)), ("k", (n, h, dk)), ("v", (n, hv, dv)), ("dout", (n, hv, dv))):
        t, c[k + "64"] = rounded(0.8 * r.standard_normal(shape) + 0.05, dtype)
        c[k] = strided(t, pad) if pad and k != "dout" else t
    c["g"], c["g64"] = f32(decays(r, hv) if log_decay is None else log_decay)
    c["pool"], c["pool64"] = f32(0.3 * r.standard_normal((b + extra, hv, dv, dk)))
    c["dstate"], c["dstate64"] = f32(0.1 * r.standard_normal((b, hv, dv, dk)))
    c["idx"] = r.permutation(b + extra)[:b]
    for k, v in dead:
        c["idx"][k] = v
    return c


def args64(c, pool=True):
    return (c["q64"], c["k64"], c["v64"], c["g64"], c["scale"], c["pool64"] if pool else None, c["idx"], c["cu"])


def forward(c, decode=False, pool=True, **kw):
    import gated_deltanet_prefill_gdn_amd as gdn
    state = c["pool"].clone() if pool else None
    out = torch.full(c["v"].shape, 7.5, dtype=c["v"].dtype, device=DEV)
    a = (c["q"], c["k"], c["v"], c["g"], state, i64(c["idx"]) if pool else None)
    if decode:
        gdn.gdn_linear_decode_fwd(*a, scale=c["scale"], out=out, **kw)
    else:
        gdn.gdn_linear_prefill_fwd(*a, i64(c["cu"]), scale=c["scale"], out=out, **kw)
    torch.cuda.synchronize()
    return out, state


def check_forward(c, out, state, what, pool=True):
    ref, new, mag, mags, written = L.linear_fwd(*args64(c, pool))
    got, h = np64(out), HALF[c["dtype"]]
    assert (got[~written] == 7.5).all(), "a padding row was written"
    within(got[written], ref[written], (h * np.abs(ref) + (1 + h) * OUT[c["dtype"]] * mag + 1e-38)[written], what)
    if pool:
        within(state, new, STATE * mags + 1e-38, what + " state")
        touched = {s for s, n in zip(c["idx"], np.diff(c["cu"])) if n and 0 <= s < len(new)}
        for s in set(range(len(new))) - touched:
            np.testing.assert_array_equal(state[s].cpu().numpy(), c["pool"][s].cpu().numpy())


def backward(c, pool=True, dstate=True, **kw):
    import gated_deltanet_prefill_gdn_amd as gdn
    g = gdn.gdn_linear_bwd(c["q"], c["k"], c["v"], c["g"], c["pool"] if pool else None,
                           i64(c["idx"]) if pool else None, i64(c["cu"]), c["dout"],
                           c["dstate"] if dstate else None, scale=c["scale"], **kw)
    torch.cuda.synchronize()
    return g


def check_backward(c, g, what, pool=True, dstate=True):
    ref = L.linear_bwd(*args64(c, pool), c["dout64"], c["dstate64"] if dstate else None)
    written = np.zeros(len(c["v64"]), bool)
    for b in range(len(c["cu"]) - 1):
        if not pool or 0 <= c["idx"][b] < len(c["pool64"]):
            written[c["cu"][b]:c["cu"][b + 1]] = True
    h = HALF[c["dtype"]]
    assert set(g) == {"dq", "dk", "dv"} | ({"dstate0"} if pool else set())
    for k in ("dq", "dk", "dv"):
        allow = h * np.abs(ref[k]) + (1 + h) * OUT[c["dtype"]] * ref[k + "_mag"] + 1e-38
        within(np64(g[k])[written], ref[k][written], allow[written], f"{what} {k}")
        assert g[k].dtype is DT[c["dtype"]] and g[k].is_contiguous()
    if pool:
        within(g["dstate0"], ref["dstate0"], STATE * ref["dstate0_mag"] + 1e-38, what + " dstate0")


LENGTHS = {
    "one": [1], "chunk": [64], "edges": [63, 65, 1, 0, 128, 127, 2], "ragged": [200, 0, 31, 333, 17],
    "long": [1500, 700], "zero": [0, 0, 5, 0], "few": [4, 2, 3, 1, 4, 0, 1, 2],
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("h,hv,dk,dv", [(1, 2, 128, 64), (2, 2, 64, 64), (1, 3, 64, 128), (2, 2, 128, 128)])
def test_linear_prefill_and_gradients(dtype, lengths, h, hv, dk, dv):
    c = make(len(lengths) + hv, LENGTHS[lengths], h, hv, dk, dv, dtype, pad=8 * (hv - 1))
    what = f"linear {dtype} {lengths} H={h} HV={hv} dk={dk} dv={dv}"
    check_forward(c, *forward(c), what)
    check_backward(c, backward(c), what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(256, 64), (64, 256), (256, 128), (128, 256), (256, 256)])
def test_linear_wide_heads(dtype, dk, dv):
    c = make(dk + dv, [150, 1, 70], 1, 2, dk, dv, dtype)
    check_forward(c, *forward(c), f"linear {dtype} dk={dk} dv={dv}")
    check_backward(c, backward(c), f"linear {dtype} dk={dk} dv={dv}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,hv", [(1, 33), (3, 15), (8, 8)])
def test_linear_many_heads_and_requests(dtype, h, hv):
    r = np.random.default_rng(3)
    c = make(5, list(r.integers(0, 90, 24)), h, hv, 64, 64, dtype)
    check_forward(c, *forward(c), f"linear {dtype} 24 requests H={h} HV={hv}")
    check_backward(c, backward(c), f"linear {dtype} 24 requests H={h} HV={hv}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[5003], [1, 3001, 640, 0, 1100]])
def test_linear_long_requests(dtype, lengths):
    """Long enough to be cut into pieces that are joined again, with states that live over
    thousands of tokens beside heads that forget at once."""
    c = make(8, lengths, 1, 3, 128, 64, dtype, log_decay=[-2.0 ** -11, -3.0, 0.0])
    check_forward(c, *forward(c), f"linear {dtype} {lengths}")
    check_backward(c, backward(c), f"linear {dtype} {lengths}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_extreme_decays(dtype):
    """Nothing kept (-inf, and -200 and -90, whose powers underflow), everything kept (0, and an
    entry above 0, which counts as 0), and a decay that falls below fp32 within a tile."""
    g = [-np.inf, -200.0, -90.0, -9.0, 0.0, 3.0, -1e-30, -3e38]
    c = make(9, [70, 130, 1, 900], 8, 8, 64, 64, dtype, log_decay=g)
    check_forward(c, *forward(c), f"linear {dtype} extreme decays")
    check_backward(c, backward(c), f"linear {dtype} extreme decays")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dead,tail", [([(0, -1), (2, 99)], 0), ([], 37), ([(1, 5)], 3)])
def test_linear_padding(dtype, dead, tail):
    """Requests without a slot, and rows behind the last request: nothing of them is written."""
    c = make(10, [66, 130, 9], 2, 2, 64, 64, dtype, extra=2, dead=dead, tail=tail)
    check_forward(c, *forward(c), f"linear {dtype} padding")
    g = backward(c)
    check_backward(c, g, f"linear {dtype} padding")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[65, 0, 3], [1300]])
def test_linear_without_a_pool(dtype, lengths):
    c = make(11, lengths, 1, 2, 64, 64, dtype)
    out, _ = forward(c, pool=False)
    check_forward(c, out, None, f"linear {dtype} no pool", pool=False)
    check_backward(c, backward(c, pool=False, dstate=False), f"linear {dtype} no pool", pool=False, dstate=False)
    check_backward(c, backward(c, dstate=False), f"linear {dtype} no dstate", dstate=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b", [1, 5, 130])
@pytest.mark.parametrize("h,hv,dk,dv", [(2, 4, 128, 64), (1, 1, 64, 256), (2, 2, 256, 128), (3, 3, 128, 128)])
def test_linear_decode(dtype, b, h, hv, dk, dv):
    c = make(b + hv, [1] * b, h, hv, dk, dv, dtype, pad=16, dead=[(3, -5)] if b > 3 else ())
    check_forward(c, *forward(c, decode=True), f"linear decode {dtype} B={b} dk={dk} dv={dv}")


def test_linear_gradients_by_differences():
    """The loss is linear in q, in k, and in (v, start state) together, so a difference of the forward
    call over any step is a derivative. fp32, whose outputs are 2^-16 of their magnitude off."""
    c = make(12, [90, 700, 33], 1, 2, 64, 64, "f32")
    g = backward(c)
    r = torch.Generator(device=DEV).manual_seed(1)

    def loss(**kw):
        out, state = forward({**c, **kw})
        return ((out.double() * c["dout"].double()).sum()
                + (state[i64(c["idx"])].double() * c["dstate"].double()).sum()).item()

    for name in ("q", "k", "v", "pool"):
        d = torch.randn(c[name].shape, generator=r, device=DEV)
        num = (loss(**{name: c[name] + d}) - loss(**{name: c[name] - d})) / 2
        back = g["dstate0"].double() if name == "pool" else g["d" + name].double()
        at = d[i64(c["idx"])] if name == "pool" else d
        want = (back * at.double()).sum().item()
        size = (back * at.double()).abs().sum().item()
        print(f"[linear] d{name}: {num:.6e} against {want:.6e}, terms {size:.2e}", flush=True)
        assert abs(num - want) <= 2.0 ** -14 * size


def test_linear_non_finite_values_stay_in_their_request():
    """An infinite or NaN entry may reach its own request's head; the others keep their bits."""
    c = make(13, [100, 90, 3], 2, 2, 64, 64, "bf16")
    clean, _ = forward(c)
    gclean = backward(c)
    for name in ("q", "k", "v"):
        bad = {**c, name: c[name].clone()}
        bad[name][50, 0, 3] = float("nan")
        bad[name][60, 0, 3] = float("inf")
        out, _ = forward(bad)
        assert torch.equal(out[100:], clean[100:]) and torch.equal(out[:, 1], clean[:, 1])
        assert not torch.isfinite(out[50:100, 0]).all()
        g = backward(bad)
        for k in ("dq", "dk", "dv"):
            assert torch.equal(g[k][100:], gclean[k][100:]) and torch.equal(g[k][:, 1], gclean[k][:, 1])


def test_linear_large_values():
    """Finite values up to the largest of bf16 next to small ones. Here an entry of q times one of k
    is about 1e-38: fp32 ends at 2^-126 = 1.2e-38, and a score whose 64 products each lose up to that
    is 64 2^-126 off, which v, the decays and the scale carry into the output."""
    c = make(14, [80], 1, 1, 64, 64, "bf16", log_decay=[-0.1])
    for name, scale in (("q", 1e-20), ("k", 1e-18), ("v", 1e37)):
        c[name], c[name + "64"] = rounded(scale * c[name + "64"], "bf16")
    c["pool"], c["pool64"] = f32(1e18 * c["pool64"])
    out, state = forward(c)
    ref, new, mag, mags, _ = L.linear_fwd(*args64(c))
    lost = np.zeros_like(ref)
    carried = 0.0
    for t in range(80):
        carried = np.exp(-0.1) * carried + np.abs(c["v64"][t])
        lost[t] = c["scale"] * 64 * 2.0 ** -126 * carried
    h = HALF["bf16"]
    within(out, ref, h * np.abs(ref) + (1 + h) * (OUT["bf16"] * mag + lost), "linear large values")
    within(state, new, STATE * mags, "linear large values, state")


def test_linear_wide_range_of_values():
    """Values of very different sizes whose products stay inside fp32's range."""
    for q, k, v, pool in ((1e-12, 1e-18, 1e37, 1e18), (1e15, 1e15, 1e-30, 1e-14), (1e-15, 1e25, 1e10, 1e34)):
        c = make(14, [80], 1, 1, 64, 64, "bf16", log_decay=[-0.1])
        for name, scale in (("q", q), ("k", k), ("v", v)):
            c[name], c[name + "64"] = rounded(scale * c[name + "64"], "bf16")
        c["pool"], c["pool64"] = f32(pool * c["pool64"])
        check_forward(c, *forward(c), f"linear values of {q}, {k}, {v}")


def test_linear_calls_repeat_to_the_bit():
    c = make(15, [700, 64, 1], 1, 2, 128, 128, "bf16")
    (a, sa), (b, sb) = forward(c), forward(c)
    assert torch.equal(a, b) and torch.equal(sa, sb)
    ga, gb = backward(c), backward(c)
    assert all(torch.equal(ga[k], gb[k]) for k in ga)


def test_linear_state_pool_past_32_bits():
    import gated_deltanet_prefill_gdn_amd as gdn
    slots, hv, d = 70000, 4, 64
    pool = torch.empty(slots, hv, d, d, device=DEV)  # 4.6 GB
    c = make(16, [70, 1, 1], hv, hv, d, d, "bf16", extra=0)
    at = [slots - 1, 65536, 3]
    pool[at] = c["pool"]
    c["idx"] = np.arange(3)
    out = torch.full(c["v"].shape, 7.5, dtype=c["v"].dtype, device=DEV)
    gdn.gdn_linear_prefill_fwd(c["q"], c["k"], c["v"], c["g"], pool, i64(at), i64(c["cu"]), scale=c["scale"], out=out)
    torch.cuda.synchronize()
    check_forward(c, out, pool[at], "linear pool past 32 bits")


def test_linear_tokens_past_32_bits():
    """Tokens more than 2^31 elements into their tensors; the last ones are checked."""
    import gated_deltanet_prefill_gdn_amd as gdn
    n, stride = 600000, 4096
    wide = torch.zeros(n, stride, dtype=torch.bfloat16, device=DEV)  # 4.9 GB
    g = torch.Generator(device=DEV).manual_seed(3)
    wide[-200:, :192] = torch.randn(200, 192, device=DEV, generator=g).bfloat16()
    q, k, v = (wide[:, 64 * i:64 * i + 64].unflatten(1, (1, 64)) for i in range(3))
    decay = torch.tensor([-0.05], device=DEV)
    pool = torch.zeros(2, 1, 64, 64, device=DEV)
    out = gdn.gdn_linear_prefill_fwd(q, k, v, decay, pool, i64([0, 1]), i64([0, n - 100, n]))
    tail = [t[-200:].double().cpu().numpy() for t in (q, k, v)]
    ref, new, mag, mags, _ = L.linear_fwd(*tail, np64(decay), 0.125, np.zeros((2, 1, 64, 64)), [0, 1], [0, 100, 200])
    h = HALF["bf16"]
    within(out[-200:], ref, h * np.abs(ref) + (1 + h) * OUT["bf16"] * mag + 1e-38, "linear tokens past 32 bits")
    within(pool, new, STATE * mags + 1e-38, "linear tokens past 32 bits, state")
