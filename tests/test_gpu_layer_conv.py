"""The short causal convolution, its single-token form and its gradients against the fp64 oracle.

Tolerances, derived: with u = 2^-24, pre is a sum of W + 1 fp32 terms, so its error is at most
(W + 1) u M, M the sum of the terms' magnitudes; silu has slope at most 1.1, and its own
evaluation (exponential with argument error |x| u and two steps, reciprocal one step, product)
costs (8 + 2 |pre|) u relative; then one rounding to the output type. Gradients: g = dout
silu'(pre) moves by at most 0.5 per unit of pre, so by (W + 12) u |dout| (1.1 + 0.5 M) altogether
(the oracle's magnitudes hold that factor); sums over W taps add W u, sums over tokens at most
one u per step of the longest chain of additions (128 tokens of a run, 4 runs, one partial row per
32 or more tokens, added 8 chains wide)."""
import numpy as np
import pytest

from layer_util import DEV, HALF, U32, f32, i64, rounded, strided, within
from oracle import layer as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

LENGTHS = {
    "one": [1], "short": [1, 0, 2, 3, 0, 0, 4, 5], "ragged": [37, 0, 1, 130, 2, 64, 3, 29],
    "tile": [32, 64, 1, 31, 33], "long": [1300],
}


def make(seed, lengths, dims, w, dtype, bias, stateful, pool_extra=3, pad=0, offset=0, dead=()):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(int)
    n, ch, b = int(cu[-1]), sum(dims), len(lengths)
    c = dict(cu=cu, dims=dims)
    c["x"], c["x64"] = rounded(r.standard_normal((n, ch)), dtype)
    c["x"] = strided(c["x"], pad, offset) if pad or offset else c["x"]
    c["weight"], c["weight64"] = f32(0.5 * r.standard_normal((ch, w)))
    c["bias"], c["bias64"] = f32(0.3 * r.standard_normal(ch)) if bias else (None, None)
    c["pool"], c["pool64"], c["idx"] = None, None, None
    if stateful:
        c["pool"], c["pool64"] = rounded(r.standard_normal((b + pool_extra, w - 1, ch)), dtype)
        c["idx"] = r.permutation(b + pool_extra)[:b]
        for k, v in dead:
            c["idx"][k] = v
    return c


def call(c, silu, fn=None, **kw):
    import gated_deltanet_prefill_gdn_amd as gdn
    pool = None if c["pool"] is None else c["pool"].clone()
    idx = None if c["idx"] is None else i64(c["idx"])
    outs = tuple(torch.full((c["x"].shape[0], d), 7.5, dtype=c["x"].dtype, device=DEV)
                 for d in c["dims"])
    (fn or gdn.gdn_conv_fwd)(c["x"], c["weight"], c["bias"], pool, idx,
                             *(() if fn else (i64(c["cu"]),)), dims=c["dims"], silu=silu, outs=outs,
                             **kw)
    torch.cuda.synchronize()
    return outs, pool


def check(c, silu, dtype, w, outs, pool, what):
    ref, new, mag, written = L.conv_fwd(c["x64"], c["weight64"], c["bias64"], c["pool64"], c["idx"],
                                        c["cu"], silu)
    got = torch.cat(outs, 1).double().cpu().numpy()
    assert (got[~written] == 7.5).all(), "a padding row was written"
    pre = L.conv_fwd(c["x64"], c["weight64"], c["bias64"], c["pool64"], c["idx"], c["cu"], False)[0]
    allow = (HALF[dtype] * np.abs(ref) + U32 * (1.1 * (w + 1) * mag + (8 + 2 * np.abs(pre)) * np.abs(ref))
             + 1e-38)
    allow = allow + HALF[dtype] * (allow - HALF[dtype] * np.abs(ref))
    within(got[written], ref[written], allow[written], what)
    if pool is not None:
        np.testing.assert_array_equal(pool.double().cpu().numpy(), new)  # rows are moved, not computed


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("w", [2, 3, 4])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dims", [(64, 32, 96), (5, 3, 9), (2056,)])
def test_conv_forward(dtype, w, lengths, dims):
    if len(dims) == 1 and lengths not in ("tile", "ragged"):
        pytest.skip("the wide case runs at two length patterns")
    k = len(lengths) + w
    c = make(k, LENGTHS[lengths], dims, w, dtype, bias=k % 2 == 0, stateful=lengths != "tile" or w == 4)
    outs, pool = call(c, silu=k % 3 != 0)
    check(c, k % 3 != 0, dtype, w, outs, pool, f"conv {dtype} W={w} {lengths} {dims}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (40, 8), (3, 0), (16, 1)])
def test_conv_rows_of_a_wider_tensor(dtype, pad, offset):
    """Row strides and starts that allow 16-byte vectors and ones that do not, NaN between."""
    c = make(11, [9, 50], (64, 64, 128), 4, dtype, True, True, pad=pad, offset=offset)
    outs, pool = call(c, True)
    check(c, True, dtype, 4, outs, pool, f"conv strided {dtype} +{pad} @{offset}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_conv_padding_requests_and_rows(dtype):
    """Cache indices outside the pool, rows behind the last request: left as they were, and what
    stands there (NaN) reaches nobody."""
    c = make(12, [5, 40, 2, 70, 1], (16, 16), 4, dtype, True, True,
             dead=((1, -1), (2, 8), (4, 1 << 40)))
    c["x"][5:47] = float("nan")
    c["x"] = torch.cat([c["x"], torch.full((13, 32), float("nan"), dtype=c["x"].dtype, device=DEV)])
    c["x64"] = np.concatenate([c["x64"], np.zeros((13, 32))])
    outs, pool = call(c, True)
    check(c, True, dtype, 4, outs, pool, f"conv padding {dtype}")
    assert all((o[118:] == 7.5).all() for o in outs)


def test_conv_nan_and_infinity_stay_in_their_request():
    c = make(13, [20, 20, 20], (32,), 4, "f32", False, True)
    c["x"][25, 3], c["x"][30, 4] = float("nan"), float("inf")
    (out,), _ = call(c, False)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[25:29, 3], want[30:34, 4] = True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,dims", [(1, (64, 64, 128)), (3, (5, 3, 1)), (33, (2048, 8)), (300, (72,))])
def test_conv_decode_is_the_forward_of_one_token(dtype, b, dims):
    import gated_deltanet_prefill_gdn_amd as gdn
    for w in (2, 3, 4):
        c = make(20 + w, [1] * b, dims, w, dtype, True, True, dead=((b // 2, -3),) if b > 3 else ())
        outs, pool = call(c, True, gdn.gdn_conv_decode_fwd)
        check(c, True, dtype, w, outs, pool, f"conv decode {dtype} B={b} W={w}")
        outs2, pool2 = call(c, True)
        assert all(torch.equal(a, d) for a, d in zip(outs, outs2)) and torch.equal(pool, pool2)


def test_conv_prompt_in_pieces_is_the_prompt_at_once():
    """A prompt, then its continuation token by token, gives the same bits as one call."""
    import gated_deltanet_prefill_gdn_amd as gdn
    c = make(30, [45], (64, 64), 4, "bf16", True, True)
    outs, pool = call(c, True)
    p, idx = c["pool"].clone(), i64(c["idx"])
    got = [gdn.gdn_conv_fwd(c["x"][:40], c["weight"], c["bias"], p, idx, i64([0, 40]), dims=c["dims"])]
    got += [gdn.gdn_conv_decode_fwd(c["x"][t:t + 1], c["weight"], c["bias"], p, idx, dims=c["dims"])
            for t in range(40, 45)]
    for i in range(2):
        assert torch.equal(torch.cat([g[i] for g in got]), outs[i])
    assert torch.equal(p, pool)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dout_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dims", [(64, 32, 32), (5, 3, 9)])
def test_conv_backward(dtype, dout_dtype, lengths, dims):
    import gated_deltanet_prefill_gdn_amd as gdn
    w = 2 + (len(lengths) + len(dtype) + len(dout_dtype)) % 3
    silu, stateful, bias = lengths != "short", lengths != "tile", lengths != "one"
    c = make(40 + w, LENGTHS[lengths], dims, w, dtype, bias, stateful,
             dead=((3, -1),) if lengths == "ragged" else ())
    r = np.random.default_rng(99)
    n, ch, b = c["x"].shape[0], sum(dims), len(LENGTHS[lengths])
    dout, dout64 = rounded(r.standard_normal((n, ch)), dout_dtype)
    dstate, dstate64 = f32(r.standard_normal((b, w - 1, ch))) if lengths != "long" else (None, None)
    dx = strided(torch.full((n, ch), 7.5, dtype=c["x"].dtype, device=DEV), 8) if lengths == "ragged" else None
    before = None if c["pool"] is None else c["pool"].clone()
    g = gdn.gdn_conv_bwd(c["x"], c["weight"], c["bias"], c["pool"],
                         None if c["idx"] is None else i64(c["idx"]), i64(c["cu"]),
                         [d.contiguous() for d in dout.split(dims, 1)], dstate, silu=silu, dx=dx)
    torch.cuda.synchronize()
    ref = L.conv_bwd(c["x64"], c["weight64"], c["bias64"], c["pool64"], c["idx"], c["cu"], dout64,
                     dstate64, silu)
    assert before is None or torch.equal(before, c["pool"])
    assert set(g) == {"dx", "dweight"} | ({"dbias"} if bias else set()) | ({"dstate0"} if stateful else set())
    chain = 128 + 4 + n / 32 / 8 + 1
    what = f"conv bwd {dtype}/{dout_dtype} W={w} {lengths} {dims}"
    live = np.ones(n, bool)
    if lengths == "ragged":
        live[c["cu"][3]:c["cu"][4]] = False
        assert (g["dx"].float().cpu().numpy()[~live] == 7.5).all(), "a padding row was written"
    steps = 2 * w + 13
    within(g["dx"].double().cpu().numpy()[live], ref["dx"][live],
           (HALF[dtype] * np.abs(ref["dx"]) + (1 + HALF[dtype]) * U32 * steps * ref["dx_mag"] + 1e-38)[live],
           what + " dx")
    within(g["dweight"], ref["dweight"], U32 * (chain + steps) * ref["dweight_mag"] + 1e-38, what + " dweight")
    if bias:
        within(g["dbias"], ref["dbias"], U32 * (chain + steps) * ref["dbias_mag"] + 1e-38, what + " dbias")
    if stateful:
        within(g["dstate0"], ref["dstate0"], U32 * steps * ref["dstate0_mag"] + 1e-38, what + " dstate0")


def test_conv_backward_without_tokens():
    import gated_deltanet_prefill_gdn_amd as gdn
    c = make(50, [0, 0], (16,), 4, "bf16", True, True)
    dstate = torch.randn(2, 3, 16, device=DEV)
    g = gdn.gdn_conv_bwd(c["x"], c["weight"], c["bias"], c["pool"], i64(c["idx"]), i64([0, 0, 0]),
                         [torch.empty(0, 16, device=DEV)], dstate)
    torch.cuda.synchronize()
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all() and torch.equal(g["dstate0"], dstate)


def test_conv_backward_repeats_bit_for_bit():
    import gated_deltanet_prefill_gdn_amd as gdn
    c = make(51, [700, 0, 900, 3], (256, 128), 4, "bf16", True, True)
    douts = [torch.randn(1603, d, device=DEV) for d in c["dims"]]
    a, b = (gdn.gdn_conv_bwd(c["x"], c["weight"], c["bias"], c["pool"], i64(c["idx"]), i64(c["cu"]), douts)
            for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)
