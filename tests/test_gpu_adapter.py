"""Low-rank adapters of many requests beside a shared projection against their definition in fp64.

Tolerances, derived. Let M be the same sums over absolute values (the oracle's magnitude). x A^T and
its product with B^T are fp32 sums of at most 4200 and 128 terms, of which a chain of some hundred
additions touches each (2^-16 M with room); for bf16 the low-rank row enters the second product with
16 bits, the last cut off (2^-16), as three parts of 24 bits for fp32: together 2^-15 M. Then one
rounding to the output type."""
import numpy as np
import pytest

from layer_util import DEV, DT, HALF, f32, i64, np64, rounded, strided, within
from oracle import linear as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SUM = 2.0 ** -15


def make(seed, lengths, k, m, rank, adapters, dtype, pad=0, offset=0, tail=0, idx=None):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(int)
    n, b = int(cu[-1]) + tail, len(lengths)
    c = dict(cu=cu, dtype=dtype)
    for name, shape, s in (("x", (n, k), 1), ("base", (n, m), 1), ("A", (adapters, rank, k), k ** -0.5),
                           ("B", (adapters, m, rank), rank ** -0.5)):
        t, c[name + "64"] = rounded(s * r.standard_normal(shape), dtype)
        c[name] = strided(t, pad, offset) if (pad or offset) and name in ("x", "base") else t
    c["s"], c["s64"] = f32(r.uniform(-2, 2, adapters))
    c["idx"] = r.integers(-1, adapters + 1, b) if idx is None else np.asarray(idx)
    return c


def call(c, decode=False, **kw):
    import gated_deltanet_prefill_gdn_amd as gdn
    a = (c["x"], c["base"], c["A"], c["B"], c["s"], i64(c["idx"]))
    out = (gdn.gdn_adapter_decode_fwd(*a, **kw) if decode else gdn.gdn_adapter_fwd(*a, i64(c["cu"]), **kw))
    torch.cuda.synchronize()
    return out


def check(c, out, what):
    ref, mag, written = L.adapter(c["x64"], c["base64"], c["A64"], c["B64"], c["s64"], c["idx"], c["cu"])
    h = HALF[c["dtype"]]
    got = np64(out)
    within(got[written], ref[written], (h * np.abs(ref) + (1 + h) * SUM * mag + 1e-38)[written], what)
    for b, a in enumerate(c["idx"]):
        if not 0 <= a < len(c["A64"]):  # no adapter: the very bits of base
            rows = slice(c["cu"][b], c["cu"][b + 1])
            np.testing.assert_array_equal(got[rows], c["base64"][rows])


LENGTHS = {"one": [1], "tile": [64], "edges": [15, 16, 17, 1, 0, 33, 63, 65], "ragged": [200, 0, 31, 133, 17],
           "singles": [1] * 40, "zero": [0, 0, 5, 0]}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("k,m,rank", [(256, 384, 16), (64, 64, 8), (131, 77, 5), (512, 200, 64), (72, 1000, 33)])
def test_adapter(dtype, lengths, k, m, rank):
    c = make(rank + len(lengths), LENGTHS[lengths], k, m, rank, 4, dtype)
    check(c, call(c), f"adapter {dtype} {lengths} K={k} M={m} R={rank}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rank", [1, 2, 15, 31, 32, 48, 65, 100, 127, 128])
def test_adapter_ranks(dtype, rank):
    c = make(rank, [70, 3, 40], 320, 136, rank, 3, dtype)
    check(c, call(c), f"adapter {dtype} R={rank}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k,m", [(1, 1), (3, 2), (7, 4097), (4097, 7), (4096, 8), (8, 4096), (4104, 4104)])
def test_adapter_sizes(dtype, k, m):
    c = make(k + m, [20, 1, 13], k, m, 16, 3, dtype)
    check(c, call(c), f"adapter {dtype} K={k} M={m}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k,m,rank", [(1027, 333, 100), (2051, 517, 40), (4095, 263, 9), (513, 1021, 17)])
@pytest.mark.parametrize("lengths", [[70, 1, 40], [5, 2]])
def test_adapter_odd_rows(dtype, k, m, rank, lengths):
    """Rows of no whole number of vectors, long enough that most of a row is read in vectors."""
    c = make(k + rank, lengths, k, m, rank, 2, dtype, pad=5, offset=1)
    check(c, call(c), f"adapter {dtype} K={k} M={m} R={rank}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (1, 0), (0, 3), (13, 1)])
def test_adapter_strides_and_alignment(dtype, pad, offset):
    """Rows any stride apart, starting anywhere: vectors where all of them allow it."""
    c = make(pad, [33, 2, 50], 128, 192, 16, 3, dtype, pad=pad, offset=offset)
    check(c, call(c), f"adapter {dtype} pad={pad} offset={offset}")
    wide = torch.full((85, 192 + pad + offset), 3.0, dtype=DT[dtype], device=DEV)
    view = wide[:, offset:offset + 192]
    check(c, call(c, out=view), f"adapter {dtype} strided out")
    assert (wide[:, :offset] == 3.0).all() and (wide[:, offset + 192:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_adapter_in_place(dtype):
    c = make(3, [33, 2, 50, 7], 128, 192, 16, 3, dtype, pad=8, idx=[2, -1, 0, 3])
    out = c["base"].clone(memory_format=torch.preserve_format)
    wide = strided(c["base"].contiguous(), 8)
    given = {**c, "base": wide}
    got = call(given, out=wide)
    assert got.data_ptr() == wide.data_ptr()
    check(c, got, f"adapter {dtype} in place")
    assert torch.equal(out, c["base"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,adapters", [(1, 1), (7, 2), (130, 5), (512, 32), (65, 64)])
@pytest.mark.parametrize("k,m,rank", [(256, 512, 16), (100, 37, 6)])
def test_adapter_decode(dtype, b, adapters, k, m, rank):
    c = make(b, [1] * b, k, m, rank, adapters, dtype)
    check(c, call(c, decode=True), f"adapter decode {dtype} B={b} adapters={adapters}")
    assert torch.equal(call(c, decode=True), call(c)), "single tokens are requests of one token"


def test_adapter_padding_rows_are_not_written():
    c = make(5, [20, 9], 64, 96, 8, 2, "bf16", tail=11, idx=[1, 0])
    out = torch.full((40, 96), 7.5, dtype=torch.bfloat16, device=DEV)
    check({**c, "base64": c["base64"]}, call(c, out=out), "adapter padding")
    assert (out[29:] == 7.5).all()


@pytest.mark.parametrize("idx", [[-1, -7, 9], [0, 0, 0], [2, 2, 0]])
def test_adapter_shared_and_missing(idx):
    c = make(6, [40, 17, 70], 64, 96, 8, 3, "bf16", idx=idx)
    check(c, call(c), f"adapter indices {idx}")


def test_adapter_without_a_bank():
    c = make(7, [5, 3], 64, 96, 8, 1, "bf16", idx=[0, 0])
    c["A"], c["B"], c["s"] = c["A"][:0], c["B"][:0], c["s"][:0]
    assert torch.equal(call(c), c["base"])


@pytest.mark.parametrize("adapters,b", [(4096, 300), (1000, 3000)])
def test_adapter_many_adapters_and_requests(adapters, b):
    r = np.random.default_rng(b)
    c = make(8, list(r.integers(0, 4, b)), 64, 64, 4, adapters, "bf16")
    check(c, call(c), f"adapter {adapters} adapters {b} requests")


def test_adapter_non_finite_values_stay_in_their_rows():
    c = make(9, [40, 40], 128, 96, 16, 2, "bf16", idx=[1, 1])
    clean = call(c)
    bad = {**c, "x": c["x"].clone(), "base": c["base"].clone()}
    bad["x"][5, 7], bad["base"][60, 3] = float("nan"), float("inf")
    out = call(bad)
    keep = torch.ones_like(clean, dtype=torch.bool)
    keep[5], keep[60, 3] = False, False
    assert torch.equal(out[keep], clean[keep]) and out[5].isnan().all() and out[60, 3].isinf()
    bad = {**c, "A": c["A"].clone()}
    bad["A"][0, 0, 0] = float("nan")  # an adapter that nobody asked for
    assert torch.equal(call(bad), clean)


def test_adapter_large_values():
    """A low-rank row beyond the range of bf16's products, brought back by a small B."""
    c = make(10, [30], 64, 64, 8, 1, "bf16", idx=[0])
    for name, s in (("x", 1e25), ("A", 1e11), ("B", 1e-36)):
        c[name], c[name + "64"] = rounded(s * c[name + "64"], "bf16")
    check(c, call(c), "adapter large values")


def test_adapter_rows_past_32_bits():
    import gated_deltanet_prefill_gdn_amd as gdn
    n, stride = 600000, 4096
    wide = torch.zeros(n, stride, dtype=torch.bfloat16, device=DEV)  # 4.9 GB
    g = torch.Generator(device=DEV).manual_seed(3)
    wide[-100:] = torch.randn(100, stride, device=DEV, generator=g).bfloat16()
    A, B = (torch.randn(2, *s, device=DEV, generator=g).bfloat16() for s in ((8, 64), (64, 8)))
    s = torch.ones(2, device=DEV)
    x, base = wide[:, :64], wide[:, 64:128]
    out = gdn.gdn_adapter_fwd(x, base, A, B, s, i64([0, 1]), i64([0, n - 70, n]), out=wide[:, 128:192])
    ref, mag, _ = L.adapter(*(np64(t) for t in (x[-100:], base[-100:], A, B, s)), [0, 1], [0, 30, 100])
    h = HALF["bf16"]
    within(out[-100:], ref, h * np.abs(ref) + (1 + h) * SUM * mag + 1e-38, "adapter rows past 32 bits")


def test_adapter_graph_and_stream():
    """Captured twice with a shared workspace and replayed with new inputs and indices between eager
    work; on another stream."""
    import gated_deltanet_prefill_gdn_amd as gdn
    cs = [make(20 + i, [1] * 24, 256, 320, 16, 4, "bf16") for i in range(2)]
    idx = [i64(c["idx"]) for c in cs]
    outs = [torch.empty(24, 320, dtype=torch.bfloat16, device=DEV) for _ in cs]
    need = gdn.gdn_adapter_workspace_size(gdn.adapter_problem(cs[0]["x"], cs[0]["base"], cs[0]["A"], 24))
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)

    def go(i, out=None, workspace=None, stream=None):
        c = cs[i]
        return gdn.gdn_adapter_decode_fwd(c["x"], c["base"], c["A"], c["B"], c["s"], idx[i], out=out,
                                          workspace=workspace, stream=stream)

    for i in range(2):
        go(i, outs[i], ws)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            go(i, outs[i], ws)
    for step in range(3):
        for i in range(2):
            cs[i]["x"].normal_()
            idx[i].copy_((idx[i] + 1 + step) % 6 - 1)
            graphs[i].replay()
        want = [go(i) for i in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = go(0, stream=s)
    s.synchronize()
    assert torch.equal(got, want[0])
