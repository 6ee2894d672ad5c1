"""Linear attention and adapters as a layer uses them: projection with its requests' adapters,
convolution, linear attention, norm, over prompts and then token by token; backwards; on other streams;
captured into HIP graphs that are replayed among other work; workspaces of exactly the stated size."""
import numpy as np
import pytest

from layer_util import DEV, HALF, f32, i64, np64, rounded, within
from oracle import layer as OL
from oracle import linear as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def linear_inputs(seed, n, h=2, hv=4, dk=64, dv=64, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, device=DEV, generator=g).to(dtype)  # noqa: E731
    return [rn(n, h, dk), rn(n, h, dk), rn(n, hv, dv), -torch.exp2(-torch.arange(1, hv + 1, device=DEV).float())]


class Layer:
    """x -> packed row [q | k | v | gate] by a shared weight and adapters -> convolution of q, k, v ->
    linear attention -> gated norm, weights and pools of its own."""

    def __init__(self, seed, lengths, hidden=128, h=2, d=64, rank=8, adapters=3):
        r = np.random.default_rng(seed)
        self.cu = np.concatenate([[0], np.cumsum(lengths)]).astype(int)
        self.n, self.b, self.h, self.d = int(self.cu[-1]), len(lengths), h, d
        self.ch = 3 * h * d
        self.x, self.x64 = rounded(r.standard_normal((self.n, hidden)), "bf16")
        self.W, self.W64 = rounded(hidden ** -0.5 * r.standard_normal((self.ch + h * d, hidden)), "bf16")
        self.A, self.A64 = rounded(hidden ** -0.5 * r.standard_normal((adapters, rank, hidden)), "bf16")
        self.B, self.B64 = rounded(rank ** -0.5 * r.standard_normal((adapters, self.ch + h * d, rank)), "bf16")
        self.s, self.s64 = f32(r.uniform(0.5, 1.5, adapters))
        self.which = r.integers(-1, adapters, self.b)
        self.cw, self.cw64 = f32(0.5 * r.standard_normal((self.ch, 4)))
        self.g, self.g64 = f32(-np.exp2(-np.arange(1, h + 1) * 3.0))
        self.gain, self.gain64 = f32(1 + 0.2 * r.standard_normal(d))
        self.idx = r.permutation(self.b + 1)[:self.b]
        self.conv_pool = torch.zeros(self.b + 1, 3, self.ch, dtype=torch.bfloat16, device=DEV)
        self.pool = torch.zeros(self.b + 1, h, d, d, device=DEV)

    def run(self, x, cu, conv_pool, pool):
        """cu None: one token per request. Returns (row, q, k, v, attention, output)."""
        import gated_deltanet_prefill_gdn_amd as gdn
        row = x @ self.W.t().contiguous()
        which, idx = i64(self.which), i64(self.idx)
        if cu is None:
            gdn.gdn_adapter_decode_fwd(x, row, self.A, self.B, self.s, which, out=row)
            q, k, v = gdn.gdn_conv_decode_fwd(row[:, :self.ch], self.cw, None, conv_pool, idx, dims=(self.h * self.d,) * 3)
        else:
            gdn.gdn_adapter_fwd(x, row, self.A, self.B, self.s, which, i64(cu), out=row)
            q, k, v = gdn.gdn_conv_fwd(row[:, :self.ch], self.cw, None, conv_pool, idx, i64(cu), dims=(self.h * self.d,) * 3)
        q, k, v = (t.unflatten(1, (self.h, self.d)) for t in (q, k, v))
        if cu is None:
            o = gdn.gdn_linear_decode_fwd(q, k, v, self.g, pool, idx)
        else:
            o = gdn.gdn_linear_prefill_fwd(q, k, v, self.g, pool, idx, i64(cu))
        z = row[:, self.ch:].unflatten(1, (self.h, self.d))
        return row, q, k, v, o, gdn.gdn_norm_fwd(o, self.gain, None, z)


def test_layer_with_adapters_over_prompts():
    """Each step against its oracle on what the step before really gave."""
    lay = Layer(1, [90, 1, 300])
    row, q, k, v, o, y = lay.run(lay.x, lay.cu, lay.conv_pool, lay.pool)
    torch.cuda.synchronize()
    h = HALF["bf16"]
    base = np64(lay.x @ lay.W.t().contiguous())
    ref, mag, _ = L.adapter(lay.x64, base, lay.A64, lay.B64, lay.s64, lay.which, lay.cu)
    within(row, ref, h * np.abs(ref) + (1 + h) * 2.0 ** -15 * mag, "chain adapters")
    ref, _, mag, _ = OL.conv_fwd(np64(row)[:, :lay.ch], lay.cw64, None, np.zeros((lay.b + 1, 3, lay.ch)), lay.idx, lay.cu, True)
    got = np.concatenate([np64(t).reshape(lay.n, -1) for t in (q, k, v)], 1)
    within(got, ref, h * np.abs(ref) + 2.0 ** -18 * (1 + mag), "chain convolution")
    ref, new, mag, mags, _ = L.linear_fwd(np64(q), np64(k), np64(v), lay.g64, lay.d ** -0.5,
                                          np.zeros((lay.b + 1, lay.h, lay.d, lay.d)), lay.idx, lay.cu)
    within(o, ref, h * np.abs(ref) + (1 + h) * 2.0 ** -14 * mag + 1e-38, "chain attention")
    within(lay.pool, new, 2.0 ** -16 * mags + 1e-38, "chain states")
    ref, mag = OL.norm_fwd(np64(o), lay.gain64, None, np64(row)[:, lay.ch:].reshape(lay.n, lay.h, lay.d),
                           float(np.float32(1e-6)), True, "last")
    within(y, ref, h * np.abs(ref) + 2.0 ** -18 * (mag + 1), "chain norm")


def test_tokens_after_a_prompt_continue_it():
    """A prompt, then single tokens, against the whole prompt, on the same q, k and v: the two ways of
    the attention are each 2^-14 of their magnitude off, and each is rounded to bf16."""
    import gated_deltanet_prefill_gdn_amd as gdn
    lay = Layer(2, [100, 60])
    _, q, k, v, whole, _ = lay.run(lay.x, lay.cu, lay.conv_pool, lay.pool)
    pool, idx = torch.zeros_like(lay.pool), i64(lay.idx)
    keep = torch.tensor([t for b in range(2) for t in range(lay.cu[b], lay.cu[b + 1] - 6)], device=DEV)
    o = torch.empty_like(whole)
    o[keep] = gdn.gdn_linear_prefill_fwd(q[keep], k[keep], v[keep], lay.g, pool, idx, i64([0, 94, 148]))
    for i in range(6):
        t = torch.tensor([lay.cu[1] - 6 + i, lay.cu[2] - 6 + i], device=DEV)
        o[t] = gdn.gdn_linear_decode_fwd(q[t], k[t], v[t], lay.g, pool, idx)
    torch.cuda.synchronize()
    _, _, mag, mags, _ = L.linear_fwd(np64(q), np64(k), np64(v), lay.g64, lay.d ** -0.5,
                                      np.zeros((3, lay.h, lay.d, lay.d)), lay.idx, lay.cu)
    a, b = np64(o), np64(whole)
    assert (np.abs(a - b) <= 2.0 ** -8 * (np.abs(a) + np.abs(b)) + 2 * 2.0 ** -14 * mag + 1e-38).all()
    assert (np.abs(np64(pool) - np64(lay.pool)) <= 2 * 2.0 ** -16 * mags + 1e-38).all()


def test_layer_token_by_token():
    """The layer over single tokens, each step against its oracle on what the step before gave."""
    lay = Layer(4, [1] * 7)
    conv0, pool0 = torch.randn_like(lay.conv_pool), torch.randn_like(lay.pool)
    row, q, k, v, o, _ = lay.run(lay.x, None, conv_pool=(cp := conv0.clone()), pool=(pp := pool0.clone()))
    torch.cuda.synchronize()
    h = HALF["bf16"]
    ref, mag, _ = L.adapter(lay.x64, np64(lay.x @ lay.W.t().contiguous()), lay.A64, lay.B64, lay.s64, lay.which, lay.cu)
    within(row, ref, h * np.abs(ref) + (1 + h) * 2.0 ** -15 * mag, "steps: adapters")
    ref, new, mag, _ = OL.conv_fwd(np64(row)[:, :lay.ch], lay.cw64, None, np64(conv0), lay.idx, lay.cu, True)
    got = np.concatenate([np64(t).reshape(lay.n, -1) for t in (q, k, v)], 1)
    within(got, ref, h * np.abs(ref) + 2.0 ** -18 * (1 + mag), "steps: convolution")
    np.testing.assert_array_equal(np64(cp), new)
    ref, new, mag, mags, _ = L.linear_fwd(np64(q), np64(k), np64(v), lay.g64, lay.d ** -0.5, np64(pool0), lay.idx, lay.cu)
    within(o, ref, h * np.abs(ref) + (1 + h) * 2.0 ** -14 * mag + 1e-38, "steps: attention")
    within(pp, new, 2.0 ** -16 * mags + 1e-38, "steps: states")


def test_layer_gradients():
    """norm backward -> attention backward -> convolution backward, each against its oracle."""
    import gated_deltanet_prefill_gdn_amd as gdn
    lay = Layer(3, [70, 45])
    conv0, pool0 = lay.conv_pool.clone(), lay.pool.clone()
    row, q, k, v, o, _ = lay.run(lay.x, lay.cu, lay.conv_pool, lay.pool)
    idx, cu = i64(lay.idx), i64(lay.cu)
    dy = torch.randn(o.shape, device=DEV).bfloat16()
    z = row[:, lay.ch:].unflatten(1, (lay.h, lay.d))
    gn = gdn.gdn_norm_bwd(o, lay.gain, None, z, dy)
    gl = gdn.gdn_linear_bwd(q, k, v, lay.g, pool0, idx, cu, gn["dx"])
    gc = gdn.gdn_conv_bwd(row[:, :lay.ch], lay.cw, None, conv0, idx, cu, [gl[n].flatten(1) for n in ("dq", "dk", "dv")])
    torch.cuda.synchronize()
    ref = L.linear_bwd(np64(q), np64(k), np64(v), lay.g64, lay.d ** -0.5, np64(pool0), lay.idx, lay.cu, np64(gn["dx"]), None)
    h = HALF["bf16"]
    for n in ("dq", "dk", "dv"):
        within(gl[n], ref[n], h * np.abs(ref[n]) + (1 + h) * 2.0 ** -14 * ref[n + "_mag"] + 1e-38, "chain " + n)
    ref = OL.conv_bwd(np64(row)[:, :lay.ch], lay.cw64, None, np64(conv0), lay.idx, lay.cu,
                      np.concatenate([np64(gl[n]).reshape(lay.n, -1) for n in ("dq", "dk", "dv")], 1), None, True)
    for n, tol in (("dx", 2.0 ** -8), ("dweight", 1e-5)):
        assert np.linalg.norm(np64(gc[n]) - ref[n]) <= tol * np.linalg.norm(ref[n]), n


def test_other_stream_and_whose_memory():
    """On a stream of the caller's, inputs made there; what a call allocates is memory of that stream."""
    import gated_deltanet_prefill_gdn_amd as gdn
    s = torch.cuda.Stream()
    c, idx, cu = linear_inputs(5, 3000), i64([1, 0]), i64([0, 2600, 3000])
    pool = torch.randn(2, 4, 64, 64, device=DEV)
    p1, p2 = pool.clone(), pool.clone()
    want = gdn.gdn_linear_prefill_fwd(*c, p1, idx, cu)
    gwant = gdn.gdn_linear_bwd(*c, pool, idx, cu, want)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        c2 = [t + 0 for t in c]
    out = gdn.gdn_linear_prefill_fwd(*c2, p2, idx, cu, stream=s)
    g = gdn.gdn_linear_bwd(*c2, pool, idx, cu, out, stream=s)
    one = gdn.gdn_linear_decode_fwd(*(t[:2] for t in c2[:3]), c2[3], p2.clone(), idx, stream=s)
    x, A, B = torch.randn(9, 32, device=DEV), torch.randn(2, 4, 32, device=DEV), torch.randn(2, 40, 4, device=DEV)
    base = torch.randn(9, 44, device=DEV)[:, :40]
    a = gdn.gdn_adapter_fwd(x, base, A, B, torch.ones(2, device=DEV), idx, i64([0, 5, 9]), stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(p1, p2) and all(torch.equal(g[k], gwant[k]) for k in g)
    segments = torch.cuda.memory_snapshot()
    for t in (out, one, a, *g.values()):
        owner, = [m["stream"] for m in segments if m["address"] <= t.data_ptr() < m["address"] + m["total_size"]]
        assert owner == s.cuda_stream


def test_captured_calls_replay_to_the_eager_results():
    """Prompts, gradients and single tokens, two graphs that share a workspace, replayed with new inputs
    between eager work; every replay equals the eager calls bit for bit."""
    import gated_deltanet_prefill_gdn_amd as gdn
    n, cu, idx = 1900, i64([0, 1500, 1500, 1900]), i64([2, 0, 1])
    c = [linear_inputs(6 + i, n, h=1 + i) for i in range(2)]
    pools = [torch.zeros(3, 4, 64, 64, device=DEV) for _ in range(2)]
    prob = [gdn.linear_problem(*c[i][:3], 3, 3) for i in range(2)]
    ws = torch.empty(max(max(gdn.gdn_linear_workspace_size(p), gdn.gdn_linear_bwd_workspace_size(p)) for p in prob),
                     dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(c[i][2]) for i in range(2)]
    one = torch.empty(3, 4, 64, dtype=torch.bfloat16, device=DEV)

    def go(i, pool, out, workspace):
        gdn.gdn_linear_prefill_fwd(*c[i], pool, idx, cu, out=out, workspace=workspace)
        g = gdn.gdn_linear_bwd(*c[i], pool, idx, cu, out, workspace=workspace)
        o = gdn.gdn_linear_decode_fwd(*(t[:3] for t in c[i][:3]), c[i][3], pool, idx)
        return g, o

    for i in range(2):
        go(i, pools[i].clone(), outs[i], ws)
    torch.cuda.synchronize()
    graphs, got = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            got.append(go(i, pools[i], outs[i], ws))
    for p in pools:
        p.zero_()
    eager = [p.clone() for p in pools]
    for step in range(3):
        for i in range(2):
            for t in c[i][:3]:
                t.normal_()
            graphs[i].replay()
        want = []
        for i in range(2):
            out = torch.empty_like(outs[i])
            want.append((out, *go(i, eager[i], out, None)))
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i][0]) and torch.equal(pools[i], eager[i])
            assert torch.equal(got[i][1], want[i][2])
            assert all(torch.equal(got[i][0][k], want[i][1][k]) for k in want[i][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,h,hv,dk,dv", [([1500, 700], 2, 2, 128, 64), ([5003], 1, 3, 64, 128), ([40] * 9, 1, 2, 256, 256),
                                                ([300, 1, 0, 90, 4000], 4, 4, 64, 64)])
def test_nothing_is_written_behind_a_workspace(dtype, lengths, h, hv, dk, dv):
    import gated_deltanet_prefill_gdn_amd as gdn
    cu = np.concatenate([[0], np.cumsum(lengths)])
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    c = linear_inputs(8, int(cu[-1]), h, hv, dk, dv, dt)
    b = len(lengths)
    pool, idx = torch.zeros(b, hv, dv, dk, device=DEV), i64(range(b))
    prob = gdn.linear_problem(*c[:3], b, b)
    for need, call in ((gdn.gdn_linear_workspace_size(prob), lambda w: gdn.gdn_linear_prefill_fwd(*c, pool.clone(), idx, i64(cu), workspace=w)),
                       (gdn.gdn_linear_bwd_workspace_size(prob), lambda w: gdn.gdn_linear_bwd(*c, pool, idx, i64(cu), c[2], workspace=w))):
        wide = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        call(wide[:need] if need else wide[:256])
        torch.cuda.synchronize()
        assert (wide[need if need else 256:] == 0x5A).all()
        if need:
            with pytest.raises(gdn.GdnError):
                call(wide[:need - 1])


@pytest.mark.parametrize("n,k,m,rank,adapters,b", [(4096, 64, 64, 128, 5, 7), (100, 512, 96, 16, 40, 100), (333, 40, 77, 33, 3, 9)])
def test_nothing_is_written_behind_an_adapter_workspace(n, k, m, rank, adapters, b):
    import gated_deltanet_prefill_gdn_amd as gdn
    g = torch.Generator(device=DEV).manual_seed(1)
    rn = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()  # noqa: E731
    x, base, A, B = rn(n, k), rn(n, m), rn(adapters, rank, k), rn(adapters, m, rank)
    cu = i64(np.linspace(0, n, b + 1).astype(int))
    need = gdn.gdn_adapter_workspace_size(gdn.adapter_problem(x, base, A, b))
    wide = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    gdn.gdn_adapter_fwd(x, base, A, B, torch.ones(adapters, device=DEV), i64(np.arange(b) % adapters), cu, workspace=wide[:need])
    torch.cuda.synchronize()
    assert (wide[need:] == 0x5A).all()


def test_calls_without_tokens():
    import gated_deltanet_prefill_gdn_amd as gdn
    c = linear_inputs(9, 0)
    pool = torch.randn(3, 4, 64, 64, device=DEV)
    dstate = torch.randn(2, 4, 64, 64, device=DEV)
    before = pool.clone()
    assert gdn.gdn_linear_prefill_fwd(*c, pool, i64([1, 7]), i64([0, 0, 0])).shape == (0, 4, 64)
    g = gdn.gdn_linear_bwd(*c, pool, i64([1, 7]), i64([0, 0, 0]), c[2], dstate)
    torch.cuda.synchronize()
    assert torch.equal(pool, before) and torch.equal(g["dstate0"][0], dstate[0]) and (g["dstate0"][1] == 0).all()
    assert gdn.gdn_linear_decode_fwd(*c, pool, i64([])).shape == (0, 4, 64)
    A, B = torch.zeros(2, 4, 8, device=DEV), torch.zeros(2, 6, 4, device=DEV)
    e = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    assert gdn.gdn_adapter_fwd(e(0, 8), e(0, 6), A, B, e(2), i64([0]), i64([0, 0])).shape == (0, 6)
    assert gdn.gdn_adapter_decode_fwd(e(0, 8), e(0, 6), A, B, e(2), i64([])).shape == (0, 6)


def test_a_decay_that_is_no_number_stays_in_its_head():
    import gated_deltanet_prefill_gdn_amd as gdn
    c, cu, idx = linear_inputs(10, 700, h=4), i64([0, 700]), i64([0])
    pool = torch.zeros(1, 4, 64, 64, device=DEV)
    p1, p2 = pool.clone(), pool.clone()
    want = gdn.gdn_linear_prefill_fwd(*c, p1, idx, cu)
    c[3] = c[3].clone()
    c[3][1] = float("nan")
    got = gdn.gdn_linear_prefill_fwd(*c, p2, idx, cu)
    torch.cuda.synchronize()
    keep = [0, 2, 3]
    assert torch.equal(got[:, keep], want[:, keep]) and torch.equal(p2[:, keep], p1[:, keep])
    assert got[-1, 1].isnan().all()


@pytest.mark.parametrize("seed", range(12))
def test_random_calls(seed):
    """Shapes, packings, types and strides at random, forward and backward, against the oracle."""
    import test_gpu_linear as T
    r = np.random.default_rng(100 + seed)
    h = int(r.integers(1, 4))
    hv = h * int(r.integers(1, 4))
    dk, dv = (int(r.choice([64, 128, 256])) for _ in range(2))
    b = int(r.integers(1, 9))
    lengths = [int(x) for x in np.exp(r.uniform(0, np.log(900), b)).astype(int) - 1]
    dtype = str(r.choice(["bf16", "f32"]))
    dead = [(int(r.integers(0, b)), -1)] if r.random() < 0.3 else []
    c = T.make(seed, lengths, h, hv, dk, dv, dtype, dead=dead, pad=8 * int(r.integers(0, 5)), tail=int(r.integers(0, 20)))
    what = f"random {dtype} {lengths} H={h} HV={hv} dk={dk} dv={dv}"
    T.check_forward(c, *T.forward(c), what)
    T.check_backward(c, T.backward(c), what)


def test_many_requests_are_not_cut():
    """Above 512 requests none is cut; a long one among them is walked whole."""
    import test_gpu_linear as T
    c = T.make(20, [20] * 520 + [700], 1, 1, 64, 64, "bf16")
    T.check_forward(c, *T.forward(c), "521 requests")
    T.check_backward(c, T.backward(c), "521 requests")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_short_requests_of_a_large_batch(dtype):
    """Mostly single tokens: short requests take the token kernel, the others the chunks."""
    import test_gpu_linear as T
    r = np.random.default_rng(21)
    lengths = [int(x) for x in r.choice([0, 1, 1, 2, 3, 4], 600)] + [90, 5]
    c = T.make(21, lengths, 2, 4, 64, 64, dtype, dead=[(7, -1), (600, 9999)])
    T.check_forward(c, *T.forward(c), f"{dtype} 602 short requests")
    out, _ = T.forward(c, pool=False)
    T.check_forward(c, out, None, f"{dtype} 602 short requests, no pool", pool=False)
