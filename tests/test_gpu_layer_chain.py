"""The layer operators as a layer uses them: convolution, recurrence, gated norm over prompts and
then token by token; the same backwards; on another stream; captured into HIP graphs that are
replayed among other work."""
import numpy as np
import pytest

from layer_util import DEV, f32, i64, np64, rounded
from oracle import layer as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class Layer:
    """Weights, pools and one packed projection row [q | k | v | gate] per token."""

    def __init__(self, seed, lengths, h=2, hv=4, d=64, w=4):
        r = np.random.default_rng(seed)
        self.cu = np.concatenate([[0], np.cumsum(lengths)]).astype(int)
        self.n, self.b, self.h, self.hv, self.d = int(self.cu[-1]), len(lengths), h, hv, d
        self.dims = (h * d, h * d, hv * d)
        self.ch = sum(self.dims)
        self.proj, self.proj64 = rounded(r.standard_normal((self.n, self.ch + hv * d)), "bf16")
        self.wt, self.wt64 = f32(0.5 * r.standard_normal((self.ch, w)))
        self.a, self.a64 = f32(r.standard_normal((self.n, hv)))
        self.bt, self.bt64 = f32(r.standard_normal((self.n, hv)))
        self.A_log, self.A_log64 = f32(np.log(r.uniform(1, 4, hv)))
        self.dtb, self.dtb64 = f32(0.1 * r.standard_normal(hv))
        self.gain, self.gain64 = f32(1 + 0.2 * r.standard_normal(d))
        self.conv_pool = torch.zeros(self.b + 1, w - 1, self.ch, dtype=torch.bfloat16, device=DEV)
        self.state_pool = torch.zeros(self.b + 1, hv, d, d, device=DEV)
        self.idx = r.permutation(self.b + 1)[:self.b]

    def split(self, rows):
        return rows[:, :self.ch], rows[:, self.ch:].unflatten(1, (self.hv, self.d))

    def prefill(self, lo, hi, cu, conv_pool, state_pool):
        import gated_deltanet_prefill_gdn_amd as gdn
        x, z = self.split(self.proj[lo:hi])
        q, k, v = gdn.gdn_conv_fwd(x, self.wt, None, conv_pool, i64(self.idx),
                                   i64(cu), dims=self.dims)
        n = hi - lo
        o = gdn.gdn_prefill_fwd(q.view(n, self.h, self.d), k.view(n, self.h, self.d),
                                v.view(n, self.hv, self.d), self.a[lo:hi], self.bt[lo:hi], self.A_log,
                                self.dtb, state_pool, i64(self.idx),
                                i64(cu))
        return o, gdn.gdn_norm_fwd(o, self.gain, None, z)

    def decode(self, rows, a, b, conv_pool, state_pool, idx):
        import gated_deltanet_prefill_gdn_amd as gdn
        x, z = self.split(rows)
        q, k, v = gdn.gdn_conv_decode_fwd(x, self.wt, None, conv_pool, idx, dims=self.dims)
        m = rows.shape[0]
        o = gdn.gdn_decode_fwd(q.view(m, self.h, self.d), k.view(m, self.h, self.d), v.view(m, self.hv, self.d),
                               a, b, self.A_log, self.dtb, state_pool, idx)
        return o, gdn.gdn_norm_fwd(o, self.gain, None, z)


def test_layer_prompt_then_tokens():
    """A prompt prefilled and continued token by token gives what the whole prompt gives. Both
    ways round the recurrence's outputs to bf16 (2^-8 each) and the chunked one is within 2e-2 of
    their rms beyond that, so two of them differ by at most twice both; the norm of the joined
    outputs, row by row, is the joined norm to the bit."""
    import gated_deltanet_prefill_gdn_amd as gdn
    lay = Layer(1, [90, 70])
    whole, _ = lay.prefill(0, lay.n, lay.cu, lay.conv_pool.clone(), lay.state_pool.clone())
    conv, state, idx = lay.conv_pool.clone(), lay.state_pool.clone(), i64(lay.idx)
    pick = torch.tensor([t for b in range(2) for t in range(lay.cu[b], lay.cu[b + 1] - 8)], device=DEV)
    kept = {k: getattr(lay, k) for k in ("proj", "a", "bt")}
    for k, t in kept.items():
        setattr(lay, k, t[pick].contiguous())
    o, y = torch.empty_like(whole), torch.empty_like(whole)
    o[pick], y[pick] = lay.prefill(0, 144, [0, 82, 144], conv, state)
    for k, t in kept.items():
        setattr(lay, k, t)
    for i in range(8):
        t = torch.tensor([lay.cu[1] - 8 + i, lay.cu[2] - 8 + i], device=DEV)
        o[t], y[t] = lay.decode(lay.proj[t], lay.a[t], lay.bt[t], conv, state, idx)
    torch.cuda.synchronize()
    assert torch.equal(y, gdn.gdn_norm_fwd(o, lay.gain, None, lay.split(lay.proj)[1]))
    a, b = np64(o), np64(whole)
    d, rms = np.abs(a - b), np.sqrt((b ** 2).mean())
    print(f"[layer] pieces against whole: max {d.max() / rms:.2e} of the rms", flush=True)
    assert (d <= 2 * 2e-2 * rms + 2.0 ** -8 * (np.abs(a) + np.abs(b))).all()


def test_layer_gradients_through_all_three():
    """norm backward -> recurrence backward -> convolution backward in the library's calls,
    against the fp64 oracles chained the same way on the same (rounded) intermediates."""
    import gated_deltanet_prefill_gdn_amd as gdn
    from oracle import backward as OB
    import gdn_synth
    lay = Layer(2, [40, 25], h=1, hv=2)
    n, idx, cu = lay.n, i64(lay.idx), i64(lay.cu)
    x, z = lay.split(lay.proj)
    conv0, state0 = lay.conv_pool.clone(), lay.state_pool.clone()
    q, k, v = gdn.gdn_conv_fwd(x, lay.wt, None, lay.conv_pool, idx, cu, dims=lay.dims)
    q3, k3, v3 = q.view(n, 1, 64), k.view(n, 1, 64), v.view(n, 2, 64)
    o = gdn.gdn_prefill_fwd(q3, k3, v3, lay.a, lay.bt, lay.A_log, lay.dtb, lay.state_pool, idx, cu)
    dy = torch.randn(n, 2, 64, device=DEV).bfloat16()
    gn = gdn.gdn_norm_bwd(o, lay.gain, None, z, dy)
    gr = gdn.gdn_prefill_bwd(q3, k3, v3, lay.a, lay.bt, lay.A_log, lay.dtb, state0, idx, cu, gn["dx"],
                             torch.zeros(2, 2, 64, 64, device=DEV))
    gc = gdn.gdn_conv_bwd(x, lay.wt, None, conv0, idx, cu,
                          [gr["dq"].view(n, -1), gr["dk"].view(n, -1), gr["dv"].view(n, -1)])
    torch.cuda.synchronize()
    ref = L.norm_bwd(np64(o), lay.gain64, None, np64(z), np64(dy), float(np.float32(1e-6)), True, "last")
    for kk in ("dx", "dz", "dweight"):
        err = np.linalg.norm(np64(gn[kk]) - ref[kk]) / np.linalg.norm(ref[kk])
        assert err <= 2.0 ** -8, (kk, err)
    ref = L.conv_bwd(np64(x), lay.wt64, None, np64(conv0), lay.idx, lay.cu,
                     np.concatenate([np64(gr[kk]).reshape(n, -1) for kk in ("dq", "dk", "dv")], 1), None, True)
    for kk, tol in (("dx", 2.0 ** -8), ("dweight", 1e-5), ("dstate0", 1e-5)):
        err = np.linalg.norm(np64(gc[kk]) - ref[kk]) / np.linalg.norm(ref[kk])
        assert err <= tol, (kk, err)


def scan_inputs(seed, n, h=1, hv=4, dk=128, dv=64):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    return dict(C=(0.5 * rn(n, h, dk)).bfloat16(), B=(0.5 * rn(n, h, dk)).bfloat16(), x=rn(n, hv, dv).bfloat16(),
                dt=rn(n, hv), A_log=torch.zeros(hv, device=DEV), dt_bias=torch.full((hv,), -3.0, device=DEV),
                D=torch.ones(hv, device=DEV))


def test_other_stream():
    """On a stream of the caller's, inputs made there; nothing runs on the current one."""
    import gated_deltanet_prefill_gdn_amd as gdn
    s = torch.cuda.Stream()
    ones = torch.ones(64, device=DEV)
    pool = torch.zeros(3, 4, 64, 128, device=DEV)
    p2, idx, cu = pool.clone(), i64([2, 0]), i64([0, 100, 357])
    c = scan_inputs(3, 357)
    want = gdn.gdn_ssm_prefill_fwd(*c.values(), p2, idx, cu)
    y2 = gdn.gdn_norm_fwd(want, ones)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        c2 = {k: v + 0 for k, v in c.items()}
    out = gdn.gdn_ssm_prefill_fwd(*c2.values(), pool, idx, cu, stream=s)
    y = gdn.gdn_norm_fwd(out, ones, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(pool, p2) and torch.equal(y, y2)


def test_outputs_belong_to_the_stream_of_the_call():
    """What a call allocates is memory of the stream it runs on: freed, it is not handed to work
    of another stream while the kernels still use it."""
    import gated_deltanet_prefill_gdn_amd as gdn
    s = torch.cuda.Stream()
    c, idx, cu = scan_inputs(4, 300), i64([0]), i64([0, 300])
    pool = torch.zeros(1, 4, 64, 128, device=DEV)
    x, w = torch.randn(300, 64, device=DEV), torch.randn(64, 4, device=DEV)
    rows, scale = torch.randn(300, 1, 64, device=DEV), torch.ones(64, device=DEV)
    torch.cuda.synchronize()
    made = [gdn.gdn_ssm_prefill_fwd(*c.values(), pool, idx, cu, stream=s),
            gdn.gdn_conv_fwd(x, w, None, None, None, cu, stream=s)[0],
            *gdn.gdn_conv_bwd(x, w, None, None, None, cu, (x,), stream=s).values(),
            gdn.gdn_norm_fwd(rows, scale, stream=s),
            *gdn.gdn_norm_bwd(rows, scale, None, rows, rows, stream=s).values()]
    s.synchronize()
    segments = torch.cuda.memory_snapshot()
    for t in made:
        at = t.data_ptr()
        owner, = [g["stream"] for g in segments
                  if g["address"] <= at < g["address"] + g["total_size"]]
        assert owner == s.cuda_stream


def test_captured_layer_replays_to_the_eager_result():
    """Decode steps of a whole layer and a prefill of the scan, each captured once and replayed
    with new inputs between other eager work; two graphs that share a workspace run one after the
    other. Every replay equals the eager calls bit for bit."""
    import gated_deltanet_prefill_gdn_amd as gdn
    lay = Layer(4, [30, 20, 41])
    idx = i64(lay.idx)
    conv, state = lay.conv_pool, lay.state_pool
    rows, a, b = lay.proj[:3].clone(), lay.a[:3].clone(), lay.bt[:3].clone()
    lay.decode(rows, a, b, conv.clone(), state.clone(), idx)  # warm up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, out = lay.decode(rows, a, b, conv, state, idx)
    conv.zero_(), state.zero_()
    econv, estate = conv.clone(), state.clone()
    for step in range(4):
        t = torch.tensor([step, 30 + step, 50 + step], device=DEV)
        rows.copy_(lay.proj[t]), a.copy_(lay.a[t]), b.copy_(lay.bt[t])
        graph.replay()
        _, want = lay.decode(lay.proj[t], lay.a[t], lay.bt[t], econv, estate, idx)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(conv, econv) and torch.equal(state, estate)

    n = 700
    c = [scan_inputs(10 + i, n) for i in range(2)]
    cu, sidx = i64([0, 600, 700]), i64([1, 0])
    ws = torch.empty(gdn.gdn_ssm_workspace_size(gdn.make_problem(n, 2, 1, 4, 128, 64, 2, gdn.GDN_DTYPE_BF16)),
                     dtype=torch.uint8, device=DEV)
    pools = [torch.zeros(2, 4, 64, 128, device=DEV) for _ in range(2)]
    outs = [torch.empty(n, 4, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for i in range(2):
        gdn.gdn_ssm_prefill_fwd(*c[i].values(), pools[i], sidx, cu, out=outs[i], workspace=ws)
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            gdn.gdn_ssm_prefill_fwd(*c[i].values(), pools[i], sidx, cu, out=outs[i], workspace=ws)
    for p in pools:
        p.zero_()
    eager = [torch.zeros(2, 4, 64, 128, device=DEV) for _ in range(2)]
    for step in range(3):
        for i in range(2):
            graphs[i].replay()
        want = [gdn.gdn_ssm_prefill_fwd(*c[i].values(), eager[i], sidx, cu) for i in range(2)]
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i]) and torch.equal(pools[i], eager[i])


def test_captured_backward_replays_to_the_eager_result():
    import gated_deltanet_prefill_gdn_amd as gdn
    lay = Layer(5, [300, 212])
    x, z = lay.split(lay.proj)
    cu, idx = i64(lay.cu), i64(lay.idx)
    o = torch.randn(lay.n, lay.hv, lay.d, device=DEV).bfloat16()
    dy = torch.randn(lay.n, lay.hv, lay.d, device=DEV).bfloat16()
    douts = [torch.randn(lay.n, d, device=DEV) for d in lay.dims]

    def back():
        g = gdn.gdn_norm_bwd(o, lay.gain, None, z, dy)
        return {**g, **{"c" + k: v for k, v in gdn.gdn_conv_bwd(x, lay.wt, None, lay.conv_pool, idx, cu, douts).items()}}

    back()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = back()
    for _ in range(3):
        dy.normal_()
        douts[0].normal_()
        graph.replay()
        want = back()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
