"""Measured cases of two more operators of a recurrent token mixer's layer: linear attention with
a fixed decay for each head (prompts, single tokens, gradients), and the low-rank adapters of many
requests beside the shared projection in front of it (prompts, single tokens).

Requests of different lengths are packed into one row axis (cu_seqlens), recurrent states live in a
pool addressed by cache_indices and adapters in a bank addressed by adapter_indices, as in the
library's other calls.
"""
import math
import random

import torch

own = False

_F32, _F64 = torch.float32, torch.float64
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a ragged prefill batch, 32 heads of 128, q, k and v slices of one projection row with
        # the output gate behind them
        dict(name="linear_ragged_bf16", op="linear_prefill", dtype="bf16", requests=8,
             tokens=33860, ragged=True, groups=32, heads=32, dv=128, dk=128, pad=4096),
        # one very long prompt: the heads and the token axis are all there is to spread
        dict(name="linear_long_bf16", op="linear_prefill", dtype="bf16", requests=1,
             tokens=131072, ragged=False, groups=16, heads=16, dv=128, dk=128, pad=0),
        # heads of 256, value heads sharing queries and keys by two
        dict(name="linear_wide_bf16", op="linear_prefill", dtype="bf16", requests=1,
             tokens=16384, ragged=False, groups=4, heads=8, dv=256, dk=256, pad=0),
        # three short fp32 requests, lengths that end inside a chunk
        dict(name="linear_short_f32", op="linear_prefill", dtype="f32", requests=3, tokens=333,
             ragged=True, groups=8, heads=8, dv=64, dk=64, pad=8),
        # one new token for each of 512 served requests, 1 GiB of touched states
        dict(name="linear_decode_bf16", op="linear_decode", dtype="bf16", requests=512,
             tokens=512, ragged=False, groups=32, heads=32, dv=128, dk=128, pad=4096),
        # one request being answered alone
        dict(name="linear_decode_one_bf16", op="linear_decode", dtype="bf16", requests=1,
             tokens=1, ragged=False, groups=16, heads=16, dv=128, dk=128, pad=0),
        # a training batch of 4 x 4096 tokens, 16 heads of 128
        dict(name="linear_backward_bf16", op="linear_bwd", dtype="bf16", requests=4,
             tokens=16384, ragged=False, groups=16, heads=16, dv=128, dk=128, pad=0),
        # gradients of packed fp32 documents of odd lengths, value heads sharing queries and keys
        dict(name="linear_backward_shared_f32", op="linear_bwd", dtype="f32", requests=5,
             tokens=2047, ragged=True, groups=4, heads=8, dv=128, dk=64, pad=0),
        # adapters of a ragged prefill batch on the packed q/k/v projection
        dict(name="adapter_prompts_bf16", op="adapter", dtype="bf16", requests=8, tokens=33860,
             ragged=True, inputs=4096, outputs=8192, rank=16, adapters=8, pad=4096),
        # many requests of some tokens each, larger adapters
        dict(name="adapter_mixed_bf16", op="adapter", dtype="bf16", requests=64, tokens=4096,
             ragged=True, inputs=4096, outputs=4096, rank=64, adapters=16, pad=0),
        # one new token for each of 512 served requests, 32 adapters among them
        dict(name="adapter_decode_bf16", op="adapter_decode", dtype="bf16", requests=512,
             tokens=512, ragged=False, inputs=4096, outputs=8192, rank=16, adapters=32, pad=4096),
        # short fp32 requests, sizes that no vector width divides
        dict(name="adapter_short_odd_f32", op="adapter", dtype="f32", requests=5, tokens=77,
             ragged=True, inputs=595, outputs=333, rank=5, adapters=3, pad=5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear_prefill", "linear_prefill", "linear_decode", "linear_bwd",
                     "linear_bwd", "adapter", "adapter", "adapter_decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("linear"):
        groups = rng.choice([1, 2, 3, 8, 16])
        heads = groups * rng.choice([1, 1, 1, 2, 4])
        dv, dk = rng.choice([64, 128, 128, 256]), rng.choice([64, 128, 128, 256])
        unit = 128 * 128 / (heads * dv * dk * (4 if dtype == "f32" else 1))
        if op == "linear_decode":
            tokens = requests = _log(rng, 1, max(1, min(512, 512 * 32 * 128 * 128 // (heads * dv * dk))))
        else:
            most = (131072 if op == "linear_prefill" else 16384) * 16 * unit
            tokens = _log(rng, 1, max(1, int(min(65536, most))))
            requests = _log(rng, 1, min(64, tokens))
        return dict(op=op, dtype=dtype, requests=requests, tokens=tokens,
                    ragged=op != "linear_decode" and rng.random() < 0.8, groups=groups,
                    heads=heads, dv=dv, dk=dk, pad=rng.choice([0, 0, 8, 1024]))
    unit = rng.choice([1, 8, 8, 64])
    inputs, outputs = (unit * _log(rng, max(1, 16 // unit), 8192 // unit) for _ in range(2))
    rank = rng.choice([1, 4, 8, 16, 16, 32, 64, 128, _log(rng, 1, 128)])
    adapters = _log(rng, 1, min(64, 1024 // rank))
    if op == "adapter_decode":
        tokens = requests = _log(rng, 1, 512)
    else:
        most = 33860 * (4096 + 8192) // ((inputs + outputs) * (2 if dtype == "f32" else 1))
        tokens = _log(rng, 1, min(65536, most))
        requests = _log(rng, 1, min(64, tokens))
    return dict(op=op, dtype=dtype, requests=requests, tokens=tokens,
                ragged=op == "adapter" and rng.random() < 0.8, inputs=inputs, outputs=outputs,
                rank=rank, adapters=adapters, pad=rng.choice([0, 0, 8, 13, 1024]))


def _lengths(case):
    n, b = case["tokens"], case["requests"]
    if not case["ragged"]:
        return [n // b + (1 if i < n % b else 0) for i in range(b)]
    r = random.Random(1000003 * n + b)
    cuts = [0] + sorted(r.randrange(n + 1) for _ in range(b - 1)) + [n]
    return [cuts[i + 1] - cuts[i] for i in range(b)]


# ---------------------------------------------------------------- inputs

class _State:
    pass


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, mean=0.0, dtype=dt):
        return torch.randn(*shape, device="cuda", generator=g).mul_(scale).add_(mean).to(dtype)

    s = _State()
    s.case, s.op = case, case["op"]
    n, b = case["tokens"], case["requests"]
    lens = torch.tensor(_lengths(case), dtype=torch.int64)
    s.cu_seqlens = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).cuda()
    if s.op.startswith("adapter"):
        k, m, r, na = case["inputs"], case["outputs"], case["rank"], case["adapters"]
        s.x = randn(n, k)
        s.base = randn(n, m + case["pad"])[:, :m]  # the shared projection's rows
        s.A = randn(na, r, k, scale=k ** -0.5)
        s.B = randn(na, m, r, scale=r ** -0.5)
        s.scaling = torch.rand(na, device="cuda", generator=g).add_(0.5)
        # one request in eight has no adapter
        pick = torch.rand(b, device="cuda", generator=g)
        some = torch.randint(0, na, (b,), device="cuda", generator=g)
        s.adapter_indices = torch.where(pick < 0.125, torch.full_like(some, -1), some)
        return s
    hg, hv, dv, dk = case["groups"], case["heads"], case["dv"], case["dk"]
    s.pool_size = b + 3
    s.cache_indices = torch.randperm(s.pool_size, device="cuda", generator=g)[:b].contiguous()
    row = randn(n, 2 * hg * dk + hv * dv + case["pad"], scale=0.8, mean=0.05)
    s.q = row[:, :hg * dk].unflatten(1, (hg, dk))
    s.k = row[:, hg * dk:2 * hg * dk].unflatten(1, (hg, dk))
    s.v = row[:, 2 * hg * dk:2 * hg * dk + hv * dv].unflatten(1, (hv, dv))
    # per-token decays e^-0.84 .. e^-0.004, geometric over the heads
    i = torch.arange(1, hv + 1, device="cuda", dtype=_F32)
    s.log_decay = -torch.exp2(-8 * i / hv)
    s.scale = dk ** -0.5
    s.state_pool = randn(s.pool_size, hv, dv, dk, scale=0.5, dtype=_F32)
    if s.op == "linear_bwd":
        s.dout = randn(n, hv, dv)
        s.dstate = randn(b, hv, dv, dk, scale=0.1, dtype=_F32)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return {"linear_prefill": _linear_prefill, "linear_decode": _linear_decode,
            "linear_bwd": _linear_bwd, "adapter": _adapter, "adapter_decode": _adapter}[state.op](state)


def _run_own(s):
    import gated_deltanet_prefill_gdn_amd as gdn
    if s.op == "linear_prefill":
        out = gdn.gdn_linear_prefill_fwd(s.q, s.k, s.v, s.log_decay, s.state_pool,
                                         s.cache_indices, s.cu_seqlens, scale=s.scale)
        return {"out": out, "state_pool": s.state_pool}
    if s.op == "linear_decode":
        out = gdn.gdn_linear_decode_fwd(s.q, s.k, s.v, s.log_decay, s.state_pool,
                                        s.cache_indices, scale=s.scale)
        return {"out": out, "state_pool": s.state_pool}
    if s.op == "linear_bwd":
        return gdn.gdn_linear_bwd(s.q, s.k, s.v, s.log_decay, s.state_pool, s.cache_indices,
                                  s.cu_seqlens, s.dout, s.dstate, scale=s.scale)
    if s.op == "adapter":
        return gdn.gdn_adapter_fwd(s.x, s.base, s.A, s.B, s.scaling, s.adapter_indices,
                                   s.cu_seqlens)
    return gdn.gdn_adapter_decode_fwd(s.x, s.base, s.A, s.B, s.scaling, s.adapter_indices)


# ---------------------------------------------------------------- plain forms: linear attention

def _walk(s, q, k, v, first, reverse, chunk=128):
    """Linear attention over every request's tokens, forwards or backwards in time: q, k
    [N, HV, dk] and v [N, HV, dv] fp32, first [B, HV, dv, dk] the state in front. Chunks that
    restart at every request: products within a chunk, and between the chunks of a request the
    sums of decayed chunk states. Returns the reads S q and the states behind."""
    n, hv, dk = q.shape
    dv, b, dev = v.shape[2], first.shape[0], q.device
    g = s.log_decay.to(_F64)
    lens = s.cu_seqlens[1:] - s.cu_seqlens[:-1]
    off = torch.cat([torch.zeros_like(lens[:1]), ((lens + chunk - 1) // chunk).cumsum(0)])
    c = torch.arange(n // chunk + b, device=dev)
    live = c < off[-1]
    req = (torch.searchsorted(off, c, right=True) - 1).clamp(max=b - 1)
    head = live & (c == off[req])
    i = torch.arange(chunk, device=dev)
    p = ((c - off[req]) * chunk)[:, None] + i
    valid = live[:, None] & (p < lens[req][:, None])
    at = (s.cu_seqlens[1:][req][:, None] - 1 - p) if reverse else (s.cu_seqlens[req][:, None] + p)
    tok = torch.where(valid, at, n).flatten()

    def chunks(t):  # [N, H, d] -> [chunks, H, tokens, d], zero rows past a request's end
        t = torch.cat([t, torch.zeros_like(t[:1])])[tok]
        return t.unflatten(0, (-1, chunk)).transpose(1, 2).contiguous()

    q, k, v = chunks(q), chunks(k), chunks(v)
    count = valid.sum(1)                                              # tokens of a chunk
    lag = (i[:, None] - i[None, :]).to(_F64)
    decay = torch.exp((lag * g[:, None, None]).masked_fill_(lag < 0, float("-inf"))).float()
    y = torch.matmul(torch.matmul(q, k.transpose(2, 3).contiguous()) * decay, v)
    left = (count[:, None] - 1 - i[None, :]).clamp(min=0).to(_F64)    # tokens behind, in the chunk
    to_end = torch.exp(g[None, :, None] * left[:, None, :]).float()
    local = torch.matmul((v * to_end[..., None]).transpose(2, 3).contiguous(), k)
    # states behind every chunk
    end = g[:, None] * count.cumsum(0).to(_F64)                       # [H, chunks]
    start = end - g[:, None] * count.to(_F64)
    same = (req[:, None] == req[None, :]) & (c[:, None] >= c[None, :]) & live[:, None]
    m = (end[:, :, None] - end[:, None, :]).masked_fill_(~same, float("-inf"))
    m = torch.exp(m).float()
    from0 = torch.exp(end - start[:, off[req].clamp(max=c.numel() - 1)]).float()
    after = torch.matmul(m, local.transpose(0, 1).flatten(2)).unflatten(2, (dv, dk))
    del m, local
    after = after.transpose(0, 1) + from0.t()[..., None, None] * first[req]
    before = torch.where(head[:, None, None, None], first[req], after[(c - 1).clamp(min=0)])
    into = torch.exp(g[:, None] * (i + 1).to(_F64)).float()
    y += into[..., None] * torch.matmul(q, before.transpose(2, 3).contiguous())
    out = torch.zeros(n + 1, hv, dv, device=dev, dtype=_F32)
    out[tok] = y.transpose(1, 2).flatten(0, 1)
    last = (off[1:] - 1).clamp(min=0)
    return out[:n], torch.where((lens > 0)[:, None, None, None], after[last], first)


def _heads(s, t):
    return t.float().repeat_interleave(s.case["heads"] // s.case["groups"], 1)


def _linear_prefill(s):
    out, s.state_pool[s.cache_indices] = _walk(s, _heads(s, s.q), _heads(s, s.k), s.v.float(),
                                               s.state_pool[s.cache_indices], False)
    return {"out": (out * s.scale).to(s.v.dtype), "state_pool": s.state_pool}


def _linear_decode(s):
    q, k, v = _heads(s, s.q), _heads(s, s.k), s.v.float()
    st = s.state_pool[s.cache_indices] * torch.exp(s.log_decay)[:, None, None]
    st += v[..., :, None] * k[..., None, :]
    s.state_pool[s.cache_indices] = st
    return {"out": ((st * q[..., None, :]).sum(-1) * s.scale).to(s.v.dtype),
            "state_pool": s.state_pool}


def _linear_bwd(s):
    """dq reads the forward states with dout; dk and dv read the states' gradients, which run
    backwards in time and take in q and dout as the forward ones take in k and v."""
    q, k, v, do = _heads(s, s.q) * s.scale, _heads(s, s.k), s.v.float(), s.dout.float()
    groups = (s.case["groups"], s.case["heads"] // s.case["groups"])
    out = {}
    first = s.state_pool[s.cache_indices].transpose(2, 3).contiguous()
    dq, _ = _walk(s, do, v, k, first, False)
    out["dq"] = (dq * s.scale).unflatten(1, groups).sum(2).to(s.q.dtype)
    # walking backwards a read follows its token's write, and the decay comes before it: the
    # state behind the last token is decayed by none
    back = s.dstate * torch.exp(-s.log_decay)[:, None, None]
    dv, behind = _walk(s, k, q, do, back, True)
    out["dv"] = dv.to(s.v.dtype)
    dk, _ = _walk(s, v, do, q, back.transpose(2, 3).contiguous(), True)
    out["dk"] = dk.unflatten(1, groups).sum(2).to(s.k.dtype)
    out["dstate0"] = behind * torch.exp(s.log_decay)[:, None, None]
    return out


# ---------------------------------------------------------------- plain forms: adapters

def _adapter(s):
    """All adapters' products at once, those of other adapters masked."""
    n, na, r = s.x.shape[0], s.case["adapters"], s.case["rank"]
    t = torch.arange(n, device=s.x.device)
    req = torch.searchsorted(s.cu_seqlens, t, right=True) - 1
    mine = s.adapter_indices[req]
    h = torch.matmul(s.x.float(), s.A.float().flatten(0, 1).t().contiguous())
    mask = (mine[:, None] == torch.arange(na, device=t.device)).float() * s.scaling
    h = (h.unflatten(1, (na, r)) * mask[..., None]).flatten(1)
    delta = torch.matmul(h, s.B.float().transpose(1, 2).flatten(0, 1).contiguous())
    return (s.base.float() + delta).to(s.base.dtype)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if s.op.startswith("adapter"):
            return _exact_adapter(s)
        return _exact_bwd(s) if s.op == "linear_bwd" else _exact_linear(s)


def _rows(t):  # fp64, with a row of zeros for the requests that have ended
    return torch.cat([t.double(), torch.zeros_like(t[:1], dtype=_F64)])


def _exact_linear(s):
    """Token by token, all requests side by side."""
    n, hv, dv = s.v.shape
    rep = hv // s.q.shape[1]
    q, k = (_rows(t).repeat_interleave(rep, 1) for t in (s.q, s.k))
    q, k, v = q[..., :, None], k[..., None, :], _rows(s.v)[..., :, None]
    a = torch.exp(s.log_decay.double())[:, None, None]
    pool = s.state_pool.double()
    st = pool[s.cache_indices]
    begin, lens = s.cu_seqlens[:-1], s.cu_seqlens[1:] - s.cu_seqlens[:-1]
    out = torch.zeros(n + 1, hv, dv, 1, device=v.device, dtype=_F64)
    counts = _lengths(s.case)
    if len(counts) == 1:
        for t in range(n):
            st.mul_(a).addcmul_(v[t], k[t])
            torch.matmul(st, q[t], out=out[t:t + 1])
    else:
        for t in range(max(counts)):
            i = torch.where(t < lens, begin + t, n)
            live = (t < lens)[:, None, None, None]
            st.mul_(torch.where(live, a, torch.ones_like(a))).addcmul_(v[i], k[i])
            out[i] = torch.matmul(st, q[i])
    pool[s.cache_indices] = st
    return {"out": out[:n, :, :, 0] * s.scale, "state_pool": pool}


def _exact_bwd(s):
    """The recurrence token by token and its adjoint from the last token to the first."""
    n, hv, dv = s.v.shape
    rep, dk = hv // s.q.shape[1], s.q.shape[2]
    q, k = (_rows(t).repeat_interleave(rep, 1) for t in (s.q, s.k))
    v, do = _rows(s.v), _rows(s.dout)
    a = torch.exp(s.log_decay.double())[:, None, None]
    one = torch.ones_like(a)
    begin, lens = s.cu_seqlens[:-1], s.cu_seqlens[1:] - s.cu_seqlens[:-1]
    dq, dkk = (torch.zeros(n + 1, hv, dk, device=v.device, dtype=_F64) for _ in range(2))
    dvv = torch.zeros(n + 1, hv, dv, device=v.device, dtype=_F64)
    longest = max(_lengths(s.case))
    st = s.state_pool[s.cache_indices].double()
    for t in range(longest):
        i = torch.where(t < lens, begin + t, n)
        st.mul_(torch.where((t < lens)[:, None, None, None], a, one))
        st.addcmul_(v[i][..., :, None], k[i][..., None, :])
        dq[i] = s.scale * torch.matmul(do[i][..., None, :], st)[..., 0, :]
    ds = s.dstate.double()
    for t in reversed(range(longest)):
        live = (t < lens)[:, None, None, None]
        i = torch.where(t < lens, begin + t, n)
        ds.addcmul_(do[i][..., :, None], s.scale * q[i][..., None, :])
        dvv[i] = torch.matmul(ds, k[i][..., :, None])[..., 0]
        dkk[i] = torch.matmul(v[i][..., None, :], ds)[..., 0, :]
        ds.mul_(torch.where(live, a, one))
    return {"dq": dq[:n].unflatten(1, (-1, rep)).sum(2), "dv": dvv[:n],
            "dk": dkk[:n].unflatten(1, (-1, rep)).sum(2), "dstate0": ds}


def _exact_adapter(s):
    """Request by request."""
    out = s.base.double()
    for b, (a, lo, hi) in enumerate(zip(s.adapter_indices.tolist(), s.cu_seqlens[:-1].tolist(),
                                        s.cu_seqlens[1:].tolist())):
        if a >= 0 and hi > lo:
            low = torch.matmul(s.x[lo:hi].double(), s.A[a].double().t())
            out[lo:hi] += s.scaling[a].double() * torch.matmul(low, s.B[a].double().t())
    return out


# ---------------------------------------------------------------- work

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    n, b = case["tokens"], case["requests"]
    if case["op"].startswith("adapter"):
        k, m, r = case["inputs"], case["outputs"], case["rank"]
        used = min(case["adapters"], b)
        return {"bytes": n * es * (k + 2 * m) + used * r * (k + m) * es + 16 * b,
                "flops": 2 * n * r * (k + m)}
    hg, hv, dv, dk = case["groups"], case["heads"], case["dv"], case["dk"]
    states = 4 * b * hv * dv * dk
    rows = n * es * (2 * hg * dk + hv * dv)  # q, k and v
    # the recurrence itself: decay, write and read of a state by every token
    if case["op"] == "linear_bwd":
        return {"bytes": 2 * rows + n * es * hv * dv + 3 * states + 16 * b,
                "flops": 12 * n * hv * dv * dk}
    return {"bytes": rows + n * es * hv * dv + 2 * states + 16 * b,
            "flops": 5 * n * hv * dv * dk}
