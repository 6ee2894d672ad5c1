"""Host-side checks of linear attention and of the adapters, through the C ABI (dummy pointers: every
call here is refused, or has nothing to do, before any launch) and through the binding (CPU tensors)."""
import ctypes

import pytest
import torch

import gated_deltanet_prefill_gdn_amd as gdn

P = ctypes.c_void_p
BIG = 1 << 42
INV, UNS, WS, OK = (gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE, gdn.GDN_OK)
POINTERS = {"prefill": 8, "decode": 7, "bwd": 13}


def prob(n=64, b=4, pool=8, qs=None, ks=None, vs=None, h=2, hv=4, dk=128, dv=64, dtype=gdn.GDN_DTYPE_BF16,
         scale=1.0, flags=0, res=0):
    return gdn.GdnLinearProblem(n, b, pool, h * dk if qs is None else qs, h * dk if ks is None else ks,
                                hv * dv if vs is None else vs, h, hv, dk, dv, dtype, scale, flags, res)


def linear(kind, null=(), nonnull=True, misalign=None, ws=BIG, ws_ptr=1 << 20, **kw):
    a = [P(4096) if nonnull else None] * POINTERS[kind]
    for i in null:
        a[i] = None
    if misalign is not None:
        a[misalign] = P(4096 + 8)
    lib, p = gdn.load_library(), prob(**kw)
    if kind == "decode":
        return lib.gdn_linear_decode_fwd(*a, ctypes.byref(p), None)
    fn = lib.gdn_linear_prefill_fwd if kind == "prefill" else lib.gdn_linear_bwd
    return fn(*a, ctypes.byref(p), P(ws_ptr), ws, None)


@pytest.mark.parametrize("kind", list(POINTERS))
def test_linear_refusals(kind):
    n = dict(n=4) if kind == "decode" else {}
    for kw in (dict(n=-1), dict(b=-1), dict(pool=-1), dict(h=0), dict(hv=0), dict(h=3), dict(dk=0), dict(dv=-64),
               dict(dtype=2), dict(flags=1), dict(res=1), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(qs=255), dict(ks=248), dict(vs=192), dict(qs=260), dict(ks=257), dict(vs=258),
               dict(vs=258, dtype=gdn.GDN_DTYPE_F32), dict(pool=0)):
        assert linear(kind, **{**n, **kw}) == INV, kw
    for kw in (dict(dk=96), dict(dv=32), dict(dk=512), dict(h=1, hv=70000), dict(qs=1 << 23), dict(vs=1 << 23),
               dict(h=1 << 15, hv=1 << 15, dk=256)):
        assert linear(kind, **{**n, **kw}) == UNS, kw
    big = (1 << 28) if kind == "decode" else (1 << 30)
    assert linear(kind, n=big, b=1 << 28, h=1, hv=1024, pool=1 << 28) == UNS  # beyond the grid limits
    assert linear(kind, nonnull=False, **n) == INV
    required = {"prefill": (0, 1, 2, 3, 5, 6, 7), "decode": range(7), "bwd": (0, 1, 2, 3, 5, 6, 7, 9, 10, 11)}[kind]
    for i in required:
        assert linear(kind, null=(i,), **n) == INV, i
    aligned = {"prefill": (0, 1, 2, 4, 7), "decode": (0, 1, 2, 4, 6), "bwd": (0, 1, 2, 4, 7, 8, 9, 10, 11, 12)}[kind]
    for i in aligned:
        assert linear(kind, misalign=i, **n) == INV, i
    lib = gdn.load_library()
    assert {"prefill": lambda: lib.gdn_linear_prefill_fwd(*[None] * 10, 0, None),
            "decode": lambda: lib.gdn_linear_decode_fwd(*[None] * 9),
            "bwd": lambda: lib.gdn_linear_bwd(*[None] * 15, 0, None)}[kind]() == INV


def test_linear_limits():
    assert linear("bwd", h=1, hv=32768, dk=256, dv=64) == UNS  # rows of the partial sums
    assert linear("bwd", n=0, b=0, pool=0, nonnull=False, ws=0, ws_ptr=0) == OK
    # many requests, or hardly more than one token each: none is cut, and nothing has to be kept
    for n, b in ((513 * 64, 513), (15 * 100, 100), (100, 100), (64, 1)):
        assert gdn.gdn_linear_workspace_size(prob(n=n, b=b, h=1, hv=1)) == 0, (n, b)
    assert gdn.gdn_linear_workspace_size(prob(n=100000, b=1, h=1, hv=1)) > 0


@pytest.mark.parametrize("kind", ["prefill", "bwd"])
@pytest.mark.parametrize("dtype", [gdn.GDN_DTYPE_BF16, gdn.GDN_DTYPE_F32])
def test_linear_workspace_holds_the_states_of_cut_requests_and_no_more(kind, dtype):
    """Pieces are whole multiples of 64 tokens, at least 128 of them: a piece's state is kept once (and
    once more for gradients), so the workspace is never above that of pieces of 128 tokens."""
    size = gdn.gdn_linear_workspace_size if kind == "prefill" else gdn.gdn_linear_bwd_workspace_size
    for n, b, h, dk, dv in ((131072, 1, 16, 128, 128), (33860, 8, 32, 128, 128), (4096, 1, 2, 256, 64),
                            (2047, 5, 4, 64, 128), (600, 512, 1, 64, 64), (8192, 512, 4, 64, 64)):
        state = h * dk * dv * 4
        most = (n // 128 + min(b, n // 128)) * state * (1 if kind == "prefill" else 2)
        need = size(prob(n=n, b=b, h=h, hv=h, dk=dk, dv=dv, dtype=dtype))
        assert need <= most + 512 and need % state < 512, (n, b, need)


def test_linear_workspaces_and_empty_calls():
    for kind, size in (("prefill", gdn.gdn_linear_workspace_size), ("bwd", gdn.gdn_linear_bwd_workspace_size)):
        kw = dict(n=100000, b=1)
        need = size(prob(**kw))
        assert need % 256 == 0 and size(prob(dk=96)) == 0
        if need:
            assert linear(kind, ws=need - 1, **kw) == WS and linear(kind, ws_ptr=0, **kw) == WS
            assert linear(kind, ws_ptr=(1 << 20) + 128, **kw) == WS
        assert linear(kind, b=0, pool=0, nonnull=False, ws=0, ws_ptr=0) == OK
    assert linear("prefill", n=0, nonnull=False, ws=0, ws_ptr=0) == OK
    assert linear("decode", n=0, b=0, pool=0, nonnull=False) == OK
    assert linear("decode", n=5, b=4) == INV


def aprob(n=64, b=4, xs=None, bs=None, os=None, k=96, m=80, r=16, adapters=3, dtype=gdn.GDN_DTYPE_BF16, res=0):
    return gdn.GdnAdapterProblem(n, b, k if xs is None else xs, m if bs is None else bs, m if os is None else os,
                                 k, m, r, adapters, dtype, res)


def adapter(decode=False, null=(), nonnull=True, ws=BIG, ws_ptr=1 << 20, same=False, **kw):
    a = [P(4096 * (i + 1)) if nonnull else None for i in range(7 if decode else 8)]
    if same:
        a[-1] = a[1]
    for i in null:
        a[i] = None
    lib, p = gdn.load_library(), aprob(**kw)
    fn = lib.gdn_adapter_decode_fwd if decode else lib.gdn_adapter_fwd
    return fn(*a, ctypes.byref(p), P(ws_ptr), ws, None)


@pytest.mark.parametrize("decode", [False, True])
def test_adapter_refusals(decode):
    n = dict(n=4) if decode else {}
    for kw in (dict(n=-1), dict(b=-1), dict(k=0), dict(m=0), dict(r=0), dict(adapters=-1), dict(dtype=3), dict(res=1),
               dict(xs=95), dict(bs=79), dict(os=79), dict(same=True, os=96)):
        assert adapter(decode, **{**n, **kw}) == INV, kw
    for kw in (dict(r=129), dict(adapters=4097), dict(k=1 << 21, xs=1 << 21), dict(xs=1 << 31), dict(m=1 << 21, bs=1 << 22, os=1 << 22)):
        assert adapter(decode, **{**n, **kw}) == UNS, kw
    assert adapter(decode, nonnull=False, **n) == INV
    for i in range(7 if decode else 8):
        assert adapter(decode, null=(i,), **n) == INV, i
    lib = gdn.load_library()
    assert (lib.gdn_adapter_decode_fwd(*[None] * 9, 0, None) if decode
            else lib.gdn_adapter_fwd(*[None] * 10, 0, None)) == INV


def test_adapter_workspace_and_empty_calls():
    need = gdn.gdn_adapter_workspace_size(aprob())
    assert need % 256 == 0 and gdn.gdn_adapter_workspace_size(aprob(r=129)) == 0
    if need:
        assert adapter(ws=need - 1) == WS and adapter(ws_ptr=0) == WS and adapter(ws_ptr=(1 << 20) + 128) == WS
    assert adapter(n=0, nonnull=False, ws=0, ws_ptr=0) == OK and adapter(b=0, nonnull=False, ws=0, ws_ptr=0) == OK
    assert adapter(True, n=5, b=4) == INV


# ---- the binding

F32 = torch.float32
CU, IDX = torch.tensor([0, 3, 6]), torch.tensor([1, 0])


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def linear_args(**kw):
    a = dict(q=z(6, 2, 64), k=z(6, 2, 64), v=z(6, 4, 64), log_decay=z(4, dtype=F32),
             state_pool=z(3, 4, 64, 64, dtype=F32), cache_indices=IDX, cu_seqlens=CU)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(v=z(6, 4, 64, dtype=torch.float16)), TypeError),
    (dict(q=z(6, 128)), ValueError),
    (dict(k=z(6, 2, 64, dtype=F32)), TypeError),
    (dict(q=z(6, 1, 64)), ValueError),
    (dict(k=z(5, 2, 64)), ValueError),
    (dict(v=z(64, 4, 6).permute(2, 1, 0)), ValueError),
    (dict(q=z(1, 2, 64).expand(6, 2, 64)), ValueError),
    (dict(log_decay=z(4)), TypeError),
    (dict(log_decay=z(5, dtype=F32)), ValueError),
    (dict(state_pool=z(3, 4, 64, 32, dtype=F32)), ValueError),
    (dict(state_pool=z(3, 4, 64, 64)), TypeError),
    (dict(cache_indices=None), ValueError),
    (dict(cache_indices=IDX.int()), TypeError),
    (dict(cu_seqlens=torch.tensor([0, 6])), ValueError),
    ({}, ValueError),  # CPU tensors
])
def test_linear_binding_refusals(kw, err):
    with pytest.raises(err):
        gdn.gdn_linear_prefill_fwd(**linear_args(**kw))
    with pytest.raises(err):
        gdn.gdn_linear_bwd(**linear_args(dout=z(6, 4, 64), **kw))


def test_linear_other_binding_refusals():
    with pytest.raises(ValueError):
        gdn.gdn_linear_prefill_fwd(**linear_args(out=z(6, 4, 32)))
    for kw, err in ((dict(dout=z(6, 4, 64, dtype=F32)), TypeError), (dict(dout=z(5, 4, 64)), ValueError),
                    (dict(dstate=z(2, 4, 64, 32, dtype=F32)), ValueError),
                    (dict(dstate=z(3, 4, 64, 64, dtype=F32)), ValueError),
                    (dict(cu_seqlens=None, cache_indices=torch.arange(6)), ValueError)):
        with pytest.raises(err):
            gdn.gdn_linear_bwd(**{**linear_args(dout=z(6, 4, 64)), **kw})
    a = linear_args()
    a.pop("cu_seqlens")
    for kw in ({}, dict(state_pool=None), dict(cache_indices=None)):  # two indices for six rows
        with pytest.raises(ValueError):
            gdn.gdn_linear_decode_fwd(**{**a, **kw})


def adapter_args(**kw):
    a = dict(x=z(6, 24), base=z(6, 40), A=z(3, 8, 24), B=z(3, 40, 8), scaling=z(3, dtype=F32), adapter_indices=IDX,
             cu_seqlens=CU)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(x=z(6, 24, dtype=torch.float16)), TypeError),
    (dict(x=z(5, 24)), ValueError),
    (dict(base=z(6, 40, 1)), ValueError),
    (dict(base=z(6, 40, dtype=F32)), TypeError),
    (dict(base=z(40, 6).t()), ValueError),
    (dict(base=z(1, 40).expand(6, 40)), ValueError),
    (dict(A=z(3, 8, 25)), ValueError),
    (dict(A=z(8, 24)), ValueError),
    (dict(A=z(3, 24, 8).transpose(1, 2)), ValueError),
    (dict(B=z(3, 8, 40)), ValueError),
    (dict(B=z(2, 40, 8)), ValueError),
    (dict(scaling=z(3)), TypeError),
    (dict(scaling=z(2, dtype=F32)), ValueError),
    (dict(adapter_indices=IDX.int()), TypeError),
    (dict(cu_seqlens=torch.tensor([0, 6])), ValueError),
    (dict(cu_seqlens=None), ValueError),
    (dict(out=z(6, 41)), ValueError),
    (dict(out=z(6, 40, dtype=F32)), TypeError),
    ({}, ValueError),
])
def test_adapter_binding_refusals(kw, err):
    with pytest.raises(err):
        gdn.gdn_adapter_fwd(**adapter_args(**kw))


def test_adapter_decode_binding_refusals():
    a = adapter_args()
    a.pop("cu_seqlens")
    with pytest.raises(ValueError):
        gdn.gdn_adapter_decode_fwd(**a)
