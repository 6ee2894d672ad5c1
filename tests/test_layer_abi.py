"""Host-side checks of the layer operators, through the C ABI (dummy pointers: every call here is
refused, or has nothing to do, before any launch) and through the binding (CPU tensors, whose
shapes, types and strides are checked before the device is)."""
import ctypes
import os
import re

import pytest
import torch

import gated_deltanet_prefill_gdn_amd as gdn

P = ctypes.c_void_p
BIG = 1 << 40


def conv_prob(n=64, b=4, pool=8, stride=48, dx_stride=48, ch=(16, 16, 16), w=4,
              dtype=gdn.GDN_DTYPE_BF16, dout=gdn.GDN_DTYPE_F32, flags=gdn.GDN_CONV_SILU, res=0):
    return gdn.GdnConvProblem(n, b, pool, stride, dx_stride, (ctypes.c_int32 * 3)(*ch), w, dtype,
                              dout, flags, res)


def conv(kind="fwd", nonnull=True, null=(), ws=BIG, ws_ptr=1 << 20, **kw):
    p = conv_prob(**kw)
    a = [P(4096) if nonnull else None] * {"fwd": 9, "decode": 8, "bwd": 14}[kind]
    for i in null:
        a[i] = None
    fn = getattr(gdn.load_library(), {"fwd": "gdn_conv_fwd", "decode": "gdn_conv_decode_fwd",
                                      "bwd": "gdn_conv_bwd"}[kind])
    tail = [P(ws_ptr), ws, None] if kind == "bwd" else [None]
    return fn(*a, ctypes.byref(p), *tail)


INV, UNS, WS, OK = (gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE,
                    gdn.GDN_OK)


@pytest.mark.parametrize("kind", ["fwd", "decode", "bwd"])
def test_conv_refusals(kind):
    n = dict(n=4) if kind == "decode" else {}
    for kw in (dict(n=-1), dict(b=-1), dict(pool=-1), dict(stride=47), dict(ch=(0, 16, 16)),
               dict(ch=(16, -1, 16)), dict(dtype=2), dict(dout=5), dict(flags=2), dict(res=1),
               dict(w=0), dict(pool=0)):
        assert conv(kind, **{**n, **kw}) == INV, kw
    for kw in (dict(w=1), dict(w=5), dict(ch=(1 << 25, 0, 0), stride=1 << 26, dx_stride=1 << 26),
               dict(stride=1 << 29)):
        assert conv(kind, **{**n, **kw}) == UNS, kw
    assert conv(kind, nonnull=False, **n) == INV
    for i in {"fwd": (0, 1, 4, 5, 6, 7, 8), "decode": (0, 1, 3, 4, 5, 6, 7),
              "bwd": (0, 1, 4, 5, 6, 7, 8, 10, 11, 12)}[kind]:
        assert conv(kind, null=(i,), **n) == INV, i
    fn = {"fwd": lambda L: L.gdn_conv_fwd(*[None] * 11),
          "decode": lambda L: L.gdn_conv_decode_fwd(*[None] * 10),
          "bwd": lambda L: L.gdn_conv_bwd(*[None] * 16, 0, None)}[kind]
    assert fn(gdn.load_library()) == INV


def test_conv_decode_takes_one_token_per_request():
    assert conv("decode", n=5, b=4) == INV


def test_conv_backward_workspace():
    need = gdn.gdn_conv_bwd_workspace_size(conv_prob())
    assert need > 0 and need % 256 == 0
    assert gdn.gdn_conv_bwd_workspace_size(conv_prob(w=7)) == 0
    assert conv("bwd", ws=need - 1) == WS
    assert conv("bwd", ws_ptr=(1 << 20) + 64) == WS
    assert conv("bwd", ws_ptr=0) == WS
    assert conv("bwd", dx_stride=40) == INV
    assert conv("bwd", null=(2,)) == INV  # a dbias without a bias


def test_conv_grid_limits():
    assert conv("fwd", n=1 << 31, b=1, ch=(1 << 24, 0, 0), stride=1 << 24) == UNS


def test_conv_without_tokens_is_a_no_op():
    assert conv("fwd", n=0, nonnull=False) == OK
    assert conv("fwd", b=0, nonnull=False) == OK
    assert conv("decode", n=0, b=0, nonnull=False) == OK


def ssm(kind="prefill", n=64, b=4, h=2, hv=4, dk=128, dv=64, pool=8, dtype=gdn.GDN_DTYPE_BF16,
        flags=0, null=(), nonnull=True, misalign=None, ws=BIG, ws_ptr=1 << 20):
    p = gdn.make_problem(n, b, h, hv, dk, dv, pool, dtype, flags)
    k = 11 if kind == "prefill" else 10
    a = [P(4096) if nonnull else None] * k
    for i in null:
        a[i] = None
    if misalign is not None:
        a[misalign] = P(4096 + 8)
    lib = gdn.load_library()
    if kind == "prefill":
        return lib.gdn_ssm_prefill_fwd(*a, ctypes.byref(p), P(ws_ptr), ws, None)
    return lib.gdn_ssm_decode_fwd(*a, ctypes.byref(p), None)


@pytest.mark.parametrize("kind", ["prefill", "decode"])
def test_ssm_refusals(kind):
    n = dict(n=4) if kind == "decode" else {}
    for kw in (dict(n=-1), dict(b=-1), dict(pool=-1), dict(h=0), dict(hv=0), dict(h=3), dict(dk=0),
               dict(dv=-64), dict(dtype=2), dict(flags=1), dict(pool=0)):
        assert ssm(kind, **{**n, **kw}) == INV, kw
    for kw in (dict(dk=96), dict(dv=32), dict(h=1, hv=70000)):
        assert ssm(kind, **{**n, **kw}) == UNS, kw
    big = (1 << 28) if kind == "decode" else (1 << 30)
    assert ssm(kind, n=big, b=1 << 28, h=1, hv=1024, pool=1 << 28) == UNS  # beyond the grid limits
    assert ssm(kind, nonnull=False, **n) == INV
    last = 10 if kind == "prefill" else 9
    for i in [i for i in range(last + 1) if i != 6]:
        assert ssm(kind, null=(i,), **n) == INV, i
    for i in (0, 1, 2, 7, last):
        assert ssm(kind, misalign=i, **n) == INV, i
    lib = gdn.load_library()
    assert (lib.gdn_ssm_prefill_fwd(*[None] * 13, 0, None) if kind == "prefill"
            else lib.gdn_ssm_decode_fwd(*[None] * 12)) == INV


def test_ssm_workspace_and_empty_calls():
    need = gdn.gdn_ssm_workspace_size(gdn.make_problem(64, 4, 2, 4, 128, 64, 8, 1))
    assert need > 0 and need % 256 == 0
    assert gdn.gdn_ssm_workspace_size(gdn.make_problem(64, 4, 2, 4, 96, 64, 8, 1)) == 0
    assert ssm(ws=need - 1) == WS and ssm(ws_ptr=0) == WS and ssm(ws_ptr=(1 << 20) + 128) == WS
    assert ssm("decode", n=5, b=4) == INV
    assert ssm(n=0, nonnull=False, ws=0, ws_ptr=0) == OK
    assert ssm(b=0, pool=0, nonnull=False, ws=0, ws_ptr=0) == OK
    assert ssm("decode", n=0, b=0, pool=0, nonnull=False) == OK


def norm_prob(n=8, xs=256, zs=256, dzs=256, heads=2, dim=128, dtype=gdn.GDN_DTYPE_BF16, flags=0,
              eps=1e-6, res=0):
    return gdn.GdnNormProblem(n, xs, zs, dzs, heads, dim, dtype, flags, eps, res)


def norm(kind="fwd", null=(), nonnull=True, ws=BIG, ws_ptr=1 << 20, **kw):
    p = norm_prob(**kw)
    a = [P(4096) if nonnull else None] * (5 if kind == "fwd" else 9)
    for i in null:
        a[i] = None
    lib = gdn.load_library()
    if kind == "fwd":
        return lib.gdn_norm_fwd(*a, ctypes.byref(p), None)
    return lib.gdn_norm_bwd(*a, ctypes.byref(p), P(ws_ptr), ws, None)


@pytest.mark.parametrize("kind", ["fwd", "bwd"])
def test_norm_refusals(kind):
    for kw in (dict(n=-1), dict(heads=0), dict(dim=0), dict(dtype=9), dict(flags=4), dict(eps=-1.0),
               dict(eps=float("nan")), dict(res=3), dict(xs=255), dict(zs=255),
               dict(flags=gdn.GDN_NORM_GATE_FIRST, null=(3,))):
        assert norm(kind, **kw) == INV, kw
    wide = dict(xs=1 << 29, zs=1 << 29, dzs=1 << 29)
    assert norm(kind, dim=16385, **wide) == UNS
    assert norm(kind, dim=16384, heads=1 << 15, **wide) == UNS
    assert norm(kind, nonnull=False) == INV
    for i in ((0, 1, 4) if kind == "fwd" else (0, 1, 4, 5, 6, 7, 8, 2, 3)):
        assert norm(kind, null=(i,)) == INV, i


def test_norm_backward_workspace_and_empty_call():
    need = gdn.gdn_norm_bwd_workspace_size(norm_prob())
    assert need > 0 and need % 256 == 0
    assert gdn.gdn_norm_bwd_workspace_size(norm_prob(dim=0)) == 0
    assert norm("bwd", ws=need - 1) == WS and norm("bwd", ws_ptr=0) == WS
    assert norm("bwd", dzs=100) == INV
    assert norm("fwd", n=0, nonnull=False) == OK


def test_header_constants_match_the_binding():
    text = open(os.path.join(os.path.dirname(gdn.PKG), "include", "gdn.h")).read()
    for name in ("GDN_CONV_SILU", "GDN_NORM_RMS", "GDN_NORM_GATE_FIRST"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(gdn, name)


# ---- the binding

def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


F32 = torch.float32
CU, IDX = torch.tensor([0, 3, 6]), torch.tensor([1, 0])


def conv_args(**kw):
    a = dict(x=z(6, 24), weight=z(24, 4, dtype=F32), bias=None, state_pool=z(3, 3, 24),
             cache_indices=IDX, cu_seqlens=CU, dims=(8, 8, 8))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(x=z(6, 24, dtype=torch.float16)), TypeError),
    (dict(x=z(6, 24, 1)), ValueError),
    (dict(dims=(8, 8)), ValueError),
    (dict(dims=(6, 6, 6, 6)), ValueError),
    (dict(weight=z(24, 4)), TypeError),
    (dict(weight=z(4, 24, dtype=F32).t()), ValueError),
    (dict(weight=z(25, 4, dtype=F32)), ValueError),
    (dict(bias=z(23, dtype=F32)), ValueError),
    (dict(state_pool=z(3, 2, 24)), ValueError),
    (dict(state_pool=z(3, 3, 24, dtype=F32)), TypeError),
    (dict(cache_indices=None), ValueError),
    (dict(cache_indices=torch.tensor([1, 0, 2])), ValueError),
    (dict(cu_seqlens=CU.int()), TypeError),
    (dict(x=z(24, 6).t()), ValueError),
    (dict(x=z(1, 24).expand(6, 24)), ValueError),
    (dict(outs=(z(6, 8), z(6, 8))), ValueError),
    (dict(outs=(z(6, 8), z(6, 8), z(6, 9))), ValueError),
    ({}, ValueError),  # CPU tensors
])
def test_conv_binding_refusals(kw, err):
    with pytest.raises(err):
        gdn.gdn_conv_fwd(**conv_args(**kw))


def test_conv_decode_and_backward_binding_refusals():
    a = conv_args()
    a.pop("cu_seqlens")
    for kw in (dict(state_pool=None), dict(x=z(5, 24)), {}, dict(state_pool=torch.zeros(())),
               dict(state_pool=None, cache_indices=None)):
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.gdn_conv_decode_fwd(**{**a, **kw})
    b = conv_args(douts=(z(6, 8, dtype=F32),) * 3)
    b.pop("dims")
    for kw, err in ((dict(douts=(z(6, 8, dtype=F32),) * 2), ValueError),
                    (dict(douts=(z(6, 8, dtype=F32), z(6, 8), z(6, 8))), TypeError),
                    (dict(douts=(z(5, 8, dtype=F32),) * 3), ValueError), (dict(douts=()), ValueError),
                    (dict(dstate=z(2, 2, 24, dtype=F32)), ValueError), (dict(dx=z(5, 24)), ValueError),
                    (dict(dx=z(6, 24, dtype=F32)), TypeError), ({}, ValueError)):
        with pytest.raises(err):
            gdn.gdn_conv_bwd(**{**b, **kw})


def ssm_args(**kw):
    a = dict(C=z(6, 2, 64), B=z(6, 2, 64), x=z(6, 4, 64), dt=z(6, 4, dtype=F32),
             A_log=z(4, dtype=F32), dt_bias=z(4, dtype=F32), D=None,
             state_pool=z(3, 4, 64, 64, dtype=F32), cache_indices=IDX, cu_seqlens=CU)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(x=z(6, 4, 64, dtype=torch.float16)), TypeError),
    (dict(B=z(6, 2, 64, dtype=F32)), TypeError),
    (dict(C=z(6, 1, 64)), ValueError),
    (dict(x=z(64, 4, 6).permute(2, 1, 0)), ValueError),
    (dict(dt=z(6, 4)), TypeError),
    (dict(A_log=z(5, dtype=F32)), ValueError),
    (dict(D=z(2, dtype=F32)), ValueError),
    (dict(state_pool=z(3, 4, 64, 32, dtype=F32)), ValueError),
    (dict(state_pool=z(3, 4, 64, 64)), TypeError),
    (dict(cu_seqlens=torch.tensor([0, 6])), ValueError),
    (dict(out=z(6, 4, 32)), ValueError),
    ({}, ValueError),
])
def test_ssm_binding_refusals(kw, err):
    with pytest.raises(err):
        gdn.gdn_ssm_prefill_fwd(**ssm_args(**kw))


def test_ssm_decode_binding_refusals():
    a = ssm_args()
    a.pop("cu_seqlens")
    with pytest.raises(ValueError):  # two indices for six rows
        gdn.gdn_ssm_decode_fwd(**a)


@pytest.mark.parametrize("kw,err", [
    (dict(x=z(6, 64)), ValueError),
    (dict(x=z(6, 2, 64, dtype=torch.float64)), TypeError),
    (dict(weight=z(64)), TypeError),
    (dict(weight=z(63, dtype=F32)), ValueError),
    (dict(bias=z(1, 64, dtype=F32)), ValueError),
    (dict(z=z(6, 2, 32)), ValueError),
    (dict(z=z(6, 2, 64, dtype=F32)), TypeError),
    (dict(z=z(6, 64, 2).transpose(1, 2)), ValueError),
    (dict(z=z(1, 2, 64).expand(6, 2, 64)), ValueError),
    (dict(gate_first=True), ValueError),
    (dict(out=z(6, 2, 32)), ValueError),
    ({}, ValueError),
])
def test_norm_binding_refusals(kw, err):
    with pytest.raises(err):
        gdn.gdn_norm_fwd(**{**dict(x=z(6, 2, 64), weight=z(64, dtype=F32)), **kw})
    if "out" not in kw:
        kw = {**dict(bias=None, z=None), **kw}
        with pytest.raises(err):
            gdn.gdn_norm_bwd(**{**dict(x=z(6, 2, 64), weight=z(64, dtype=F32), dout=z(6, 2, 64)), **kw})


def test_norm_backward_binding_refusals():
    a = dict(x=z(6, 2, 64), weight=z(64, dtype=F32), bias=None, z=None, dout=z(6, 2, 64))
    for kw, err in ((dict(dout=z(6, 2, 64, dtype=F32)), TypeError), (dict(dz=z(6, 2, 64)), ValueError),
                    (dict(z=z(6, 2, 64), dz=z(6, 2, 64, dtype=F32)), TypeError)):
        with pytest.raises(err):
            gdn.gdn_norm_bwd(**{**a, **kw})


def test_prefill_measurements_do_not_depend_on_the_layer_sources():
    """The stored counters of the prefill stay valid when a layer kernel changes."""
    import bench
    csrc = os.path.join(os.path.dirname(gdn.__file__), "csrc")
    own = {f for f in os.listdir(csrc)
           if f.startswith(("gdn_layer", "gdn_conv", "gdn_norm", "gdn_ssm"))}
    assert set(bench.LAYER_SOURCES) == own
