"""The layer operators where element offsets pass 32 bits: rows far apart, slots far into a pool,
calls of billions of entries. The same values in compact tensors give the same bits, since neither
strides nor slots change the arithmetic; a long scan is checked at its far end against the fp64
recurrence."""
import numpy as np
import pytest

from layer_util import DEV, i64, np64, within
from oracle import layer as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
FAR = 1 << 26  # elements between rows


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def rn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


def far_rows(t):
    """t's values as rows FAR elements apart (t has 70 rows: the last is past 2^32)."""
    wide = torch.empty(t.shape[0] * FAR, dtype=t.dtype, device=DEV)
    view = wide.as_strided(t.shape, (FAR,) + t[0].stride())
    view.copy_(t)
    return view


@pytest.mark.parametrize("ch", [64, 33])  # in vectors; element by element
def test_conv_rows_far_apart(ch):
    import gated_deltanet_prefill_gdn_amd as gdn
    x, w, b = rn(1, 70, ch, dtype=torch.bfloat16), rn(2, ch, 4), rn(3, ch)
    cu, dout = i64([0, 30, 70]), rn(4, 70, ch)
    wide, dx = far_rows(x), far_rows(torch.zeros_like(x))
    want, = gdn.gdn_conv_fwd(x, w, b, None, None, cu)
    got, = gdn.gdn_conv_fwd(wide, w, b, None, None, cu)
    assert torch.equal(got, want)
    want = gdn.gdn_conv_bwd(x, w, b, None, None, cu, (dout,))
    got = gdn.gdn_conv_bwd(wide, w, b, None, None, cu, (dout,), dx=dx)
    for k in want:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("dim", [64, 33])
def test_norm_rows_far_apart(dim):
    import gated_deltanet_prefill_gdn_amd as gdn
    x, z = rn(1, 70, 2, dim, dtype=torch.bfloat16), rn(2, 70, 2, dim, dtype=torch.bfloat16)
    w, dout = rn(3, dim), rn(4, 70, 2, dim, dtype=torch.bfloat16)
    wx, wz, dz = far_rows(x), far_rows(z), far_rows(torch.zeros_like(z))
    assert torch.equal(gdn.gdn_norm_fwd(wx, w, None, wz), gdn.gdn_norm_fwd(x, w, None, z))
    want = gdn.gdn_norm_bwd(x, w, None, z, dout)
    got = gdn.gdn_norm_bwd(wx, w, None, wz, dout, dz=dz)
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_slots_far_into_the_pools():
    import gated_deltanet_prefill_gdn_amd as gdn
    n, h, hv, dk, dv = 90, 1, 64, 128, 64
    slots = (1 << 32) // (hv * dv * dk) + 2
    cu, near, far = i64([0, 80, 90]), i64([1, 0]), i64([slots - 1, slots - 2])
    start = 0.3 * rn(1, 2, hv, dv, dk)
    big = torch.empty(slots, hv, dv, dk, device=DEV)
    small = start.clone()
    big[slots - 2:] = start
    bf = torch.bfloat16
    a = (rn(2, n, h, dk, dtype=bf), rn(3, n, h, dk, dtype=bf), rn(4, n, hv, dv, dtype=bf),
         rn(5, n, hv), rn(6, hv), rn(7, hv) - 3, None)
    want = gdn.gdn_ssm_prefill_fwd(*a, small, near, cu)
    got = gdn.gdn_ssm_prefill_fwd(*a, big, far, cu)
    assert torch.equal(got, want) and torch.equal(big[slots - 2:], small)
    a = tuple(t[:2].contiguous() if t is not None and t.dim() > 1 else t for t in a)
    want = gdn.gdn_ssm_decode_fwd(*a, small, near)
    got = gdn.gdn_ssm_decode_fwd(*a, big, far)
    assert torch.equal(got, want) and torch.equal(big[slots - 2:], small)
    del big

    ch = 8192
    slots = (1 << 32) // (3 * ch) + 3
    x, w, start = rn(8, n, ch, dtype=bf), rn(9, ch, 4), rn(10, 2, 3, ch, dtype=bf)
    far, big, small = i64([slots - 1, slots - 2]), torch.empty(slots, 3, ch, dtype=bf, device=DEV), start.clone()
    big[slots - 2:] = start
    bwd = [gdn.gdn_conv_bwd(x, w, None, p, i, cu, (x,)) for p, i in ((small, near), (big, far))]
    for k in bwd[0]:
        assert torch.equal(bwd[0][k], bwd[1][k]), k
    for call in (lambda p, i: gdn.gdn_conv_fwd(x, w, None, p, i, cu),
                 lambda p, i: gdn.gdn_conv_decode_fwd(x[:2], w, None, p, i)):
        assert torch.equal(call(big, far)[0], call(small, near)[0])
        assert torch.equal(big[slots - 2:], small)


@pytest.mark.parametrize("lengths", [[139000, 60], [4] * 35000])  # chunks; token by token
def test_scan_of_billions_of_entries(lengths):
    """The last request of a call whose rows end past 2^31 entries. Outputs: half a step of bf16,
    and 1.5 x 2^-8 of the magnitude for the bf16 scores and states inside."""
    import gated_deltanet_prefill_gdn_amd as gdn
    n, hv, dk, dv, heads = sum(lengths), 64, 64, 256, [0, 63]
    assert n * hv * dv > 1 << 31
    bf, b = torch.bfloat16, len(lengths)
    C, B, x = 0.6 * rn(1, n, 1, dk), 0.6 * rn(2, n, 1, dk), torch.empty(n, hv, dv, dtype=bf, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(3))
    C, B, dt, A, bias, D = C.to(bf), B.to(bf), rn(4, n, hv), rn(5, hv), rn(6, hv) - 3, rn(7, hv)
    # every request but the last shares nothing with it: one slot each, or padding requests
    pool = 0.3 * rn(8, 2, hv, dv, dk)
    idx = np.full(b, -1)
    idx[0], idx[-1] = 0, 1
    start = np64(pool[1:, heads])
    cu = np.concatenate([[0], np.cumsum(lengths)])
    out = gdn.gdn_ssm_prefill_fwd(C, B, x, dt, A, bias, D, pool, i64(idx), i64(cu))
    t = slice(n - lengths[-1], n)
    ref, new, mag, mags, _ = L.ssm(np64(C[t]), np64(B[t]), np64(x[t][:, heads]), np64(dt[t][:, heads]),
                                   np64(A[heads]), np64(bias[heads]), np64(D[heads]), start, [0],
                                   [0, lengths[-1]])
    within(out[t][:, heads], ref, 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * 1.5 * 2.0 ** -8 * mag + 1e-38,
           "last request")
    within(pool[1:, heads], new, 2.0 ** -16 * mags + 1e-38, "last request's state")
