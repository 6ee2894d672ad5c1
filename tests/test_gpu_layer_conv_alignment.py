"""The convolution on parameters, gradients and states that start on one element, not on 16 bytes:
the same bits as from aligned copies where the element-by-element path serves both (channel counts
that no vector divides), and the oracle's values where it does not."""
import numpy as np
import pytest

from layer_util import HALF, U32, f32, i64, rounded, within
from oracle import layer as L
from test_gpu_layer_conv import call, check, make

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def shifted(t):
    """The same values, one element into a wider buffer."""
    wide = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    wide[1:] = t.flatten()
    return wide[1:].view(t.shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("w", [2, 3, 4])
@pytest.mark.parametrize("dims", [(64, 32, 32), (5, 3, 9)])
@pytest.mark.parametrize("which", ["weight", "bias", "pool"])
def test_conv_forward_of_shifted_tensors(dtype, w, dims, which):
    import gated_deltanet_prefill_gdn_amd as gdn
    c = make(60 + w, [37, 0, 1, 130, 2], dims, w, dtype, True, True)
    plain, _ = call(c, True)
    c[which] = shifted(c[which])
    assert c[which].data_ptr() % 16 != 0
    outs, pool = call(c, True)
    check(c, True, dtype, w, outs, pool, f"conv shifted {which} {dtype} W={w} {dims}")
    if dims[0] == 5:
        assert all(torch.equal(a, b) for a, b in zip(outs, plain))
    c = make(70 + w, [1] * 5, dims, w, dtype, True, True)
    c[which] = shifted(c[which])
    outs, pool = call(c, True, gdn.gdn_conv_decode_fwd)
    check(c, True, dtype, w, outs, pool, f"conv decode shifted {which} {dtype} W={w} {dims}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dout_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [(64, 32, 32), (5, 3, 9)])
@pytest.mark.parametrize("which", ["weight", "bias", "pool", "dout", "dstate"])
def test_conv_backward_of_shifted_tensors(dtype, dout_dtype, dims, which):
    import gated_deltanet_prefill_gdn_amd as gdn
    w, lengths = 4, [37, 0, 1, 130, 2]
    c = make(80, lengths, dims, w, dtype, True, True)
    r = np.random.default_rng(81)
    n, ch = c["x"].shape
    dout, dout64 = rounded(r.standard_normal((n, ch)), dout_dtype)
    c["dstate"], dstate64 = f32(r.standard_normal((len(lengths), w - 1, ch)))
    douts = [d.contiguous() for d in dout.split(dims, 1)]
    if which == "dout":
        douts = [shifted(d) for d in douts]
    else:
        c[which] = shifted(c[which])
    g = gdn.gdn_conv_bwd(c["x"], c["weight"], c["bias"], c["pool"], i64(c["idx"]), i64(c["cu"]), douts,
                         c["dstate"])
    torch.cuda.synchronize()
    ref = L.conv_bwd(c["x64"], c["weight64"], c["bias64"], c["pool64"], c["idx"], c["cu"], dout64,
                     dstate64, True)
    steps, chain = 2 * w + 13, 128 + 4 + n / 32 / 8 + 1
    what = f"conv bwd shifted {which} {dtype}/{dout_dtype} {dims}"
    h = HALF[dtype]
    within(g["dx"], ref["dx"], h * np.abs(ref["dx"]) + (1 + h) * U32 * steps * ref["dx_mag"] + 1e-38,
           what + " dx")
    for k, s in (("dweight", chain + steps), ("dbias", chain + steps), ("dstate0", steps)):
        within(g[k], ref[k], U32 * s * ref[k + "_mag"] + 1e-38, f"{what} {k}")
