"""Shared by the GPU tests of the layer operators: tensors from numpy, and element-wise bounds in
units of rounding steps."""
import numpy as np
import torch

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # a rounding's largest relative error
U32 = 2.0 ** -24


def rounded(a, dtype):
    """(device tensor of this dtype, its exact values in fp64)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DT[dtype]).to(DEV)
    return t, t.double().cpu().numpy()


def f32(a):
    return rounded(a, "f32")


def i64(a):
    return torch.tensor(list(a), dtype=torch.int64, device=DEV)


def strided(t, pad, offset=0):
    """The same values as rows of a wider tensor, `offset` elements into it."""
    n, inner = t.shape[0], t[0].numel() if t.shape[0] else int(np.prod(t.shape[1:]))
    wide = torch.full((n, inner + pad + offset), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[:, offset:offset + inner].unflatten(1, t.shape[1:])
    view.copy_(t)
    return view


def np64(t):
    return t.double().cpu().numpy()


def within(got, ref, allow, what):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not ref.size:
        return
    assert np.isfinite(got).all(), f"{what}: not finite"
    d = np.abs(got - ref)
    worst = float((d / np.maximum(allow, 1e-300)).max())
    print(f"[layer] {what}: worst error / allowance {worst:.3f}, max error {d.max():.2e}", flush=True)
    assert worst <= 1.0, f"{what}: {worst:.2f} times its allowance"
