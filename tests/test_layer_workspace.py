"""Workspaces of the layer operators cover what the kernels write into them, whatever path serves a
call. The rows are counted here from the launch rules, not from the library."""
import ctypes

import pytest

import gated_deltanet_prefill_gdn_amd as gdn


def conv_rows(n, ch, vec):
    """Workgroups along the tokens: 4 runs each of 128 tokens, halved while the grid is small."""
    cols, run = -(-(-(-ch // vec)) // 64), 128
    while run > 8 and -(-n // (4 * run)) * cols < 512:
        run //= 2
    return -(-n // (4 * run))


@pytest.mark.parametrize("n,ch", [(16384, 512), (16384, 6144), (700, 64), (1, 8), (100000, 40)])
@pytest.mark.parametrize("w", [2, 3, 4])
def test_conv_backward_workspace_covers_both_paths(n, ch, w):
    p = gdn.GdnConvProblem(n, 1, 1, ch, ch, (ctypes.c_int32 * 3)(ch, 0, 0), w, gdn.GDN_DTYPE_BF16,
                           gdn.GDN_DTYPE_F32, gdn.GDN_CONV_SILU, 0)
    rows = [conv_rows(n, ch, vec) for vec in (1, 4)]
    assert rows[1] >= rows[0]
    need = gdn.gdn_conv_bwd_workspace_size(p)
    assert max(rows) * (w + 1) * ch * 4 <= need < max(rows) * (w + 1) * ch * 4 + 256
    assert (n, ch) != (16384, 512) or rows == [64, 256]
