"""Workspaces of the layer operators cover what the kernels write into them, whatever path serves a
call. The rows are counted here from the launch rules, not from the library."""
import ctypes
import random

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


def cut_of(n, b, h, hv, dv):
    """(tokens of a piece at most, parts of a piece) of a scan, 0 where no request is cut."""
    blocks = -(-(hv // h * dv) // 128) * h
    best = None
    for k in range(1, 5):
        pieces2 = 2 * k * 512 // blocks - b
        if pieces2 > 0:
            l = -(--(-2 * n // pieces2) // 64) * 64
            best = min(best or (1 << 60, 0), (k * (l + 1000), l))
    if best is None or n <= max(best[1], 512):
        return 0, 1
    l = max(best[1], 512)
    return l, 1 if l < 2048 else 2 if l < 4096 else 4


def pieces_of(length, lseg):
    if length <= lseg:
        return 1
    n = -(-length // lseg)
    piece = -(--(-length // n) // 64) * 64
    return -(-length // piece)


SCANS = [(131072, 1, 16, 32, 128, 128), (33860, 8, 8, 64, 128, 64), (16384, 4, 16, 16, 128, 128),
         (16039, 2, 1, 256, 256, 64), (2020, 3, 1, 2, 256, 256), (333, 3, 1, 8, 64, 64)]


@pytest.mark.parametrize("n,b,h,hv,dk,dv", SCANS)
def test_scan_workspace_holds_the_states_of_cut_requests_and_no_more(n, b, h, hv, dk, dv):
    """A cut request of L tokens has at most L / lseg + 1 pieces, and there are at most min(B, N /
    lseg) of them."""
    lseg, parts = cut_of(n, b, h, hv, dv)
    places = 0 if lseg == 0 else (n // lseg + min(b, n // lseg)) * parts
    floats = [places * hv * dv * dk, places * hv]
    need = gdn.gdn_ssm_workspace_size(gdn.make_problem(n, b, h, hv, dk, dv, b, gdn.GDN_DTYPE_BF16))
    assert 0 <= need - 4 * sum(floats) < 3 * 256, (need, lseg, parts)


@pytest.mark.parametrize("seed", range(20))
def test_pieces_of_any_lengths_fit_the_places(seed):
    r = random.Random(seed)
    for _ in range(300):
        lseg = 64 * r.randrange(8, 140)
        b = r.randrange(1, 9)
        lengths = [r.choice([r.randrange(0, 4 * lseg), lseg + r.randrange(0, 70), lseg * r.randrange(1, 6)])
                   for _ in range(b)]
        places = sum(p for p in (pieces_of(x, lseg) for x in lengths) if p > 1)
        n = sum(lengths)
        assert places <= n // lseg + min(b, n // lseg), (lseg, lengths)
