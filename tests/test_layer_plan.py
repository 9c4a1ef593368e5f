"""How the scans divide sequences, read from the sizes of their workspaces (no GPU)."""
import ctypes

import pytest

from kimi_delta_attention_08_gb300 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def up(n):
    return (n + 255) // 256 * 256


def problem(B, T, dim, state):
    q = _lib.kda_scan_problem()
    q.batch, q.T, q.dim, q.state, q.groups = B, T, dim, state, 1
    return q


# channels of a CTA, and CTAs that an SM of 228 KB and 64 K registers holds, at each state size
CTA = {8: (128, 2), 16: (64, 3), 32: (64, 1), 64: (32, 1)}


@pytest.mark.parametrize("state,dim,B,cut", [
    (64, 4864, 1, False), (64, 4096, 1, False), (64, 4096, 3, False), (64, 4864, 2, False), (64, 2432, 1, True),
    (32, 4864, 2, False), (32, 4096, 2, False), (32, 4096, 7, False), (32, 4096, 3, True), (32, 4096, 5, True),
    (16, 4096, 7, False), (16, 4096, 4, True), (16, 4096, 6, True),
    (8, 4096, 9, False), (8, 4096, 8, False), (8, 4096, 7, True), (8, 4096, 10, True)])
def test_backward_is_cut_by_what_fits_an_sm(lib, state, dim, B, cut):
    """Whole sequences where they fill the turns over 152 SMs that they take."""
    T = 2048
    n = ctypes.c_size_t(0)
    q = problem(B, T, dim, state)
    assert lib.kda_scan_bwd_get_workspace_size(ctypes.byref(q), 1, ctypes.byref(n)) == 0
    ch, fit = CTA[state]
    tiles = -(-dim // ch)
    whole = up(256 + tiles * B * T * 2 * state * 4) + B * -(-dim * (state + 2) // 4) * 16
    assert (n.value > whole) if cut else (n.value == whole)
    fill = B * tiles / (152 * fit)
    fill /= -(-B * tiles // (152 * fit))
    assert (fill < (0.85 if fit == 3 else 0.8)) == cut


@pytest.mark.parametrize("state,dim,B,cut", [
    (8, 4096, 8, True), (8, 4096, 11, True), (8, 4096, 12, False), (16, 4096, 3, True), (16, 4096, 4, False),
    (16, 4096, 8, False), (32, 4096, 1, True), (32, 4096, 2, False), (64, 2048, 1, True), (64, 3200, 1, False),
    (64, 4096, 1, False)])
def test_forward_is_cut_by_the_room_that_it_takes(lib, state, dim, B, cut):
    """Whole sequences need the status word alone; in tenths of the 4 x 152 places, they stay
    whole from 6 on with 8 states, 4 with 16 and 32, 3 with 64."""
    n = ctypes.c_size_t(0)
    assert lib.kda_scan_get_workspace_size(ctypes.byref(problem(B, 4096, dim, state)), ctypes.byref(n)) == 0
    assert (n.value > 256) == cut
