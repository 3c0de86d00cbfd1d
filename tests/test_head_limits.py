"""Sizes of the head's losses and gradients at the ends of their range, asked
of the workspace queries: nothing is launched. Column numbers, padded to whole
tiles, have to fit 32 bits, and the tiles of 256 rows x 128 columns that a
launch goes through 2^30.
"""
import ctypes as C

import pytest

import token_perturbation_estimator_gb300 as dust

MOST = (1 << 31) - (1 << 16)  # rows, columns or ids


@pytest.fixture(scope="module")
def L():
    from token_perturbation_estimator_gb300 import build
    build.build()
    return dust.lib()


def _queries(L, dtype):
    n = C.c_size_t(0)
    return {
        "loss": lambda S, T, d, V: L.dust_head_loss_workspace(C.byref(n), S, T, d, V, dtype),
        "grad": lambda S, T, d, V: L.dust_head_loss_grad_workspace(C.byref(n), S, T, d, V, dtype),
        "distill": lambda S, T, d, V: L.dust_distill_loss_workspace(
            C.byref(n), S, T, d, V, 3, dtype),
        "distill_grad": lambda S, T, d, V: L.dust_distill_loss_grad_workspace(
            C.byref(n), S, T, d, V, 3, dtype),
    }, n


@pytest.mark.parametrize("dtype", [dust.BF16, dust.F32])
@pytest.mark.parametrize("name", ["loss", "grad", "distill", "distill_grad"])
def test_what_32_bits_hold(L, name, dtype):
    queries, n = _queries(L, dtype)
    ask = queries[name]
    for S, T, d, V in ((1, 4, 8, MOST), (1, MOST, 8, 4), (MOST // 4, 4, 8, 4), (1, 4, MOST, 4)):
        assert ask(S, T, d, V) == dust.OK and n.value > 0
    for S, T, d, V in ((1, 4, 8, MOST + 1), (1, MOST + 1, 8, 4), (1, 4, 8, (1 << 31) - 1),
                       (MOST // 4 + 1, 4, 8, 4), (1, 4, MOST + 1, 4)):
        assert ask(S, T, d, V) == dust.ERR_RANGE, (S, T, d, V)


@pytest.mark.parametrize("name", ["loss", "grad", "distill", "distill_grad"])
def test_more_tiles_than_a_launch_counts(L, name):
    queries, n = _queries(L, dust.BF16)
    rows, ids = 1 << 23, 1 << 22  # 2^15 x 2^15 tiles
    assert queries[name](1, rows, 8, ids) == dust.OK
    assert queries[name](1, rows + 1, 8, ids) == dust.ERR_RANGE
    assert queries[name](1, rows, 8, ids + 1) == dust.ERR_RANGE
    assert queries[name](3, 1 << 30, 8, 1) == dust.ERR_RANGE


def _bounds(R, d, V, planes):
    """What the header says a workspace has room for: G of a piece, copies of
    H and E, gH's running sums, those of up to 304 slices of either gradient,
    and 64 bytes a row."""
    up = (R + 255) // 256 * 256
    copies = 2 * planes * (R + V) * ((d + 7) // 8 * 8)
    G = 2 * max(1 << 28, 1024 * up * planes)
    sums = 4 * up * 256 * ((d + 127) // 128)  # a tile has room for 256 columns
    slices = 2 * 304 * 4 * 256 * 256
    return copies, G, copies + G + sums + slices + 64 * R + (1 << 20)


@pytest.mark.parametrize("dtype,planes", [(dust.BF16, 1), (dust.F32, 3)])
@pytest.mark.parametrize("R,d,V", [(8192, 2048, 50257), (16384, 512, 32768), (1 << 18, 64, 32768),
                                   (1 << 20, 512, 32768), ((1 << 20) + 1, 512, 32768),
                                   (1 << 24, 64, 50257)])
def test_workspaces_of_many_rows(L, R, d, V, dtype, planes):
    n = C.c_size_t(0)
    copies, G, most = _bounds(R, d, V, planes)
    assert L.dust_head_loss_grad_workspace(C.byref(n), 1, R, d, V, dtype) == dust.OK
    assert copies < n.value <= most
    if R >= 1 << 18:  # four tiles of ids for every row, and half of the most at least
        assert n.value >= copies + G // 2
    assert L.dust_head_loss_workspace(C.byref(n), 1, R, d, V, dtype) == dust.OK
    parts = 16 * ((V + 127) // 128) * ((R + 31) // 32 * 32)
    assert copies < n.value <= copies + parts + 16 * R + (1 << 20)


def test_workspaces_that_the_header_names(L):
    n = C.c_size_t(0)
    for fn, dtype, R, d, V, mb in (
            (L.dust_head_loss_workspace, dust.BF16, 8192, 2048, 50257, 291.0),
            (L.dust_head_loss_grad_workspace, dust.BF16, 8192, 2048, 50257, 843.6),
            (L.dust_head_loss_workspace, dust.F32, 8192, 2048, 50257, 769.8),
            (L.dust_head_loss_grad_workspace, dust.F32, 8192, 2048, 50257, 1343.4),
            (L.dust_head_loss_grad_workspace, dust.BF16, 1 << 20, 512, 32768, 5440.0),
            (L.dust_head_loss_workspace, dust.BF16, 1, 2048, 50257, 0.1),
            (L.dust_head_loss_grad_workspace, dust.BF16, 1, 2048, 50257, 2.5)):
        assert fn(C.byref(n), 1, R, d, V, dtype) == dust.OK
        assert abs(n.value / 1e6 - mb) <= 0.06, (R, d, V, n.value)
