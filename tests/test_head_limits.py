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
