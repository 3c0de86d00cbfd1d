"""GPU parity of the gated feed-forward block and its gradients against the
formulas in 64 bits (numpy, on the CPU).

Tolerances, normwise relative. A sum of n fp32 products of mixed signs is off by
about 2^-24 sqrt(n / 2) of its norm when added one after another; 2^-24 (16 + 2
sqrt(n)) covers it, the roundings around it and the activation's. bf16
outputs: one rounding, at most 2^-8 elementwise, 2.5e-3 normwise; the
gradients' dG and dU are rounded to bf16 before their products, whose errors
add as independent ones do: 2 x 2.5e-3 covers both roundings."""
import numpy as np
import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda, rel_fro

pytestmark = pytest.mark.gpu

BF16_TOL = 2.5e-3
ACTS = {"silu": dust.SILU, "gelu": dust.GELU, "relu2": dust.RELU2}


def f32_tol(n):
    return 2.0 ** -24 * (16 + 2 * np.sqrt(n))


def _np(t):
    return t.double().cpu().numpy()


def _inputs(T, d, f, dtype, dev, extra=0, seed=0):
    import torch
    g = torch.Generator().manual_seed(7 * T + 3 * d + f + seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def rows(n, c, scale):
        full = (torch.randn((n, c + extra), generator=g) * scale).to(dt).to(dev)
        return full[:, :c]

    return (rows(T, d, 1.0), rows(f, d, 1.5 / np.sqrt(d)), rows(f, d, 1.0 / np.sqrt(d)),
            rows(T, f, 0.5))


def act64(g, act):
    """act(g) and its slope."""
    if act == "relu2":
        r = np.maximum(g, 0.0)
        return r * r, 2.0 * r
    c, b = 2.0 * np.sqrt(2.0 / np.pi), 0.044715
    z, dz = (g, 1.0) if act == "silu" else (c * (g + b * g ** 3), c * (1 + 3 * b * g * g))
    with np.errstate(over="ignore"):
        p = 1.0 / (1.0 + np.exp(-z))
    return g * p, p + g * p * (1.0 - p) * dz


def reference(gh, X, Wg, Wu, act):
    X, Wg, Wu, gh = _np(X), _np(Wg), _np(Wu), _np(gh)
    g, u = X @ Wg.T, X @ Wu.T
    a, slope = act64(g, act)
    dG, dU = gh * u * slope, gh * a
    return a * u, dG @ Wg + dU @ Wu, dG.T @ X, dU.T @ X


SIZES = [(1, 1, 1), (1, 512, 2048), (2, 64, 128), (3, 33, 65), (5, 96, 200), (17, 8, 24),
         (64, 130, 257), (129, 64, 64), (255, 72, 300), (256, 128, 256), (257, 129, 127),
         (600, 301, 515), (40, 1100, 700), (33, 2048, 100), (1500, 40, 48), (8, 4000, 16),
         (4, 2048, 4096), (9, 512, 1111), (16, 1000, 504), (32, 257, 4099), (512, 512, 512)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f", SIZES)
def test_forward_and_gradients(T, d, f, dtype):
    dev = cuda()
    act = ["silu", "gelu", "relu2"][(T + d + f) % 3]
    X, Wg, Wu, gh = _inputs(T, d, f, dtype, dev)
    h64, gX64, gWg64, gWu64 = reference(gh, X, Wg, Wu, act)
    h = dust.dust_gated_up(X, Wg, Wu, ACTS[act])
    assert h.dtype == X.dtype and tuple(h.shape) == (T, f)
    tol = f32_tol(d) * (2 if act == "relu2" else 1)
    # Single values: each product's bound is d 2^-24 of its magnitudes.
    aX, aG, aU = (np.abs(_np(t)) for t in (X, Wg, Wu))
    eg, eu = (d + 4) * 2.0 ** -23 * (aX @ aG.T), (d + 4) * 2.0 ** -23 * (aX @ aU.T)
    g, u = _np(X) @ _np(Wg).T, _np(X) @ _np(Wu).T
    a, _ = act64(g, act)
    slope = 1.2 if act != "relu2" else 2.0 * (np.abs(g) + eg)
    e = slope * eg * (np.abs(u) + eu) + np.abs(a) * eu + 16 * 2.0 ** -24 * np.abs(h64) + 1e-37
    off = np.abs(_np(h) - h64)
    assert (off <= e + (2.0 ** -8 * (np.abs(h64) + e) if dtype == "bf16" else 0)).all()
    assert rel_fro(_np(h), h64) <= (BF16_TOL if dtype == "bf16" else 0) + 2 * tol
    out_type = X.dtype
    gX, gWg, gWu = dust.dust_gated_up_grad(gh, X, Wg, Wu, ACTS[act], gW_dtype=out_type)
    assert gX.dtype == X.dtype and gWg.dtype == out_type and tuple(gWu.shape) == (f, d)
    rounding = 2 * BF16_TOL if dtype == "bf16" else 0
    assert rel_fro(_np(gX), gX64) <= rounding + 4 * tol + f32_tol(2 * f)
    assert rel_fro(_np(gWg), gWg64) <= rounding + 4 * tol + f32_tol(T)
    assert rel_fro(_np(gWu), gWu64) <= rounding + 4 * tol + f32_tol(T)
    for x, y in zip((h, gX, gWg, gWu), (dust.dust_gated_up(X, Wg, Wu, ACTS[act]),
                                        *dust.dust_gated_up_grad(gh, X, Wg, Wu, ACTS[act],
                                                                 gW_dtype=out_type))):
        assert (x == y).all()
    assert dust.dust_last_error() == dust.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f,extra", [(50, 64, 96, 8), (50, 64, 96, 3), (3, 100, 260, 4),
                                         (300, 130, 70, 1)])
def test_strided_rows(T, d, f, extra, dtype):
    import torch
    dev = cuda()
    X, Wg, Wu, gh = _inputs(T, d, f, dtype, dev, extra=extra)
    assert not X.is_contiguous()
    h64, gX64, gWg64, gWu64 = reference(gh, X, Wg, Wu, "silu")
    out = torch.full((T, f + extra), 7.0, dtype=X.dtype, device=dev)
    h = dust.dust_gated_up(X, Wg, Wu, h=out[:, :f])
    tol = (2 * BF16_TOL if dtype == "bf16" else 0) + 5 * f32_tol(max(d, 2 * f, T))
    assert rel_fro(_np(h), h64) <= tol and (out[:, f:] == 7.0).all()
    gout = torch.full((T, d + extra), 7.0, dtype=X.dtype, device=dev)
    gX, gWg, gWu = dust.dust_gated_up_grad(gh, X, Wg, Wu, gX=gout[:, :d])
    assert gWg.dtype == torch.float32 and (gout[:, d:] == 7.0).all()
    for got, want in ((gX, gX64), (gWg, gWg64), (gWu, gWu64)):
        assert rel_fro(_np(got), want) <= tol


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_halves_of_one_matrix_and_unaligned_rows(dtype):
    import torch
    dev = cuda()
    T, d, f = 70, 72, 90
    X, Wg, Wu, gh = _inputs(T, d, f, dtype, dev)
    W = torch.cat([Wg, Wu])
    want = dust.dust_gated_up(X, Wg, Wu)
    assert (dust.dust_gated_up(X, W[:f], W[f:]) == want).all()
    flat = torch.empty(T * d + 1, dtype=X.dtype, device=dev)
    off = flat[1:].view(T, d)
    off.copy_(X)
    assert rel_fro(_np(dust.dust_gated_up(off, Wg, Wu)), _np(want)) <= 2 * BF16_TOL


@pytest.mark.parametrize("T", [3, 200])
def test_accumulates(T):
    import torch
    dev = cuda()
    d, f = 48, 130
    for dtype in ("bf16", "f32"):
        X, Wg, Wu, gh = _inputs(T, d, f, dtype, dev)
        _, gWg, gWu = dust.dust_gated_up_grad(gh, X, Wg, Wu)
        a, b = torch.full_like(gWg, 2.0), torch.full_like(gWu, -3.0)
        dust.dust_gated_up_grad(gh, X, Wg, Wu, flags=dust.ACCUMULATE, gWg=a, gWu=b)
        assert torch.allclose(a, gWg + 2.0, rtol=1e-6, atol=1e-5)
        assert torch.allclose(b, gWu - 3.0, rtol=1e-6, atol=1e-5)


def test_no_rows():
    import torch
    dev = cuda()
    X, Wg, Wu, gh = _inputs(0, 16, 24, "bf16", dev)
    assert tuple(dust.dust_gated_up(X, Wg, Wu).shape) == (0, 24)
    gX, gWg, gWu = dust.dust_gated_up_grad(gh, X, Wg, Wu)
    assert (gWg == 0).all() and (gWu == 0).all()
    a = torch.ones_like(gWg)
    dust.dust_gated_up_grad(gh, X, Wg, Wu, flags=dust.ACCUMULATE, gWg=a, gWu=a.clone())
    assert (a == 1).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "relu2"])
@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_values(act, T, dtype):
    """Gates far out on both sides: the activation is 0 or the gate itself
    there, its slope 0 or 1 (2 g), and nothing is NaN."""
    import torch
    dev = cuda()
    d, f = 16, 64
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    X = torch.zeros((T, d), dtype=dt, device=dev)
    X[:, 0] = 1.0
    X[:, 1] = 0.5
    gates = [0.0, 1.0, -1.0, 30.0, -30.0, 100.0, -100.0, 1e4, -1e4, 1e8, -1e8, 1e15, -1e15]
    Wg = torch.zeros((f, d), dtype=dt, device=dev)
    for i, v in enumerate(gates):
        Wg[i, 0] = v
    Wu = torch.zeros_like(Wg)
    Wu[:, 1] = 2.0
    gh = torch.ones((T, f), dtype=dt, device=dev)
    h64, gX64, gWg64, gWu64 = reference(gh, X, Wg, Wu, act)
    h = _np(dust.dust_gated_up(X, Wg, Wu, ACTS[act]))
    tol = 2.0 ** -8 if dtype == "bf16" else 1e-5
    # below the smallest normal number both may be 0
    assert (np.abs(h - h64) <= tol * np.abs(h64) + 1e-37).all()
    gX, gWg, gWu = dust.dust_gated_up_grad(gh, X, Wg, Wu, ACTS[act])
    for got, want in ((gWg, gWg64), (gWu, gWu64)):
        assert (np.abs(_np(got) - want) <= 2 * tol * np.abs(want) + T * 1e-12).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_gates_as_far_as_their_type_goes(act, T, dtype):
    """Gates up to 1e37 on both sides, whose slope is exactly 0 or 1: every gradient
    is finite and right. A slope, or an activation relative to its gate, is a
    handful of fp32 roundings of terms of at most 2, where the exponentials'
    argument is at most 2 and else saturates: 32 * 2^-24 = 2^-19 covers them. bf16
    rounds dG and dU (2^-8), and gX once more; n products' sum cuts off at most
    n 2^-23 of their magnitudes."""
    import torch
    dev = cuda()
    d, f = 16, 64
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    X = torch.zeros((T, d), dtype=dt, device=dev)
    X[:, 0] = 1.0
    X[:, 1] = 0.5
    Wg = torch.zeros((f, d), dtype=dt, device=dev)
    for i, v in enumerate([1.0, 1e3, 1e15, 1e30, 2e31, 1e32, 1e35, 1e37]):
        Wg[2 * i, 0], Wg[2 * i + 1, 0] = v, -v
    Wu = torch.zeros_like(Wg)
    Wu[:, 1] = 2.0
    gh = torch.full((T, f), 2.0 ** -9, dtype=dt, device=dev)
    h64, gX64, gWg64, gWu64 = reference(gh, X, Wg, Wu, act)
    gate = _np(X) @ _np(Wg).T
    a, slope = act64(gate, act)
    rounding = 2.0 ** -8 if dtype == "bf16" else 0.0
    off = np.abs(_np(dust.dust_gated_up(X, Wg, Wu, ACTS[act])) - h64)
    assert (off <= (rounding + 2.0 ** -19) * np.abs(h64) + 1e-37).all()
    dG, dU = _np(gh) * slope, _np(gh) * a  # u is 1
    eG = 2.0 ** -19 * _np(gh) + rounding * np.abs(dG) + 1e-37
    eU = (2.0 ** -19 + rounding) * np.abs(dU) + 1e-37
    gX, gWg, gWu = (_np(t) for t in dust.dust_gated_up_grad(gh, X, Wg, Wu, ACTS[act]))
    aX, aG, aU = (np.abs(_np(t)) for t in (X, Wg, Wu))
    cut = 2 * f * 2.0 ** -23
    e = (eG + cut * np.abs(dG)) @ aG + (eU + cut * np.abs(dU)) @ aU
    assert (np.abs(gX - gX64) <= e + rounding * (np.abs(gX64) + e)).all()
    cut = T * 2.0 ** -23
    assert (np.abs(gWg - gWg64) <= (eG + cut * np.abs(dG)).T @ aX).all()
    assert (np.abs(gWu - gWu64) <= (eU + cut * np.abs(dU)).T @ aX).all()


def test_fp32_gradients_beyond_bf16s_range():
    """dG and dU of both signs between bf16's largest number and fp32's, which are
    operands of their own products: those are finite, and right to fp32's
    accuracy. Each row has one unit, so that every value is one term: a handful of
    roundings in dG and dU, and what three planes leave, 2^-24.
    An operand's first plane is its value rounded to bf16, up to (1 + 2^-8) times as
    large, and the product of two such up to (1 + 2^-8)^2 times: from 2^128 by that
    on a value may be infinite (1.7e38, 2^127 as bf16, times 2), of its sign."""
    import torch
    dev = cuda()
    T, d, f = 8, 2, 8
    X, Wg, Wu, gh = (torch.zeros(n, device=dev) for n in ((T, d), (f, d), (f, d), (T, f)))
    X[:, 0], X[:, 1] = 0.5, 1.0
    Wg[:, 1] = 1.0  # the gate is 1: squared ReLU has 1 there and a slope of 2
    for i, v in enumerate((3.4e38, -3.4e38, 3.398e38, -3.392e38)):
        gh[2 * i, 2 * i], gh[2 * i + 1, 2 * i + 1] = v, v / 2  # dU
        Wu[2 * i, 0], Wu[2 * i + 1, 0] = 2.0 ** -4, 2.0        # dG: v / 16, v
    want = reference(gh, X, Wg, Wu, "relu2")[1:]
    assert all(3.39e38 < np.abs(w).max() < 3.4028e38 for w in want)
    for a, b in zip(dust.dust_gated_up_grad(gh, X, Wg, Wu, dust.RELU2), want):
        a = _np(a)
        past = np.isinf(a) & (np.abs(b) >= 2.0 ** 128 / (1 + 2.0 ** -8) ** 2) & (np.sign(a) == np.sign(b))
        assert past.sum() < b.size / 2
        assert (np.abs(a - b)[~past] <= 8 * 2.0 ** -24 * np.abs(b)[~past]).all()


@pytest.mark.parametrize("T", [1, 300])
def test_infinities_and_nan_stay_in_their_rows(T):
    import torch
    dev = cuda()
    d, f = 64, 128
    X, Wg, Wu, gh = _inputs(T + 2, d, f, "bf16", dev)
    want = dust.dust_gated_up(X, Wg, Wu)
    bad = X.clone()
    bad[T, 3] = float("nan")
    bad[T + 1, 5] = float("inf")
    h = dust.dust_gated_up(bad, Wg, Wu)
    assert (h[:T] == want[:T]).all()
    assert h[T].isnan().all() and not h[T + 1].isfinite().all()


def test_copies_of_rows_off_16_bytes_keep_every_bit():
    """Rows that are copied before their products give what rows that start on 16
    bytes do: the same products of the same values, in one order."""
    import torch
    dev = cuda()
    for dtype in ("bf16", "f32"):
        for T, d, f in ((70, 72, 90), (300, 200, 136)):
            ops = _inputs(T, d, f, dtype, dev)
            want = dust.dust_gated_up(*ops[:3]), *dust.dust_gated_up_grad(ops[3], *ops[:3])
            for which in (0, 1, 2, 3):
                moved = list(ops)
                flat = torch.empty(ops[which].numel() + 1, dtype=ops[0].dtype, device=dev)
                moved[which] = flat[1:].view(ops[which].shape)
                moved[which].copy_(ops[which])
                got = (dust.dust_gated_up(*moved[:3]), *dust.dust_gated_up_grad(moved[3], *moved[:3]))
                for a, b in zip(got, want):
                    assert torch.equal(a, b), (dtype, T, which)


def test_no_plane_of_fp32_rows_off_16_bytes_is_lost():
    """The same in fp32 against 64 bits, to fp32's accuracy (the planes behind the first
    are worth 2e-3 together)."""
    import torch
    dev = cuda()
    T, d, f = 70, 72, 90
    X, Wg, Wu, gh = (
        torch.cat([t.flatten(), t.new_zeros(3)]).roll(1)[1:-2].view(t.shape)
        for t in _inputs(T, d, f, "f32", dev))
    assert all(t.data_ptr() % 16 for t in (X, Wg, Wu, gh))
    got = dust.dust_gated_up(X, Wg, Wu), *dust.dust_gated_up_grad(gh, X, Wg, Wu)
    for a, b in zip(got, reference(gh, X, Wg, Wu, "silu")):
        assert rel_fro(_np(a), b) <= 5 * f32_tol(max(d, 2 * f, T))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 300])
def test_infinities_and_nan_reach_their_rows_gradient_alone(T, dtype):
    """A NaN and an infinity in rows of X, and in rows of gh: h and gX of all other
    rows keep their bits, these rows' are no numbers, nor are gWg and gWu, which
    all rows enter."""
    import torch
    dev = cuda()
    d, f = 64, 128
    X, Wg, Wu, gh = _inputs(T + 4, d, f, dtype, dev)
    want = dust.dust_gated_up(X, Wg, Wu)
    gX0 = dust.dust_gated_up_grad(gh, X, Wg, Wu)[0]
    bad_X, bad_gh = X.clone(), gh.clone()
    bad_X[T, 3], bad_X[T + 1, 5] = float("nan"), float("inf")
    bad_gh[T + 2, 7], bad_gh[T + 3, 9] = float("nan"), -float("inf")
    h = dust.dust_gated_up(bad_X, Wg, Wu)
    assert torch.equal(h[:T], want[:T]) and torch.equal(h[T + 2:], want[T + 2:])
    assert h[T].isnan().all() and not h[T + 1].isfinite().any()
    gX, gWg, gWu = dust.dust_gated_up_grad(bad_gh, bad_X, Wg, Wu)
    assert torch.equal(gX[:T], gX0[:T])
    assert gX[T].isnan().all() and gX[T + 2].isnan().all()
    assert not gX[T + 1].isfinite().any() and not gX[T + 3].isfinite().any()
    assert not gWg.isfinite().any() and not gWu.isfinite().any()


@pytest.mark.parametrize("act", ["silu", "gelu", "relu2"])
@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_gradient_of_far_values(act, T, dtype):
    """gX where gates are far out, each row with a unit of its own, so that no large
    term hides a small one: dG and dU are a handful of fp32 roundings (2^-19), the
    exponential's argument (100 at most until it saturates: 2^-24 * 100 < 2^-17) and
    bf16's, the product two terms, and gX is rounded once. (A slope that is far below
    the two terms it is made of is held to 1e-3 instead.)"""
    import torch
    dev = cuda()
    d, f = 16, 64
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    X = torch.zeros((T, d), dtype=dt, device=dev)
    X[:, 0], X[:, 1] = 1.0, 0.5
    Wg = torch.zeros((f, d), dtype=dt, device=dev)
    Wu = torch.zeros_like(Wg)
    Wu[:, 1] = 2.0
    gates = [0.0, 1.0, -1.0, 3.0, -3.0, 100.0, -100.0, 1e4, -1e4, 1e8, -1e8, 1e15, -1e15]
    for i, v in enumerate(gates):
        Wg[i, 0] = v
        Wg[i, 2] = 1.0
    gh = torch.zeros((T, f), dtype=dt, device=dev)
    gh[torch.arange(T), torch.arange(T) % len(gates)] = 1.0
    want = reference(gh, X, Wg, Wu, act)[1]
    gX = _np(dust.dust_gated_up_grad(gh, X, Wg, Wu, ACTS[act])[0])
    gate = _np(X) @ _np(Wg).T
    a, slope = act64(gate, act)
    size = (_np(gh) * np.maximum(np.abs(slope), 1e-3)) @ np.abs(_np(Wg)) + \
        (_np(gh) * np.abs(a)) @ np.abs(_np(Wu))
    e = (2.0 ** -19 + 2.0 ** -17) * size
    if dtype == "bf16":
        e = e + 2.0 ** -8 * size + 2.0 ** -8 * (np.abs(want) + e)
    assert np.isfinite(gX).all() and (np.abs(gX - want) <= e + 1e-37).all()


def test_gradients_against_differences():
    """Central differences of <gh, h> along random directions, fp32: at step
    e, their error is e^2 of the third derivative (1e-4 here) and the values'
    rounding 2^-24 |h| / e."""
    import torch
    dev = cuda()
    T, d, f = 37, 40, 56
    for act in ACTS:
        X, Wg, Wu, gh = _inputs(T, d, f, "f32", dev)
        gX, gWg, gWu = dust.dust_gated_up_grad(gh, X, Wg, Wu, ACTS[act])
        g = torch.Generator().manual_seed(5)
        dirs = [torch.randn(t.shape, generator=g).to(dev) * s
                for t, s in ((X, 1.0), (Wg, d ** -0.5), (Wu, d ** -0.5))]

        def value(e):
            h = dust.dust_gated_up(X + e * dirs[0], Wg + e * dirs[1], Wu + e * dirs[2], ACTS[act])
            return (h.double() * gh.double()).sum().item()

        e = 2.0 ** -8
        slope = (value(e) - value(-e)) / (2 * e)
        want = sum((a.double() * b.double()).sum().item() for a, b in zip((gX, gWg, gWu), dirs))
        scale = sum((a.double() * b.double()).norm().item() for a, b in zip((gX, gWg, gWu), dirs))
        assert abs(slope - want) <= 2e-3 * scale, act


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f", [(40, 72, 200), (700, 96, 130)])
def test_one_gradient_alone(T, d, f, dtype):
    """Through the C call, which takes NULL for what is not wanted."""
    import torch
    dev = cuda()
    X, Wg, Wu, gh = _inputs(T, d, f, dtype, dev)
    want = dust.dust_gated_up_grad(gh, X, Wg, Wu)
    code = dust.BF16 if dtype == "bf16" else dust.F32
    n = dust._query("dust_gated_up_grad_workspace", T, d, f, code)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    for keep in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)):
        outs = [torch.full_like(w, 7.0) if k else None for w, k in zip(want, keep)]
        st = dust.lib().dust_gated_up_grad(
            p(gh), gh.stride(0), p(X), X.stride(0), p(Wg), Wg.stride(0), p(Wu), Wu.stride(0), code, T,
            d, f, dust.SILU, 0, p(outs[0]), d, p(outs[1]), p(outs[2]), dust.F32, p(ws), n, None)
        assert st == dust.OK
        for a, b in zip(outs, want):
            # the slices of a sum go by the sizes alone: the same bits
            assert a is None or torch.equal(a, b), keep


def test_many_tiles_and_long_sums():
    """Several groups of row tiles, both widths of tiles, sums over thousands of
    rows and units, against 64 bits on the GPU."""
    import torch
    dev = cuda()
    for T, d, f, dtype in ((20000, 64, 96, "bf16"), (9000, 520, 1000, "bf16"), (5000, 200, 300, "f32"),
                           (300, 3000, 5000, "bf16"), (260, 1500, 2000, "f32")):
        X, Wg, Wu, gh = _inputs(T, d, f, dtype, dev)
        x, wg, wu, g64 = (t.double() for t in (X, Wg, Wu, gh))
        g, u = x @ wg.t(), x @ wu.t()
        p = 1.0 / (1.0 + torch.exp(-g))
        dG, dU = g64 * u * (p + g * p * (1 - p)), g64 * g * p
        off = 2 * BF16_TOL if dtype == "bf16" else 0
        off += 8 * f32_tol(max(T, d, 2 * f))
        got = (dust.dust_gated_up(X, Wg, Wu), *dust.dust_gated_up_grad(gh, X, Wg, Wu, gW_dtype=X.dtype))
        for a, b in zip(got, (g * p * u, dG @ wg + dU @ wu, dG.t() @ x, dU.t() @ x)):
            assert ((a.double() - b).norm() / b.norm()).item() <= off, (T, d, f)


def test_bounded_wait_that_runs_out_is_reported():
    """As for the head: the hook makes the issuing thread wait for nothing; the
    kernel gives up after its limit, reports it, and the next call is right."""
    import torch
    dev = cuda()
    X, Wg, Wu, gh = _inputs(300, 64, 700, "bf16", dev)
    want, wanted = dust.dust_gated_up(X, Wg, Wu), dust.dust_gated_up_grad(gh, X, Wg, Wu)
    assert dust.dust_last_error() == dust.OK
    dust.lib().dust_debug_inject_timeout(1)
    dust.dust_gated_up(X, Wg, Wu)
    assert dust.dust_last_error() == dust.ERR_TIMEOUT
    assert torch.equal(dust.dust_gated_up(X, Wg, Wu), want)
    dust.lib().dust_debug_inject_timeout(1)
    dust.dust_gated_up_grad(gh, X, Wg, Wu)
    assert dust.dust_last_error() == dust.ERR_TIMEOUT
    for a, b in zip(dust.dust_gated_up_grad(gh, X, Wg, Wu), wanted):
        assert torch.equal(a, b)
    assert dust.dust_last_error() == dust.OK


def test_on_another_stream_and_in_a_graph():
    import torch
    dev = cuda()
    T, d, f = 300, 96, 160
    X, Wg, Wu, gh = _inputs(T, d, f, "bf16", dev)
    want = dust.dust_gated_up(X, Wg, Wu)
    wanted = dust.dust_gated_up_grad(gh, X, Wg, Wu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h = dust.dust_gated_up(X, Wg, Wu, stream=s)
    grads = dust.dust_gated_up_grad(gh, X, Wg, Wu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert (h == want).all() and all((a == b).all() for a, b in zip(grads, wanted))
    h.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dust.dust_gated_up(X, Wg, Wu, h=h)
        outs = dust.dust_gated_up_grad(gh, X, Wg, Wu)
    X.mul_(0.5)
    graph.replay()
    assert (h == dust.dust_gated_up(X, Wg, Wu)).all()
    for a, b in zip(outs, dust.dust_gated_up_grad(gh, X, Wg, Wu)):
        assert (a == b).all()
