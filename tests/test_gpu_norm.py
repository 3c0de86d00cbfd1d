"""GPU parity of the layer norm and its gradients against the formulas in 64
bits (numpy, on the CPU).

Tolerances, normwise relative. fp32 outputs: each is a handful of fp32
roundings (2^-24 = 6e-8 each) on top of fp32 sums of n terms kept as partial
sums of at most a few hundred sequential terms, whose error is at most about
n_seq 2^-24 relative to the sum of magnitudes; 2e-6 covers sums of mixed
signs here. bf16 outputs: one rounding, half a step of 2^-8 relative, 2^-8
elementwise and 2.5e-3 normwise (the rms of a uniform half step)."""
import numpy as np
import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda, rel_fro

pytestmark = pytest.mark.gpu

F32_TOL, BF16_TOL = 2e-6, 2.5e-3

SIZES = [(1, 1), (1, 512), (2, 7), (3, 33), (37, 64), (129, 96), (300, 513), (64, 1000),
         (1000, 256), (257, 2048), (65, 1531), (33, 4096), (17, 5003), (9, 8192), (5, 20000),
         (4099, 40)]


def _np(t):
    return t.double().cpu().numpy()


def _inputs(T, d, dtype, dev, ld_extra=0, seed=0):
    import torch
    g = torch.Generator().manual_seed(1000 * T + d + seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def rows(scale, off):
        full = (torch.randn((T, d + ld_extra), generator=g) * scale + off).to(dt).to(dev)
        return full[:, :d]

    x, gy = rows(1.5, 0.7), rows(0.5, 0.05)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(dev)
    b = (0.3 * torch.randn(d, generator=g)).to(dev)
    return x, gy, w, b


def _forward(x, w, b, eps):
    x = _np(x)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    n = (x - mean[:, None]) * rstd[:, None]
    return n * (1.0 if w is None else _np(w)) + (0.0 if b is None else _np(b)), mean, rstd


def _backward(gy, x, w, mean, rstd):
    gy, x = _np(gy), _np(x)
    mean, rstd = _np(mean)[:, None], _np(rstd)[:, None]
    n = (x - mean) * rstd
    gn = gy * (1.0 if w is None else _np(w))
    gx = rstd * (gn - gn.mean(1, keepdims=True) - n * (gn * n).mean(1, keepdims=True))
    return gx, (gy * n).sum(0), gy.sum(0)


def _tol(dtype):
    return F32_TOL if dtype == "f32" else BF16_TOL


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", SIZES)
def test_forward_and_gradients(T, d, dtype):
    dev = cuda()
    x, gy, w, b = _inputs(T, d, dtype, dev)
    y, mean, rstd = dust.dust_layer_norm(x, w, b, 1e-5)
    wy, wm, wr = _forward(x, w, b, 1e-5)
    assert y.dtype == x.dtype
    assert np.abs(_np(mean) - wm).max() <= 2e-6 * max(1.0, np.abs(_np(x)).max())
    assert rel_fro(_np(rstd), wr) <= F32_TOL
    # rows of one or two values: n is a sign, and its rounding follows rstd's
    assert rel_fro(_np(y), wy) <= _tol(dtype) + (1e-5 if d < 8 else 0)
    gx, gw, gb = dust.dust_layer_norm_grad(gy, x, mean, rstd, w)
    wx, ww, wb = _backward(gy, x, w, mean, rstd)
    # gx is a difference: its error is that of its terms, rstd |gy weight|
    terms = np.linalg.norm(_np(rstd)[:, None] * _np(gy) * _np(w))
    assert np.linalg.norm(_np(gx) - wx) <= F32_TOL * terms + \
        (BF16_TOL * np.linalg.norm(wx) if dtype == "bf16" else 0)
    n = np.abs(_forward(x, None, None, 1e-5)[0])
    assert np.all(np.abs(_np(gw) - ww) <= 4e-6 * ((np.abs(_np(gy)) * n).sum(0) + 1e-30))
    assert np.all(np.abs(_np(gb) - wb) <= 4e-6 * (np.abs(_np(gy)).sum(0) + 1e-30))
    again = dust.dust_layer_norm_grad(gy, x, mean, rstd, w)
    for p, q in zip((gx, gw, gb), again):
        assert (p == q).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,extra", [(50, 512, 8), (50, 512, 3), (33, 100, 28), (20, 2048, 1)])
def test_strided_rows_and_missing_parameters(T, d, extra, dtype):
    import torch
    dev = cuda()
    x, gy, w, b = _inputs(T, d, dtype, dev, ld_extra=extra)
    assert not x.is_contiguous()
    out = torch.full((T, d + 5), 7.0, dtype=x.dtype, device=dev)
    y, mean, rstd = dust.dust_layer_norm(x, None, b, 1e-3, y=out[:, :d])
    assert rel_fro(_np(y), _forward(x, None, b, 1e-3)[0]) <= _tol(dtype)
    assert (out[:, d:] == 7.0).all()
    gx, gw, gb = dust.dust_layer_norm_grad(gy, x, mean, rstd, None)
    wx, ww, wb = _backward(gy, x, None, mean, rstd)
    assert rel_fro(_np(gx), wx) <= 2 * _tol(dtype)
    assert rel_fro(_np(gw), ww) <= 4e-6 and rel_fro(_np(gb), wb) <= 4e-6
    y2, _, _ = dust.dust_layer_norm(x, w, None, 1e-3)
    assert rel_fro(_np(y2), _forward(x, w, None, 1e-3)[0]) <= _tol(dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [1, 3])
def test_rows_that_start_off_16_bytes(dtype, off):
    import torch
    dev = cuda()
    T, d = 40, 256
    x, gy, w, b = _inputs(T, d, dtype, dev)
    flat = torch.empty(T * d + off, dtype=x.dtype, device=dev)
    xo = flat[off:].view(T, d)
    xo.copy_(x)
    y, mean, rstd = dust.dust_layer_norm(xo, w[:], b)
    y0, m0, r0 = dust.dust_layer_norm(x, w, b)
    assert rel_fro(_np(y), _np(y0)) <= _tol(dtype) and rel_fro(_np(rstd), _np(r0)) <= F32_TOL
    gx, gw, gb = dust.dust_layer_norm_grad(gy, xo, mean, rstd, w)
    wx, ww, wb = _backward(gy, x, w, mean, rstd)
    assert rel_fro(_np(gx), wx) <= 2 * _tol(dtype) and rel_fro(_np(gw), ww) <= 4e-6


@pytest.mark.parametrize("d", [96, 512, 1531, 8192])
def test_accumulates_and_runs_in_place(d):
    import torch
    dev = cuda()
    T = 77
    x, gy, w, b = _inputs(T, d, "f32", dev)
    y, mean, rstd = dust.dust_layer_norm(x, w, b)
    gx, gw, gb = dust.dust_layer_norm_grad(gy, x, mean, rstd, w)
    aw, ab = torch.full_like(gw, 2.0), torch.full_like(gb, -3.0)
    dust.dust_layer_norm_grad(gy, x, mean, rstd, w, flags=dust.ACCUMULATE, gweight=aw, gbias=ab)
    assert torch.allclose(aw, gw + 2.0, rtol=1e-6, atol=1e-6)
    assert torch.allclose(ab, gb - 3.0, rtol=1e-6, atol=1e-6)
    inplace = gy.clone()
    dust.dust_layer_norm_grad(inplace, x, mean, rstd, w, gx=inplace)
    assert torch.equal(inplace, gx)
    xi = x.clone()
    dust.dust_layer_norm(xi, w, b, y=xi)
    assert torch.equal(xi, y)


def test_offset_rows_keep_their_variance():
    """Rows far off zero: the variance comes from deviations, so an offset of
    1000 costs no more than the inputs' own rounding there (none: they are
    exact in fp32). Its error is the mean's, 1000 2^-24, against deviations
    of 1."""
    import torch
    dev = cuda()
    x = (torch.randn((64, 768), generator=torch.Generator().manual_seed(5)) + 1000.0).to(dev)
    y, mean, rstd = dust.dust_layer_norm(x)
    wy, wm, wr = _forward(x, None, None, 1e-5)
    assert rel_fro(_np(rstd), wr) <= 1e-5
    assert np.abs(_np(y) - wy).max() <= 4e-4


def test_non_finite_rows_stay_in_their_rows():
    import torch
    dev = cuda()
    x, gy, w, b = _inputs(40, 320, "bf16", dev)
    x = x.clone()
    x[3, 7], x[11, 0], x[20] = float("nan"), float("inf"), float("-inf")
    y, _, _ = dust.dust_layer_norm(x, w, b)
    bad = [3, 11, 20]
    good = [i for i in range(40) if i not in bad]
    assert torch.isnan(y[bad].float()).any(1).all()
    assert torch.isfinite(y[good].float()).all()
    assert rel_fro(_np(y[good]), _forward(x[good], w, b, 1e-5)[0]) <= BF16_TOL


@pytest.mark.parametrize("d", [24, 130])
def test_gradients_against_differences(d):
    """gx, gweight and gbias of L = sum gy y against central differences of the
    64-bit forward along random directions: step 1e-5, error of order 1e-9
    from the 64-bit side, so the fp32 gradients' own error bounds it."""
    dev = cuda()
    rng = np.random.default_rng(d)
    x, gy, w, b = _inputs(6, d, "f32", dev)
    _, mean, rstd = dust.dust_layer_norm(x, w, b)
    gx, gw, gb = (_np(v) for v in dust.dust_layer_norm_grad(gy, x, mean, rstd, w))

    def loss(xx, ww, bb):
        m = xx.mean(1, keepdims=True)
        n = (xx - m) / np.sqrt(((xx - m) ** 2).mean(1, keepdims=True) + 1e-5)
        return float((_np(gy) * (n * ww + bb)).sum())

    h = 1e-5
    for grad, k in ((gx, 0), (gw, 1), (gb, 2)):
        args = [_np(x), _np(w), _np(b)]
        u = rng.standard_normal(grad.shape)
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + h * u, args[k] - h * u
        want = (loss(*up) - loss(*dn)) / (2 * h)
        assert abs(float((grad * u).sum()) - want) <= 1e-5 * np.linalg.norm(grad) * np.linalg.norm(u)


def test_another_stream_and_empty_sizes():
    import torch
    dev = cuda()
    x, gy, w, b = _inputs(200, 512, "bf16", dev)
    y0, m0, r0 = dust.dust_layer_norm(x, w, b)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y1, m1, r1 = dust.dust_layer_norm(x, w, b, stream=st)
    g1 = dust.dust_layer_norm_grad(gy, x, m1, r1, w, stream=st)
    st.synchronize()
    assert torch.equal(y0, y1)
    g0 = dust.dust_layer_norm_grad(gy, x, m0, r0, w)
    for p, q in zip(g0, g1):
        assert torch.equal(p, q)
    e = torch.empty((0, 16), device=dev)
    z = torch.empty(0, device=dev)
    dust.dust_layer_norm(e)
    _, gw, gb = dust.dust_layer_norm_grad(e, e, z, z, gweight=torch.ones(16, device=dev),
                                          gbias=torch.ones(16, device=dev))
    assert torch.count_nonzero(gw).item() == 0 and torch.count_nonzero(gb).item() == 0
    assert dust.dust_last_error() == dust.OK


def test_binding_refuses_what_it_would_misread():
    import torch
    dev = cuda()
    x = torch.zeros((4, 8), device=dev)
    v = torch.zeros(8, device=dev)
    t = torch.zeros(4, device=dev)
    with pytest.raises(ValueError):
        dust.dust_layer_norm(x.double())
    with pytest.raises(ValueError):
        dust.dust_layer_norm(x.t())
    with pytest.raises(ValueError):
        dust.dust_layer_norm(x, v[:7])
    with pytest.raises(ValueError):
        dust.dust_layer_norm(x, v.to(torch.bfloat16))
    with pytest.raises(ValueError):
        dust.dust_layer_norm(x, v, y=x.to(torch.bfloat16))
    with pytest.raises(dust.DustError):
        dust.dust_layer_norm(x, eps=float("nan"))
    with pytest.raises(ValueError):
        dust.dust_layer_norm_grad(x, x.to(torch.bfloat16), t, t)
    with pytest.raises(ValueError):
        dust.dust_layer_norm_grad(x, x, t[:3], t)
    with pytest.raises(ValueError):
        dust.dust_layer_norm_grad(x, x, t, t, flags=dust.ACCUMULATE)
    with pytest.raises(dust.DustError):
        dust.dust_layer_norm_grad(x, x, t, t, flags=dust.CENTER)
    with pytest.raises(dust.DustError):
        dust.dust_layer_norm_grad(x, x, t, t, workspace=torch.empty(4, dtype=torch.uint8,
                                                                    device=dev))
