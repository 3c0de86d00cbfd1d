"""GPU parity of the head's cross entropy and of the distillation from top
logits, with their gradients, against the formulas in 64 bits (numpy).

Tolerances, all before the first run:
- logits: fp32 sums of d products. In 64 bits the reference is exact; the
  fp32 sum's error is below sqrt(d) 2^-24 sum|h e| ~ 4e-6 times the row's
  magnitude here. Losses and log-sums: 1e-5 absolute per unit of
  max(1, |x|max).
- fp32 gradients: exp of a logit off by 1e-5 is off by 1e-5 relative:
  normwise 2e-5.
- bf16 gradients: G is rounded to bf16 (half step 2^-9 relative, at most
  2e-3 rms after division by the largest weight) and a bf16 result once more:
  normwise 5e-3.
"""
import numpy as np
import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda, rel_fro

pytestmark = pytest.mark.gpu

GRAD_TOL = {"f32": 2e-5, "bf16": 5e-3}

# S, T, d, V: single tokens, ragged and odd sizes, sizes about the tiles'
# edges (64, 128, 256 rows and columns), vocabularies of many tiles (those of
# several pieces: test_gpu_head_pieces.py).
SIZES = [(1, 1, 8, 5), (1, 1, 512, 4096), (1, 3, 64, 2), (2, 5, 33, 17), (1, 127, 64, 255),
         (1, 128, 64, 256), (1, 129, 72, 257), (1, 256, 128, 512), (1, 257, 136, 1000),
         (3, 100, 96, 777), (1, 300, 301, 2049), (1, 64, 1024, 5000), (1, 2, 2056, 300),
         (4, 65, 40, 9001), (1, 700, 16, 640)]


def _np(t):
    return t.double().cpu().numpy()


def _inputs(S, T, d, V, dtype, dev, seed=0):
    import torch
    g = torch.Generator().manual_seed(7 * S + 31 * T + 101 * d + V + seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    H = torch.randn((S, T, d), generator=g).to(dt).to(dev)
    if S == 1:
        H = H[0]
    E = (torch.randn((V, d), generator=g) * (2.0 / d ** 0.5)).to(dt).to(dev)
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    y[torch.rand(T, generator=g) < 0.15] = -1
    gl = torch.randn(H.shape[:-1], generator=g) * 0.1
    return H, E, y.to(dev), gl.to(dev)


def _teacher(T, V, K, dev, seed=0):
    import torch
    g = torch.Generator().manual_seed(T + V + K + seed)
    ids = torch.stack([torch.randperm(max(V, K), generator=g)[:K] for _ in range(T)])
    ids = torch.where(ids < V, ids, -1).to(torch.int32)
    z = torch.randn((T, K), generator=g) * 3
    ids[torch.rand((T, K), generator=g) < 0.1] = -1
    if T > 2:
        ids[1] = -1                    # a row without entries
        z[1] = float("nan")
        z[2, : (K + 1) // 2] = float("-inf")
    return ids.to(dev), z.to(dev)


def _probs(ids, z, scale):
    ids, z = ids.cpu().numpy(), _np(z)
    q = np.zeros(z.shape)
    for t in range(ids.shape[0]):
        have = ids[t] >= 0
        if have.any() and np.isfinite(z[t][have]).any():
            e = np.exp(scale * (z[t][have] - z[t][have].max()))
            q[t, have] = e / e.sum()
    return q


def _x(H, E, scale):
    H = _np(H).reshape(-1, H.shape[-1])
    return scale * (H @ _np(E).T)


def _lse(x):
    m = x.max(1)
    return m + np.log(np.exp(x - m[:, None]).sum(1))


def _grads(H, E, G, scale):
    Hn = _np(H).reshape(-1, H.shape[-1])
    live = np.abs(G).sum(1) > 0
    gE = scale * G[live].T @ Hn[live]
    return scale * (G @ _np(E)).reshape(tuple(H.shape)), gE


def _check_grads(gH, gE, wH, wE, dtype):
    assert rel_fro(_np(gH), wH) <= GRAD_TOL[dtype]
    assert rel_fro(_np(gE), wE) <= GRAD_TOL[dtype]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,T,d,V", SIZES)
def test_loss_and_gradients(S, T, d, V, dtype):
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(S, T, d, V, dtype, dev)
    scale = 1.25
    loss, lse, *rest = dust.dust_head_loss(H, E, y, scale, changes=S > 1)
    x = _x(H, E, scale)
    wl = _lse(x)
    yn = np.tile(y.cpu().numpy(), S)
    r = np.arange(S * T)
    want = np.where(yn >= 0, wl - x[r, np.maximum(yn, 0)], 0.0)
    tol = 1e-5 * max(1.0, np.abs(x).max())
    assert np.abs(_np(lse).ravel() - wl).max() <= tol
    assert np.abs(_np(loss).ravel() - want).max() <= 2 * tol
    assert (loss.reshape(-1)[torch.from_numpy(yn < 0).to(dev)] == 0).all()
    if S > 1:
        w = want.reshape(S, T)
        assert np.abs(_np(rest[0]) - (w[1:] - w[:1])).max() <= 4 * tol
    G = np.exp(x - _np(lse).reshape(-1, 1))
    G[r, np.maximum(yn, 0)] -= 1.0
    G *= np.where(yn >= 0, _np(gl).ravel(), 0.0)[:, None]
    wH, wE = _grads(H, E, G, scale)
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl, scale)
    assert gE.dtype == torch.float32 and gH.dtype == H.dtype and gH.shape == H.shape
    _check_grads(gH, gE, wH, wE, dtype)
    assert (gH.reshape(S * T, d)[torch.from_numpy(yn < 0).to(dev)] == 0).all()
    again = dust.dust_head_loss_grad(H, E, y, lse, gl, scale)
    assert torch.equal(again[0], gH) and torch.equal(again[1], gE)
    if dtype == "bf16":
        _, gb = dust.dust_head_loss_grad(H, E, y, lse, gl, scale, gE_dtype=torch.bfloat16)
        assert gb.dtype == torch.bfloat16 and torch.equal(gb, gE.to(torch.bfloat16))
    acc = torch.full_like(gE, 0.5)
    dust.dust_head_loss_grad(H, E, y, lse, gl, scale, flags=dust.ACCUMULATE, gE=acc)
    assert torch.allclose(acc, gE + 0.5, rtol=1e-6, atol=1e-6)
    assert dust.dust_last_error() == dust.OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,T,d,V,K", [(1, 1, 8, 5, 1), (1, 7, 64, 300, 3), (2, 33, 40, 257, 5),
                                       (1, 130, 128, 1000, 64), (1, 65, 129, 5003, 33),
                                       (1, 300, 512, 4096, 128), (1, 9, 32, 20, 40),
                                       (3, 20, 72, 600, 257)])
def test_distillation_and_gradients(S, T, d, V, K, dtype):
    import torch
    dev = cuda()
    H, E, _, gl = _inputs(S, T, d, V, dtype, dev, seed=1)
    ids, z = _teacher(T, V, K, dev)
    scale = 0.5
    loss, lse, student, *rest = dust.dust_distill_loss(H, E, ids, z, scale, changes=S > 1)
    x = _x(H, E, scale)
    wl = _lse(x)
    q = np.tile(_probs(ids, z, scale), (S, 1))
    idn = np.tile(ids.cpu().numpy(), (S, 1))
    r = np.arange(S * T)[:, None]
    ws = np.where(idn >= 0, x[r, np.maximum(idn, 0)], 0.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        terms = np.where(q > 0, q * (np.log(q) - (ws - wl[:, None])), 0.0)
    tol = 1e-5 * max(1.0, np.abs(x).max())
    assert np.abs(_np(lse).ravel() - wl).max() <= tol
    assert np.abs(_np(student).reshape(S * T, K) - ws).max() <= tol
    assert np.abs(_np(loss).ravel() - terms.sum(1)).max() <= 2 * tol
    if S > 1:
        w = terms.sum(1).reshape(S, T)
        assert np.abs(_np(rest[0]) - (w[1:] - w[:1])).max() <= 4 * tol
    G = np.exp(x - _np(lse).reshape(-1, 1)) * (q.sum(1, keepdims=True) > 0)
    for j in range(K):
        np.add.at(G, (r[:, 0], np.maximum(idn[:, j], 0)), -q[:, j])
    G *= _np(gl).reshape(-1, 1)
    wH, wE = _grads(H, E, G, scale)
    gH, gE = dust.dust_distill_loss_grad(H, E, ids, z, lse, student, gl, scale)
    _check_grads(gH, gE, wH, wE, dtype)
    again = dust.dust_distill_loss_grad(H, E, ids, z, lse, student, gl, scale)
    assert torch.equal(again[0], gH) and torch.equal(again[1], gE)
    assert dust.dust_last_error() == dust.OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_id_that_comes_twice(dtype):
    import torch
    dev = cuda()
    H, E, _, gl = _inputs(1, 40, 64, 300, dtype, dev, seed=2)
    ids = torch.randint(0, 300, (40, 12), generator=torch.Generator().manual_seed(3),
                        dtype=torch.int32)
    ids[:, 7], ids[:, 9], ids[:, 3] = ids[:, 2], ids[:, 2], ids[:, 11]
    ids = ids.to(dev)
    z = torch.randn((40, 12), generator=torch.Generator().manual_seed(4)).to(dev)
    loss, lse, student = dust.dust_distill_loss(H, E, ids, z)
    x = _x(H, E, 1.0)
    q, idn, r = _probs(ids, z, 1.0), ids.cpu().numpy(), np.arange(40)
    G = np.exp(x - _np(lse)[:, None])
    for j in range(12):
        np.add.at(G, (r, idn[:, j]), -q[:, j])
    wH, wE = _grads(H, E, G * _np(gl)[:, None], 1.0)
    gH, gE = dust.dust_distill_loss_grad(H, E, ids, z, lse, student, gl)
    _check_grads(gH, gE, wH, wE, dtype)


def test_distilling_from_one_entry_is_cross_entropy():
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(1, 150, 96, 700, "bf16", dev, seed=5)
    z = torch.randn((150, 1), generator=torch.Generator().manual_seed(6)).to(dev)
    loss, lse = dust.dust_head_loss(H, E, y)
    loss2, lse2, student = dust.dust_distill_loss(H, E, y[:, None].contiguous(), z)
    assert torch.equal(lse, lse2) and torch.allclose(loss, loss2, rtol=1e-6, atol=2e-6)
    a = dust.dust_head_loss_grad(H, E, y, lse, gl)
    b = dust.dust_distill_loss_grad(H, E, y[:, None].contiguous(), z, lse, student, gl)
    for p, q in zip(a, b):
        assert rel_fro(_np(p), _np(q)) <= 2.5e-3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_without_targets_hide_what_they_hold(dtype):
    """Padding: hidden states of NaN and infinity in rows that have no target,
    or whose loss has no weight, reach neither gradient."""
    import torch
    dev = cuda()
    T = 200
    H, E, y, gl = _inputs(1, T, 72, 333, dtype, dev, seed=8)
    y = torch.randint(0, 333, (T,), generator=torch.Generator().manual_seed(9),
                      dtype=torch.int32).to(dev)
    clean = H.clone()
    y[::3] = -1
    gl[1::3] = 0.0
    gl[::3] = float("nan")
    H[::3] = float("nan")
    H[1::6] = float("inf")
    loss, lse = dust.dust_head_loss(H, E, y)
    assert (loss[::3] == 0).all()
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl)
    live = torch.arange(2, T, 3, device=dev)
    want = dust.dust_head_loss_grad(clean[live], E, y[live], lse[live], gl[live])
    assert rel_fro(_np(gE), _np(want[1])) <= 1e-6
    assert rel_fro(_np(gH[live]), _np(want[0])) <= GRAD_TOL[dtype]
    # the same bits as with ordinary values there
    same = dust.dust_head_loss_grad(clean, E, y, lse, torch.nan_to_num(gl))
    assert torch.equal(gH, same[0]) and torch.equal(gE, same[1])
    rest = torch.ones(T, dtype=torch.bool, device=dev)
    rest[live] = False
    assert (gH[rest] == 0).all()
    ids, z = _teacher(T, 333, 6, dev)
    ids[::3] = -1
    loss, lse, student = dust.dust_distill_loss(H, E, ids, z)
    assert (loss[::3] == 0).all()
    gH, gE = dust.dust_distill_loss_grad(H, E, ids, z, lse, student, gl)
    assert torch.isfinite(gE).all() and torch.isfinite(gH.float()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 9000])
def test_batches_without_any_target(dtype, V):
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(1, 70, 48, V, dtype, dev, seed=10)
    y.fill_(-1)
    loss, lse = dust.dust_head_loss(H, E, y)
    assert (loss == 0).all()
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl, gE=torch.ones((V, 48), device=dev))
    assert (gH == 0).all() and (gE == 0).all()
    kept = torch.ones((V, 48), device=dev)
    dust.dust_head_loss_grad(H, E, y, lse, gl, flags=dust.ACCUMULATE, gE=kept)
    assert (kept == 1).all()
    ids = torch.full((70, 4), -1, dtype=torch.int32, device=dev)
    z = torch.zeros((70, 4), device=dev)
    loss, lse, student = dust.dust_distill_loss(H, E, ids, z)
    assert (loss == 0).all() and (student == 0).all()
    gH, gE = dust.dust_distill_loss_grad(H, E, ids, z, lse, student, gl)
    assert (gH == 0).all() and (gE == 0).all()
    # no tokens at all
    gH, gE = dust.dust_head_loss_grad(H[:0], E, y[:0], lse[:0], gl[:0],
                                      gE=torch.ones((V, 48), device=dev))
    assert gH.shape == (0, 48) and (gE == 0).all()


def test_large_logits_neither_overflow_nor_vanish():
    """Logits of +-300: exp of them overflows fp32, and a confident row's loss
    is 0 to fp32 accuracy."""
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(1, 130, 64, 513, "bf16", dev, seed=11)
    H = (H * 40).contiguous()
    loss, lse = dust.dust_head_loss(H, E, y)
    x = _x(H, E, 1.0)
    wl = _lse(x)
    assert np.abs(x).max() > 200
    assert np.abs(_np(lse) - wl).max() <= 1e-5 * np.abs(x).max()
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl)
    yn = y.cpu().numpy()
    # exp(x - lse) with both near 300: their fp32 steps (3e-5) set its error
    G = np.exp(x - _np(lse)[:, None])
    G[np.arange(130), np.maximum(yn, 0)] -= 1
    G *= np.where(yn >= 0, _np(gl), 0.0)[:, None]
    wH, wE = _grads(H, E, G, 1.0)
    assert rel_fro(_np(gH), wH) <= 5e-3 and rel_fro(_np(gE), wE) <= 5e-3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,extra,off", [(64, 8, 0), (64, 3, 0), (100, 28, 4), (64, 0, 1)])
def test_strides_and_alignments(d, extra, off, dtype):
    import torch
    dev = cuda()
    T, V = 90, 400
    H, E, y, gl = _inputs(1, T, d, V, dtype, dev, seed=12)

    def placed(t):
        flat = torch.full((t.shape[0] * (d + extra) + off,), float("nan"), dtype=t.dtype,
                          device=dev)
        v = flat[off:].view(t.shape[0], d + extra)[:, :d]
        v.copy_(t)
        return v

    loss, lse = dust.dust_head_loss(H, E, y)
    l2, e2 = dust.dust_head_loss(placed(H), placed(E), y)
    assert np.abs(_np(loss) - _np(l2)).max() <= 1e-4 and np.abs(_np(lse) - _np(e2)).max() <= 1e-4
    a = dust.dust_head_loss_grad(H, E, y, lse, gl)
    b = dust.dust_head_loss_grad(placed(H), placed(E), y, lse, gl)
    for p, q in zip(a, b):
        assert rel_fro(_np(p), _np(q)) <= GRAD_TOL[dtype]


def test_slices_with_a_row_stride():
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(3, 50, 64, 300, "bf16", dev, seed=13)
    wide = torch.zeros((3, 50, 80), dtype=H.dtype, device=dev)
    wide[:, :, :64] = H
    a = dust.dust_head_loss(H, E, y, changes=True)
    b = dust.dust_head_loss(wide[:, :, :64], E, y, changes=True)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    with pytest.raises(ValueError):
        dust.dust_head_loss(H[:, :49], E, y[:49])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_vocabulary_of_one(dtype):
    """One row: the loss and both gradients are 0 (exp(x - lse) is 1), up to
    the fp32 rounding of lse, 1e-5 of the terms that cancel."""
    dev = cuda()
    H, E, y, gl = _inputs(1, 9, 64, 1, dtype, dev)
    y.zero_()
    loss, lse = dust.dust_head_loss(H, E, y)
    x = np.abs(_x(H, E, 1.0)).max()
    assert np.abs(_np(loss)).max() <= 1e-5 * max(1.0, x)
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl)
    g = np.abs(_np(gl)).max()
    assert np.abs(_np(gH)).max() <= 1e-5 * g * np.abs(_np(E)).max()
    assert np.abs(_np(gE)).max() <= 1e-5 * g * np.abs(_np(H)).sum(0).max()


@pytest.mark.parametrize("distill", [False, True])
def test_gradients_against_differences(distill):
    """The fp32 gradients of L = sum gl loss against central differences of the
    64-bit loss along random directions (step 1e-5)."""
    dev = cuda()
    rng = np.random.default_rng(3)
    T, d, V, K, scale = 9, 24, 60, 5, 0.7
    H, E, y, gl = _inputs(1, T, d, V, "f32", dev, seed=14)
    ids, z = _teacher(T, V, K, dev, seed=2)
    if distill:
        _, lse, student = dust.dust_distill_loss(H, E, ids, z, scale)
        gH, gE = dust.dust_distill_loss_grad(H, E, ids, z, lse, student, gl, scale)
        q = _probs(ids, z, scale)
        want = np.zeros((T, V))
        for j in range(K):
            np.add.at(want, (np.arange(T), np.maximum(ids.cpu().numpy()[:, j], 0)), q[:, j])
    else:
        _, lse = dust.dust_head_loss(H, E, y, scale)
        gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl, scale)
        want = np.zeros((T, V))
        yn = y.cpu().numpy()
        want[np.arange(T)[yn >= 0], yn[yn >= 0]] = 1.0

    def loss(h, e):
        x = scale * (h @ e.T)
        return float((_np(gl)[:, None] * want * (_lse(x)[:, None] - x)).sum())

    Hn, En, h = _np(H), _np(E), 1e-5
    u, v = rng.standard_normal(Hn.shape), rng.standard_normal(En.shape)
    for grad, w, dh, de in ((gH, u, h * u, 0 * v), (gE, v, 0 * u, h * v)):
        diff = (loss(Hn + dh, En + de) - loss(Hn - dh, En - de)) / (2 * h)
        g = _np(grad)
        assert abs(float((g * w).sum()) - diff) <= 1e-5 * np.linalg.norm(g) * np.linalg.norm(w)


def test_only_one_of_the_gradients():
    import ctypes as C
    import torch
    dev = cuda()
    T, d, V = 140, 64, 9000
    H, E, y, gl = _inputs(1, T, d, V, "bf16", dev, seed=15)
    _, lse = dust.dust_head_loss(H, E, y)
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl)
    n = C.c_size_t(0)
    L = dust.lib()
    assert L.dust_head_loss_grad_workspace(C.byref(n), 1, T, d, V, dust.BF16) == dust.OK
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    p = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    for which in ("gH", "gE"):
        oH, oE = torch.full_like(gH, 9.0), torch.full_like(gE, 9.0)
        st = L.dust_head_loss_grad(p(H), d, p(E), d, dust.BF16, 1, T, d, V, p(y), 1.0, p(lse),
                                   p(gl), 0, p(oH) if which == "gH" else None, d,
                                   p(oE) if which == "gE" else None, dust.F32, p(ws), n.value,
                                   C.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == dust.OK
        torch.cuda.synchronize()
        assert torch.equal(oH, gH if which == "gH" else torch.full_like(gH, 9.0))
        assert torch.equal(oE, gE if which == "gE" else torch.full_like(gE, 9.0))


def test_ids_past_the_vocabulary_are_absent_and_reported():
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(1, 60, 64, 300, "bf16", dev, seed=16)
    off = y.clone()
    off[5], y[5] = 300, -1
    off[59], y[59] = 2 ** 31 - 1, -1
    loss, lse = dust.dust_head_loss(H, E, y)
    assert dust.dust_last_error() == dust.OK
    l2, _ = dust.dust_head_loss(H, E, off)
    assert dust.dust_last_error() == dust.ERR_INVALID_ARG
    assert torch.equal(loss, l2)
    a = dust.dust_head_loss_grad(H, E, y, lse, gl)
    b = dust.dust_head_loss_grad(H, E, off, lse, gl)
    assert dust.dust_last_error() == dust.ERR_INVALID_ARG
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ids, z = _teacher(60, 300, 4, dev)
    ids[4, 2] = 1 << 20
    dust.dust_distill_loss(H, E, ids, z)
    assert dust.dust_last_error() == dust.ERR_INVALID_ARG
    assert dust.dust_last_error() == dust.OK


def test_another_stream_gives_the_same_bits():
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(1, 300, 128, 2000, "bf16", dev, seed=17)
    a = dust.dust_head_loss(H, E, y)
    ga = dust.dust_head_loss_grad(H, E, y, a[1], gl)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    b = dust.dust_head_loss(H, E, y, stream=st)
    gb = dust.dust_head_loss_grad(H, E, y, b[1], gl, stream=st.cuda_stream)
    st.synchronize()
    for p, q in zip(a + ga, b + gb):
        assert torch.equal(p, q)


def test_losses_of_jittered_draws_drive_the_estimate():
    """The path a training step takes: a norm, the jittered forward of a layer,
    the head's losses of every slice as loss changes, and the layer's weight
    gradient from them, against the same path in 64 bits from the same noise."""
    import torch
    import oracle
    dev = cuda()
    T, d, V, K, sigma = 256, 64, 500, 6, 0.05
    g = torch.Generator().manual_seed(18)
    x = torch.randn((T, d), generator=g).to(torch.bfloat16).to(dev)
    W = (torch.randn((d, d), generator=g) / d ** 0.5).to(torch.bfloat16).to(dev)
    E = (torch.randn((V, d), generator=g) * (3.0 / d ** 0.5)).to(torch.bfloat16).to(dev)
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).to(dev)
    X, _, _ = dust.dust_layer_norm(x)
    Y = dust.dust_forward_jitter(X, W, 3, dust.GAUSSIAN, 0, K, sigma, clean=True)
    loss, lse, delta = dust.dust_head_loss(Y, E, y, changes=True)
    so = torch.tensor([0, 100, T], dtype=torch.int32, device=dev)
    gW = dust.dust_estimate_gW(X, delta, d, so, 3, dust.GAUSSIAN, 0, sigma, 0.0, 1.0 / T,
                               dust.CENTER)
    assert dust.dust_last_error() == dust.OK
    xn = _x(Y, E, 1.0)
    want = (_lse(xn) - xn[np.arange((K + 1) * T), np.tile(y.cpu().numpy(), K + 1)]).reshape(-1, T)
    # a change is a difference of two losses near 7: fp32 steps of 5e-7 each
    assert np.abs(_np(delta) - (want[1:] - want[:1])).max() <= 1e-4
    ref = oracle.estimate_gW(_np(X), (want[1:] - want[:1]).astype(np.float32), d,
                             so.cpu().numpy(), 3, oracle.GAUSSIAN, 0, sigma, 0.0, 1.0 / T,
                             oracle.CENTER)
    assert rel_fro(_np(gW), ref) <= 1e-2


def test_binding_refuses_what_it_would_misread():
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(1, 20, 32, 50, "bf16", dev, seed=19)
    lse = torch.zeros(20, device=dev)
    ids, z = _teacher(20, 50, 3, dev)
    student = torch.zeros((20, 3), device=dev)
    with pytest.raises(ValueError):
        dust.dust_head_loss(H, E.float(), y)
    with pytest.raises(ValueError):
        dust.dust_head_loss(H, E[:, :31], y)
    with pytest.raises(ValueError):
        dust.dust_head_loss(H, E, y.long())
    with pytest.raises(ValueError):
        dust.dust_head_loss(H, E, y[:19])
    with pytest.raises(ValueError):
        dust.dust_head_loss(H.t(), E, y)
    with pytest.raises(ValueError):
        dust.dust_head_loss(H.half(), E.half(), y)
    with pytest.raises(dust.DustError):
        dust.dust_head_loss(H, E, y, scale=float("inf"))
    with pytest.raises(dust.DustError):
        dust.dust_head_loss(H, E, y, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        dust.dust_head_loss_grad(H, E, y, lse[:4], gl)
    with pytest.raises(ValueError):
        dust.dust_head_loss_grad(H, E, y, lse, gl, gH=H.float())
    with pytest.raises(ValueError):
        dust.dust_head_loss_grad(H, E, y, lse, gl, flags=dust.ACCUMULATE)
    with pytest.raises(dust.DustError):
        dust.dust_head_loss_grad(H, E, y, lse, gl, flags=dust.ACCUMULATE,
                                 gE=torch.zeros_like(E))
    with pytest.raises(dust.DustError):
        dust.dust_head_loss_grad(H.float(), E.float(), y, lse, gl, gE_dtype=torch.bfloat16)
    with pytest.raises(dust.DustError):
        dust.dust_head_loss_grad(H, E, y, lse, gl, flags=dust.CENTER)
    with pytest.raises(ValueError):
        dust.dust_distill_loss(H, E, ids, z.double())
    with pytest.raises(ValueError):
        dust.dust_distill_loss(H, E, ids, z[:, :2])
    with pytest.raises(dust.DustError):
        dust.dust_distill_loss(H, E, ids[:, :0].contiguous(), z[:, :0].contiguous())
    with pytest.raises(ValueError):
        dust.dust_distill_loss_grad(H, E, ids, z, lse, student[:, :2], gl)
    with pytest.raises(dust.DustError):
        big = torch.zeros((20, dust.MAX_TEACHER + 1), device=dev)
        dust.dust_distill_loss(H, E, big.to(torch.int32), big)


def test_bounded_wait_that_runs_out_is_reported():
    """The test hook makes the product's issuing thread wait on a barrier that
    nothing signals; the kernel gives up after its limit, reports it, and the
    next call is right."""
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(1, 300, 64, 700, "bf16", dev, seed=20)
    want = dust.dust_head_loss(H, E, y)
    assert dust.dust_last_error() == dust.OK
    dust.lib().dust_debug_inject_timeout(1)
    dust.dust_head_loss(H, E, y)
    assert dust.dust_last_error() == dust.ERR_TIMEOUT
    again = dust.dust_head_loss(H, E, y)
    assert dust.dust_last_error() == dust.OK
    for p, q in zip(want, again):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_next_to_the_largest(dtype):
    """fp32 operands are split into three bf16 planes: values next to the
    largest fp32, which would round up to infinity in bf16, stay finite. The
    scale makes ordinary logits of their products."""
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(1, 40, 16, 300, dtype, dev, seed=21)
    H *= 3.39e38 / _np(H).__abs__().max() if dtype == "f32" else 1e37
    E *= 1e-8
    assert torch.isfinite(H).all()
    scale = 1e-30
    loss, lse = dust.dust_head_loss(H, E, y, scale)
    x = _x(H, E, scale)
    assert np.abs(_np(lse) - _lse(x)).max() <= 1e-5 * max(1.0, np.abs(x).max())
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl, scale)
    assert torch.isfinite(gH.float()).all() and torch.isfinite(gE).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("d,V", [(512, 4096), (301, 1003), (2048, 700), (8, 20000)])
def test_single_tokens(R, d, V, dtype):
    """Few rows, which take their own way to the loss, against 64 bits, with
    the neighbouring row counts."""
    dev = cuda()
    H, E, y, _ = _inputs(1, R, d, V, dtype, dev, seed=22)
    loss, lse = dust.dust_head_loss(H, E, y, -0.75)
    x = _x(H, E, -0.75)
    wl = _lse(x)
    yn = y.cpu().numpy()
    want = np.where(yn >= 0, wl - x[np.arange(R), np.maximum(yn, 0)], 0.0)
    tol = 1e-5 * max(1.0, np.abs(x).max())
    assert np.abs(_np(lse) - wl).max() <= tol and np.abs(_np(loss) - want).max() <= 2 * tol
    ids, z = _teacher(R, V, 7, dev)
    loss, lse, student = dust.dust_distill_loss(H, E, ids, z, -0.75)
    idn = ids.cpu().numpy()
    ws = np.where(idn >= 0, x[np.arange(R)[:, None], np.maximum(idn, 0)], 0.0)
    assert np.abs(_np(student) - ws).max() <= tol and np.abs(_np(lse) - wl).max() <= tol


@pytest.mark.parametrize("scale", [0.0, -1.5])
def test_scales_of_zero_and_below(scale):
    dev = cuda()
    H, E, y, gl = _inputs(1, 150, 40, 600, "bf16", dev, seed=23)
    loss, lse = dust.dust_head_loss(H, E, y, scale)
    x = _x(H, E, scale)
    assert np.abs(_np(lse) - _lse(x)).max() <= 1e-5 * max(1.0, np.abs(x).max())
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl, scale)
    yn = y.cpu().numpy()
    G = np.exp(x - _np(lse)[:, None])
    G[np.arange(150), np.maximum(yn, 0)] -= 1.0
    G *= np.where(yn >= 0, _np(gl), 0.0)[:, None]
    wH, wE = _grads(H, E, G, scale)
    if scale == 0.0:
        assert (gH == 0).all() and (gE == 0).all()
    else:
        _check_grads(gH, gE, wH, wE, "bf16")


def test_what_is_not_a_number_shows():
    """A teacher's NaN at an entry present, or one in a row of H that has a
    target, gives a loss of NaN in that row alone."""
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(1, 140, 64, 500, "bf16", dev, seed=24)
    ids, z = _teacher(140, 500, 6, dev)
    ids[10], z[10] = torch.arange(6, dtype=torch.int32, device=dev), float("nan")
    ids[11], z[11, 3] = torch.arange(6, dtype=torch.int32, device=dev), float("nan")
    loss, lse, student = dust.dust_distill_loss(H, E, ids, z)
    assert torch.isnan(loss[10:12]).all() and torch.isfinite(lse).all()
    keep = torch.ones(140, dtype=torch.bool, device=dev)
    keep[10:12] = False
    assert torch.isfinite(loss[keep]).all()
    gH, _ = dust.dust_distill_loss_grad(H, E, ids, z, lse, student, gl)
    assert torch.isnan(gH[10:12].float()).any(1).all() and torch.isfinite(gH[keep].float()).all()
    H = H.clone()
    H[7, 5], y[7] = float("nan"), 3
    loss, lse = dust.dust_head_loss(H, E, y)
    keep = torch.arange(140, device=dev) != 7
    assert torch.isnan(loss[7]) and torch.isfinite(loss[keep]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("d,V", [(512, 4096), (301, 1003), (2048, 700), (8, 20000), (898, 129)])
def test_gradients_of_single_tokens(R, d, V, dtype):
    """Few rows, which take their own way to the gradients, with the
    neighbouring row counts; gE also added to what is there."""
    import torch
    dev = cuda()
    scale = 0.75
    H, E, y, gl = _inputs(1, R, d, V, dtype, dev, seed=25)
    if R > 2:
        H[1], y[1] = float("nan"), -1  # takes no part
    _, lse = dust.dust_head_loss(torch.nan_to_num(H), E, y, scale)
    out = torch.full((V, d), 0.5, device=dev)
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl, scale)
    dust.dust_head_loss_grad(H, E, y, lse, gl, scale, dust.ACCUMULATE, gE=out)
    Hz = torch.nan_to_num(H)
    x = _x(Hz, E, scale)
    p = np.exp(x - _lse(x)[:, None])
    yn = y.cpu().numpy()
    w = np.where(yn >= 0, _np(gl), 0.0)[:, None]
    G = p.copy()
    G[np.arange(R), np.maximum(yn, 0)] -= 1.0
    wH, wE = _grads(Hz, E, G * w, scale)
    if (yn >= 0).any():
        _check_grads(gH, gE, wH, wE, dtype)
        # out is 0.5 and more, rounded once: half a step of 2^-24 per value.
        assert (np.linalg.norm(_np(out) - 0.5 - wE) <=
                GRAD_TOL[dtype] * np.linalg.norm(wE) + 2.0 ** -24 * (0.5 * (V * d) ** 0.5 + np.linalg.norm(wE)))
    assert (_np(gH)[yn < 0] == 0).all()
    ids, z = _teacher(R, V, 7, dev)
    H = Hz
    loss, lse, student = dust.dust_distill_loss(H, E, ids, z, scale)
    gH, gE = dust.dust_distill_loss_grad(H, E, ids, z, lse, student, gl, scale)
    q = _probs(ids, z, scale)
    G = p * (q.sum(1) > 0)[:, None]
    idn = ids.cpu().numpy()
    for t in range(R):
        for j in range(7):
            if idn[t, j] >= 0 and q[t, j] > 0:
                G[t, idn[t, j]] -= q[t, j]
    wH, wE = _grads(H, E, G * _np(gl)[:, None], scale)
    if (q.sum(1) > 0).any():
        _check_grads(gH, gE, wH, wE, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_rows_against_more(dtype):
    """The gradients of three rows, and of the same rows among nine of which
    the others take no part: two ways to the same result."""
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(1, 9, 96, 700, dtype, dev, seed=26)
    y[:] = -1
    y[[0, 4, 8]] = torch.tensor([5, 699, 64], dtype=torch.int32, device=dev)
    _, lse = dust.dust_head_loss(H, E, y)
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl)
    few = [t[[0, 4, 8]].contiguous() for t in (H, y, lse, gl)]
    fH, fE = dust.dust_head_loss_grad(few[0], E, *few[1:])
    assert rel_fro(_np(fH), _np(gH)[[0, 4, 8]]) <= 2 * GRAD_TOL[dtype]
    assert rel_fro(_np(fE), _np(gE)) <= 2 * GRAD_TOL[dtype]


@pytest.mark.parametrize("dtype,ge", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("T", [2, 140])
@pytest.mark.parametrize("d,ld,off", [(33, 40, 0), (36, 40, 0), (64, 72, 8), (100, 101, 0), (64, 64, 1),
                                      (130, 136, 2), (8, 16, 0)])
def test_gradients_of_rows_apart(d, ld, off, T, ge, dtype):
    """gH with room between its rows, gH and gE off 16 bytes: nothing is
    written beside them, and the values are those of dense outputs (of a few
    rows: but for the order of the sums, which follows the alignment)."""
    import ctypes as C
    import torch
    dev = cuda()
    V = 333
    H, E, y, gl = _inputs(1, T, d, V, dtype, dev, seed=27)
    _, lse = dust.dust_head_loss(H, E, y)
    ge_type = torch.float32 if ge == "f32" else torch.bfloat16
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl, gE_dtype=ge_type)
    n = C.c_size_t(0)
    L = dust.lib()
    code = dust.BF16 if dtype == "bf16" else dust.F32
    assert L.dust_head_loss_grad_workspace(C.byref(n), 1, T, d, V, code) == dust.OK
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    p = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    flatH = torch.full((T * ld + off + 16,), 9.0, dtype=H.dtype, device=dev)
    flatE = torch.full((V * d + off + 16,), 9.0, dtype=ge_type, device=dev)
    st = L.dust_head_loss_grad(p(H), d, p(E), d, code, 1, T, d, V, p(y), 1.0, p(lse), p(gl), 0,
                               p(flatH[off:]), ld, p(flatE[off:]),
                               dust.F32 if ge == "f32" else dust.BF16, p(ws), n.value,
                               C.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == dust.OK
    rows = flatH[off:off + T * ld].view(T, ld)
    assert (rows[:, d:] == 9.0).all()
    for a, b in ((rows[:, :d], gH), (flatE[off:off + V * d].view(V, d), gE)):
        assert torch.equal(a, b) or T == 2 and rel_fro(_np(a), _np(b)) <= GRAD_TOL[dtype]
    for flat, end in ((flatH, off + T * ld), (flatE, off + V * d)):
        assert (flat[:off] == 9.0).all() and (flat[end:] == 9.0).all()


def test_long_sums_in_fp32():
    """fp32 gradients whose sums run over 8192 rows and 8192 ids. What the
    tensor cores add up at a time is 32 additions of 16 products; each cuts off
    less than 2^-23 of the running sum, half of that on average: together below
    32 * 2^-24 = 2e-6, to which the exponentials' own 2^-22 come."""
    dev = cuda()
    H, E, y, gl = _inputs(1, 8192, 24, 8192, "f32", dev, seed=28)
    _, lse = dust.dust_head_loss(H, E, y)
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl)
    x = _x(H, E, 1.0)
    yn = y.cpu().numpy()
    G = np.exp(x - _lse(x)[:, None])
    G[np.arange(8192), np.maximum(yn, 0)] -= 1.0
    G *= np.where(yn >= 0, _np(gl), 0.0)[:, None]
    wH, wE = _grads(H, E, G, 1.0)
    assert rel_fro(_np(gH), wH) <= 2.5e-6 and rel_fro(_np(gE), wE) <= 2.5e-6


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [1030, 4100])
def test_long_sums_of_logits(d, dtype):
    """Logits over many columns, all products of one sign, where cutting bits
    off adds up most: as above, below 2e-6 of the logit."""
    import torch
    dev = cuda()
    H, E, _, _ = _inputs(1, 40, d, 700, dtype, dev, seed=29)
    H, E = H.abs(), (E.abs() / d ** 0.5)
    ids = torch.arange(40 * 16, dtype=torch.int32, device=dev).view(40, 16)
    _, _, student = dust.dust_distill_loss(H, E, ids, torch.zeros((40, 16), device=dev))
    x = np.take_along_axis(_x(H, E, 1.0), ids.cpu().numpy().astype(np.int64), 1)
    assert (np.abs(_np(student) - x) / x).max() <= 2e-6
