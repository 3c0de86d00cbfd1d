"""Host-side refusals of the layer norm, the head's losses and the
distillation: every call here fails validation (or has nothing to do), so
nothing is enqueued. Runs only where there is no GPU: the addresses are made
up."""
import ctypes as C

import pytest

import token_perturbation_estimator_gb300 as dust

NULL = C.c_void_p(0)
FAKE = C.c_void_p(1 << 20)
ODD = C.c_void_p((1 << 20) + 1)


def _has_gpu():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


pytestmark = pytest.mark.skipif(_has_gpu(), reason="fake device addresses: CPU only")


@pytest.fixture(scope="module")
def L():
    from token_perturbation_estimator_gb300 import build
    build.build()
    return dust.lib()


def _call(fn, defaults, kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


def _norm(L, **kw):
    return _call(L.dust_layer_norm, dict(
        x=FAKE, dt=dust.F32, ld_x=16, T=4, d=16, w=NULL, b=NULL, eps=1e-5, y=FAKE, ld_y=16,
        mean=NULL, rstd=NULL, stream=NULL), kw)


def _norm_grad(L, **kw):
    return _call(L.dust_layer_norm_grad, dict(
        gy=FAKE, ld_gy=16, x=FAKE, ld_x=16, dt=dust.F32, T=4, d=16, w=NULL, mean=FAKE, rstd=FAKE,
        flags=0, gx=FAKE, ld_gx=16, gw=FAKE, gb=FAKE, ws=FAKE, wsb=1 << 30, stream=NULL), kw)


def _loss(L, **kw):
    return _call(L.dust_head_loss, dict(
        H=FAKE, ld_h=16, E=FAKE, ld_e=16, dt=dust.BF16, S=1, T=4, d=16, V=32, y=FAKE, scale=1.0,
        loss=FAKE, lse=FAKE, delta=NULL, ws=FAKE, wsb=1 << 30, stream=NULL), kw)


def _grad(L, **kw):
    return _call(L.dust_head_loss_grad, dict(
        H=FAKE, ld_h=16, E=FAKE, ld_e=16, dt=dust.BF16, S=1, T=4, d=16, V=32, y=FAKE, scale=1.0,
        lse=FAKE, gloss=FAKE, flags=0, gH=FAKE, ld_gh=16, gE=FAKE, gdt=dust.F32, ws=FAKE,
        wsb=1 << 30, stream=NULL), kw)


def _distill(L, **kw):
    return _call(L.dust_distill_loss, dict(
        H=FAKE, ld_h=16, E=FAKE, ld_e=16, dt=dust.BF16, S=1, T=4, d=16, V=32, ids=FAKE, z=FAKE,
        K=3, scale=1.0, loss=FAKE, lse=FAKE, student=FAKE, delta=NULL, ws=FAKE, wsb=1 << 30,
        stream=NULL), kw)


def _distill_grad(L, **kw):
    return _call(L.dust_distill_loss_grad, dict(
        H=FAKE, ld_h=16, E=FAKE, ld_e=16, dt=dust.BF16, S=1, T=4, d=16, V=32, ids=FAKE, z=FAKE,
        K=3, scale=1.0, lse=FAKE, student=FAKE, gloss=FAKE, flags=0, gH=FAKE, ld_gh=16, gE=FAKE,
        gdt=dust.F32, ws=FAKE, wsb=1 << 30, stream=NULL), kw)


def test_layer_norm(L):
    bad = dust.ERR_INVALID_ARG
    for kw in (dict(x=NULL), dict(y=NULL), dict(T=-1), dict(d=-1), dict(ld_x=15), dict(ld_y=15),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(dt=dust.U32),
               dict(dt=9), dict(x=ODD), dict(y=ODD)):
        assert _norm(L, **kw) == bad, kw
    assert _norm(L, T=1 << 31, d=16) == dust.ERR_RANGE
    assert _norm(L, T=1 << 30, d=1 << 12, ld_x=1 << 12, ld_y=1 << 12) == dust.ERR_RANGE
    assert _norm(L, ld_x=1 << 50) == dust.ERR_RANGE
    assert _norm(L, T=0, x=NULL, y=NULL) == dust.OK
    assert _norm(L, d=0, x=NULL, y=NULL) == dust.OK


def test_layer_norm_grad(L):
    bad = dust.ERR_INVALID_ARG
    for kw in (dict(gy=NULL), dict(x=NULL), dict(mean=NULL), dict(rstd=NULL), dict(ld_gy=8),
               dict(ld_x=8), dict(ld_gx=8), dict(flags=dust.CENTER), dict(dt=dust.U32),
               dict(gx=ODD), dict(T=-1)):
        assert _norm_grad(L, **kw) == bad, kw
    for kw in (dict(ws=NULL), dict(wsb=4), dict(ws=C.c_void_p((1 << 20) + 16))):
        assert _norm_grad(L, **kw) == dust.ERR_WORKSPACE, kw
    assert _norm_grad(L, gx=NULL, gw=NULL, gb=NULL) == dust.OK
    assert _norm_grad(L, T=0, gw=NULL, gb=NULL, gy=NULL, x=NULL) == dust.OK
    n = C.c_size_t(0)
    assert L.dust_layer_norm_grad_workspace(None, 4, 4) == bad
    assert L.dust_layer_norm_grad_workspace(C.byref(n), -1, 4) == bad
    assert L.dust_layer_norm_grad_workspace(C.byref(n), 1000, 512) == dust.OK and n.value > 0


@pytest.mark.parametrize("call", [_loss, _grad, _distill, _distill_grad])
def test_head_sizes_and_inputs(L, call):
    bad = dust.ERR_INVALID_ARG
    for kw in (dict(H=NULL), dict(E=NULL), dict(S=0), dict(T=-1), dict(d=0), dict(V=0),
               dict(ld_h=15), dict(ld_e=15), dict(scale=float("nan")), dict(dt=dust.U32),
               dict(lse=NULL), dict(H=ODD), dict(E=ODD)):
        assert call(L, **kw) == bad, kw
    for kw in (dict(T=1 << 31), dict(S=1 << 20, T=1 << 20), dict(V=1 << 31),
               dict(d=1 << 31, ld_h=1 << 31, ld_e=1 << 31), dict(ld_h=1 << 50),
               dict(ld_e=1 << 50)):
        assert call(L, **kw) == dust.ERR_RANGE, kw
    for kw in (dict(ws=NULL), dict(wsb=1), dict(ws=C.c_void_p((1 << 20) + 128))):
        assert call(L, **kw) == dust.ERR_WORKSPACE, kw


def test_head_targets_and_gradients(L):
    bad = dust.ERR_INVALID_ARG
    assert _loss(L, y=NULL) == bad and _grad(L, y=NULL) == bad
    assert _loss(L, T=0, H=NULL, y=NULL, ws=NULL, wsb=0) == dust.OK
    for call in (_distill, _distill_grad):
        assert call(L, ids=NULL) == bad
        assert call(L, z=NULL) == bad
        assert call(L, student=NULL) == bad
        assert call(L, K=0) == bad
        assert call(L, K=dust.MAX_TEACHER + 1) == dust.ERR_RANGE
    for call in (_grad, _distill_grad):
        assert call(L, gloss=NULL) == bad
        assert call(L, flags=dust.CENTER) == bad
        assert call(L, gdt=dust.U32) == bad
        assert call(L, dt=dust.F32, gdt=dust.BF16) == bad
        assert call(L, flags=dust.ACCUMULATE, gdt=dust.BF16) == bad
        assert call(L, ld_gh=15) == bad
        assert call(L, ld_gh=1 << 50) == dust.ERR_RANGE
        assert call(L, gH=ODD) == bad and call(L, gE=ODD) == bad
        assert call(L, gH=NULL, gE=NULL) == dust.OK
        assert call(L, T=0, gE=NULL) == dust.OK
        assert call(L, T=0, flags=dust.ACCUMULATE) == dust.OK


def test_workspace_queries(L):
    n, m = C.c_size_t(0), C.c_size_t(0)
    bad = dust.ERR_INVALID_ARG
    for fn in (L.dust_head_loss_workspace, L.dust_head_loss_grad_workspace):
        assert fn(None, 1, 4, 4, 4, dust.BF16) == bad
        assert fn(C.byref(n), 0, 4, 4, 4, dust.BF16) == bad
        assert fn(C.byref(n), 1, 4, 4, 4, dust.U32) == bad
        assert fn(C.byref(n), 1, 1 << 31, 4, 4, dust.BF16) == dust.ERR_RANGE
        assert fn(C.byref(n), 1, 2048, 512, 4096, dust.BF16) == dust.OK and n.value > 0
        # without the logits: far below rows times vocabulary for a large one
        assert fn(C.byref(m), 1, 8192, 512, 1 << 20, dust.BF16) == dust.OK
        assert m.value < 8192 * (1 << 20)
    for fn in (L.dust_distill_loss_workspace, L.dust_distill_loss_grad_workspace):
        assert fn(C.byref(n), 1, 4, 4, 4, 0, dust.BF16) == bad
        assert fn(C.byref(n), 1, 4, 4, 4, 4096, dust.BF16) == dust.ERR_RANGE
        assert fn(C.byref(n), 1, 4, 4, 4, 8, dust.F32) == dust.OK
