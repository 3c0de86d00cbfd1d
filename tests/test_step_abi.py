"""Host-side refusals of the gated block, the queries' and keys' norms and
rotation, the policy loss and the gradient clipping: every call here fails
validation (or has nothing to do), so nothing is enqueued. Runs only where
there is no GPU: the addresses are made up."""
import ctypes as C

import pytest

import token_perturbation_estimator_gb300 as dust

NULL = C.c_void_p(0)
FAKE = C.c_void_p(1 << 20)
ODD = C.c_void_p((1 << 20) + 1)
NAN, INF = float("nan"), float("inf")


def _has_gpu():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


class Grad(C.Structure):
    """dust_grad of include/dust.h."""
    _fields_ = [("g", C.c_void_p), ("out", C.c_void_p), ("n", C.c_int64), ("dtype", C.c_int32)]


pytestmark = pytest.mark.skipif(_has_gpu(), reason="fake device addresses: CPU only")


@pytest.fixture(scope="module")
def L():
    from token_perturbation_estimator_gb300 import build
    build.build()
    return dust.lib()


def _call(fn, defaults, kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


def _up(L, **kw):
    return _call(L.dust_gated_up, dict(
        X=FAKE, ld_x=16, Wg=FAKE, ld_wg=16, Wu=FAKE, ld_wu=16, dt=dust.BF16, T=4, d=16, f=32,
        act=dust.SILU, h=FAKE, ld_h=32, ws=FAKE, wsb=1 << 40, stream=NULL), kw)


def _up_grad(L, **kw):
    return _call(L.dust_gated_up_grad, dict(
        gh=FAKE, ld_gh=32, X=FAKE, ld_x=16, Wg=FAKE, ld_wg=16, Wu=FAKE, ld_wu=16, dt=dust.BF16, T=4,
        d=16, f=32, act=dust.SILU, flags=0, gX=FAKE, ld_gx=16, gWg=FAKE, gWu=FAKE, gdt=dust.F32,
        ws=FAKE, wsb=1 << 40, stream=NULL), kw)


@pytest.mark.parametrize("call", [_up, _up_grad])
def test_gated(L, call):
    bad = dust.ERR_INVALID_ARG
    for kw in (dict(X=NULL), dict(Wg=NULL), dict(Wu=NULL), dict(X=ODD), dict(Wg=ODD), dict(Wu=ODD),
               dict(ld_x=15), dict(ld_wg=15), dict(ld_wu=15), dict(T=-1), dict(d=0), dict(f=0),
               dict(dt=dust.U32), dict(dt=7), dict(act=3), dict(act=-1)):
        assert call(L, **kw) == bad, kw
    big = 1 << 31
    for kw in (dict(T=big), dict(d=big, ld_x=big, ld_wg=big, ld_wu=big), dict(ld_x=1 << 50),
               dict(ld_wg=1 << 50), dict(ld_wu=1 << 50),
               dict(T=1 << 30, d=1 << 10, ld_x=1 << 10, ld_wg=1 << 10, ld_wu=1 << 10)):
        assert call(L, **kw) == dust.ERR_RANGE, kw


def test_gated_outputs(L):
    bad = dust.ERR_INVALID_ARG
    for kw in (dict(h=NULL), dict(h=ODD), dict(ld_h=31)):
        assert _up(L, **kw) == bad, kw
    assert _up(L, ld_h=1 << 50) == dust.ERR_RANGE
    assert _up(L, T=0, X=NULL, h=NULL) == dust.OK
    for kw in (dict(gh=NULL), dict(gh=ODD), dict(ld_gh=31), dict(gX=ODD), dict(ld_gx=15),
               dict(gWg=ODD), dict(gWu=ODD), dict(gdt=dust.U32), dict(flags=dust.CENTER),
               dict(dt=dust.F32, gdt=dust.BF16), dict(gdt=dust.BF16, flags=dust.ACCUMULATE)):
        assert _up_grad(L, **kw) == bad, kw
    for kw in (dict(ld_gh=1 << 50), dict(ld_gx=1 << 50)):
        assert _up_grad(L, **kw) == dust.ERR_RANGE, kw
    for kw in (dict(ws=NULL), dict(wsb=1), dict(ws=C.c_void_p((1 << 20) + 128))):
        assert _up_grad(L, **kw) == dust.ERR_WORKSPACE, kw
    assert _up_grad(L, gX=NULL, gWg=NULL, gWu=NULL) == dust.OK
    assert _up_grad(L, T=0, flags=dust.ACCUMULATE) == dust.OK


def test_gated_workspaces(L):
    n = C.c_size_t(0)
    for q in (L.dust_gated_up_workspace, L.dust_gated_up_grad_workspace):
        assert q(None, 4, 16, 32, dust.BF16) == dust.ERR_INVALID_ARG
        assert q(C.byref(n), -1, 16, 32, dust.BF16) == dust.ERR_INVALID_ARG
        assert q(C.byref(n), 4, 16, 32, 5) == dust.ERR_INVALID_ARG
        assert q(C.byref(n), 1 << 31, 16, 32, dust.BF16) == dust.ERR_RANGE
        assert q(C.byref(n), 1 << 20, 1 << 20, 32, dust.BF16) == dust.ERR_RANGE
        for size in ((0, 1, 1), (1, 512, 2048), (65536, 512, 2048), (777, 301, 1003)):
            for dt in (dust.BF16, dust.F32):
                assert q(C.byref(n), *size, dt) == dust.OK


def _h(data=1 << 20, token=64, head=16):
    return C.byref(dust._Heads(data, token, head))


def _rope(L, **kw):
    return _call(L.dust_qk_norm_rope, dict(
        q=_h(), hq=4, k=_h(), hk=4, dt=dust.BF16, T=4, D=16, wq=NULL, wk=NULL, eps=1e-6, pos=FAKE,
        c=FAKE, s=FAKE, n=8, rot=16, layout=0, yq=_h(), yk=_h(), stream=NULL), kw)


def _rope_grad(L, **kw):
    return _call(L.dust_qk_norm_rope_grad, dict(
        gyq=_h(), gyk=_h(), q=_h(), hq=4, k=_h(), hk=4, dt=dust.BF16, T=4, D=16, wq=NULL, wk=NULL,
        eps=1e-6, pos=FAKE, c=FAKE, s=FAKE, n=8, rot=16, layout=0, flags=0, yq=_h(), yk=_h(),
        gwq=FAKE, gwk=FAKE, ws=FAKE, wsb=1 << 30, stream=NULL), kw)


@pytest.mark.parametrize("call", [_rope, _rope_grad])
def test_rope(L, call):
    bad = dust.ERR_INVALID_ARG
    for kw in (dict(q=None), dict(k=None), dict(yq=None), dict(yk=None), dict(q=_h(data=0)),
               dict(q=_h(data=(1 << 20) + 1)), dict(hq=-1), dict(hk=-1), dict(T=-1), dict(D=0),
               dict(dt=dust.U32), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(pos=NULL),
               dict(c=NULL), dict(s=NULL), dict(n=-1), dict(rot=15), dict(rot=18), dict(rot=-2),
               dict(layout=2), dict(q=_h(token=15)), dict(q=_h(token=63)), dict(q=_h(head=15)),
               dict(q=_h(token=16, head=63)), dict(yk=_h(token=0)), dict(k=_h(token=-64))):
        assert call(L, **kw) == bad, kw
    for kw in (dict(D=513, q=_h(token=9999, head=600)), dict(T=1 << 31), dict(hq=1 << 31),
               dict(hq=1 << 30, hk=1 << 30, T=1 << 20), dict(q=_h(token=1 << 50)),
               dict(n=1 << 62)):
        assert call(L, **kw) == dust.ERR_RANGE, kw
    if call is _rope:
        assert call(L, T=0, q=None, k=None) == dust.OK
        assert call(L, hq=0, hk=0, q=None, k=None, yq=None, yk=None) == dust.OK
    else:
        for kw in (dict(gyq=None), dict(gyk=_h(token=1)), dict(flags=dust.CENTER)):
            assert call(L, **kw) == bad, kw
        for kw in (dict(ws=NULL), dict(wsb=8), dict(ws=C.c_void_p((1 << 20) + 16))):
            assert call(L, **kw) == dust.ERR_WORKSPACE, kw
        assert call(L, T=0, flags=dust.ACCUMULATE) == dust.OK
        assert call(L, T=0, gwq=NULL, gwk=NULL) == dust.OK
    n = C.c_size_t(0)
    q = L.dust_qk_norm_rope_grad_workspace
    assert q(None, 4, 4, 4, 16) == bad and q(C.byref(n), 4, 4, 4, 0) == bad
    assert q(C.byref(n), 4, 4, 4, 513) == dust.ERR_RANGE
    assert q(C.byref(n), 4, 4, 4, 64) == dust.OK and n.value > 0


def _policy(L, **kw):
    return _call(L.dust_policy_loss, dict(
        nll=FAKE, old=FAKE, ref=FAKE, adv=FAKE, per_token=0, off=FAKE, n_seq=2, tg=FAKE, S=2, T=8,
        low=0.2, high=0.2, beta=0.1, mean=0, loss=FAKE, total=FAKE, kl=FAKE, clipped=FAKE, delta=FAKE,
        ws=FAKE, wsb=1 << 30, stream=NULL), kw)


def _policy_grad(L, **kw):
    return _call(L.dust_policy_loss_grad, dict(
        nll=FAKE, old=FAKE, ref=FAKE, adv=FAKE, per_token=0, off=FAKE, n_seq=2, tg=FAKE, S=2, T=8,
        low=0.2, high=0.2, beta=0.1, mean=0, gtotal=FAKE, gnll=FAKE, ws=FAKE, wsb=1 << 30,
        stream=NULL), kw)


@pytest.mark.parametrize("call", [_policy, _policy_grad])
def test_policy(L, call):
    bad = dust.ERR_INVALID_ARG
    for kw in (dict(nll=NULL), dict(old=NULL), dict(adv=NULL), dict(off=NULL), dict(S=0), dict(T=-1),
               dict(n_seq=-1), dict(low=-0.1), dict(low=1.1), dict(low=NAN), dict(high=-0.1),
               dict(high=NAN), dict(beta=NAN), dict(beta=INF), dict(mean=2),
               dict(adv=NULL, n_seq=0, per_token=1)):
        assert call(L, **kw) == bad, kw
    for kw in (dict(T=1 << 31), dict(S=1 << 16, T=1 << 16), dict(n_seq=1 << 31)):
        assert call(L, **kw) == dust.ERR_RANGE, kw
    for kw in (dict(ws=NULL), dict(wsb=8), dict(ws=C.c_void_p((1 << 20) + 16))):
        # (few tokens need none)
        assert call(L, T=100000, **kw) == dust.ERR_WORKSPACE, kw
    if call is _policy:
        assert call(L, T=0, total=NULL, kl=NULL, clipped=NULL, nll=NULL, off=NULL) == dust.OK
    else:
        assert call(L, gtotal=NULL) == bad and call(L, gnll=NULL) == bad
        assert call(L, T=0, nll=NULL) == dust.OK
    n = C.c_size_t(0)
    assert L.dust_policy_loss_workspace(None, 1, 4, 1) == bad
    assert L.dust_policy_loss_workspace(C.byref(n), 0, 4, 1) == bad
    assert L.dust_policy_loss_workspace(C.byref(n), 1, 0, 0) == dust.OK


def _clip(L, tensors, n=None, max_norm=1.0, norm=FAKE, ws=FAKE, wsb=1 << 20):
    arr = (Grad * max(1, len(tensors)))()
    for a, (g, o, m, dt) in zip(arr, tensors):
        a.g, a.out, a.n, a.dtype = g, o, m, dt
    return L.dust_clip_grads(C.addressof(arr), len(tensors) if n is None else n, max_norm, norm, ws, wsb,
                             NULL)


def test_clip(L):
    bad, f, b = dust.ERR_INVALID_ARG, dust.F32, dust.BF16
    fine = (1 << 20, 1 << 20, 100, f)
    for tensors in ([(0, 1 << 20, 5, f)], [(1 << 20, 1 << 21, -1, f)], [(1 << 20, 1 << 21, 5, 2)],
                    [((1 << 20) + 2, 1 << 21, 5, f)], [(1 << 20, (1 << 21) + 1, 5, b)],
                    [fine, (1 << 22, 0, 5, f)],                      # an output missing
                    [fine, fine],                                    # twice in place
                    [fine, ((1 << 20) + 396, (1 << 20) + 396, 9, f)],  # the last value shared
                    [(1 << 20, (1 << 20) + 4, 100, f)],              # onto itself, moved
                    [(1 << 20, 1 << 21, 100, f), ((1 << 21) + 8, 1 << 22, 9, f)],
                    [(1 << 20, 1 << 21, 100, f), (1 << 22, (1 << 21) + 396, 9, b)]):
        assert _clip(L, tensors) == bad, tensors
    assert _clip(L, [fine], max_norm=-1.0) == bad and _clip(L, [fine], max_norm=NAN) == bad
    assert _clip(L, [fine], norm=NULL) == bad and _clip(L, [fine], n=-1) == bad
    assert _clip(L, [fine], n=4097) == dust.ERR_RANGE
    assert _clip(L, [(1 << 20, 1 << 20, (1 << 40) + 1, f)]) == dust.ERR_RANGE
    for kw in (dict(ws=NULL), dict(wsb=8), dict(ws=C.c_void_p((1 << 20) + 16))):
        assert _clip(L, [fine], **kw) == dust.ERR_WORKSPACE, kw
    assert L.dust_clip_grads(NULL, 1, 1.0, FAKE, FAKE, 1 << 20, NULL) == bad
    n = C.c_size_t(0)
    assert L.dust_clip_grads_workspace(None, 1) == bad
    assert L.dust_clip_grads_workspace(C.byref(n), -1) == bad
    assert L.dust_clip_grads_workspace(C.byref(n), 4097) == dust.ERR_RANGE
    assert L.dust_clip_grads_workspace(C.byref(n), 0) == dust.OK and n.value > 0


def test_binding_refuses_other_tensors():
    import torch
    t = torch.zeros(4, 8)
    for call in (lambda: dust.dust_gated_up(t, t, t), lambda: dust.dust_gated_up_grad(t, t, t, t),
                 lambda: dust.dust_qk_norm_rope(t[:, None], None, None, None, t[:, 0], t, t),
                 lambda: dust.dust_policy_loss(t, t[0], t[0], t[0])):
        with pytest.raises(ValueError):
            call()
