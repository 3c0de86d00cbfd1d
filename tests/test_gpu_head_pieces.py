"""Gradients whose vocabulary is taken in several pieces (a piece's G has at
most 2^28 values over its planes), and rows in more than one group of 38 row
tiles: gH's sums run on from piece to piece, gE's rows, the targets and the
teacher's entries start anew in each, and the last piece is shorter. Compared
with the formulas in 64 bits on the GPU, in blocks of 256 rows and of 256 ids,
so that a wrong block shows beside the others.

Tolerances, before the first run: fp32 normwise 2e-5 (an exponential of a
logit off by 1e-5); bf16 5e-3 (G, and gH, rounded to bf16: 2^-9 each, half of
that on average).
"""
import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda

pytestmark = pytest.mark.gpu

TOL = {"f32": 2e-5, "bf16": 5e-3}

# S, T, d, V, dtype. Rows up to 256, ids up to 256, and planes make a piece:
# 2100 fp32 rows 151 tiles of ids at most, 16384 bf16 rows 64, 10000 bf16 102.
SIZES = [(1, 2100, 32, 40000, "f32"), (3, 701, 24, 39001, "f32"),
         (1, 16384, 16, 20000, "bf16"), (1, 10000, 72, 30011, "bf16")]


def _inputs(S, T, d, V, dtype, dev):
    import torch
    g = torch.Generator().manual_seed(S + T + d + V)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    H = torch.randn((S, T, d), generator=g).to(dt).to(dev)
    E = (torch.randn((V, d), generator=g) * (2.0 / d ** 0.5)).to(dt).to(dev)
    gl = 0.5 + torch.rand((S, T), generator=g)
    gl[:, 5::11] = 0.0
    # Ids about every 256th: pieces end on some of these.
    edge = 256 * torch.randint(0, V // 256 + 1, (T,), generator=g)
    near = edge + torch.randint(-2, 2, (T,), generator=g)
    y = torch.where(torch.rand(T, generator=g) < 0.5, near,
                    torch.randint(0, V, (T,), generator=g)).clamp(0, V - 1)
    y[::9] = -1
    return (H if S > 1 else H[0]), E, y.to(torch.int32).to(dev), (gl if S > 1 else gl[0]).to(dev)


def _compare(H, E, scale, gl, wanted, gH, gE, tol):
    """wanted(rows): the rows' probabilities to be subtracted, [rows, V] in 64
    bits, and whether each row takes part."""
    import torch
    f = torch.float64
    d, V = H.shape[-1], E.shape[0]
    Hd, Ed = H.reshape(-1, d).to(f), E.to(f)
    R = Hd.shape[0]
    w = gl.reshape(-1).to(f)
    got = gH.reshape(-1, d).to(f)
    wE = torch.zeros((V, d), dtype=f, device=E.device)
    step = max(256, (1 << 27) // V // 256 * 256)
    worst = 0.0
    for r0 in range(0, R, step):
        r = torch.arange(r0, min(R, r0 + step), device=E.device)
        G = torch.softmax(scale * Hd[r] @ Ed.t(), 1)
        q, part = wanted(r)
        G = (G * part[:, None] - q) * (scale * w[r])[:, None]
        wH = G @ Ed
        wE += G.t() @ Hd[r]
        for b in range(0, len(r), 256):
            o, n = got[r][b:b + 256] - wH[b:b + 256], wH[b:b + 256].norm()
            worst = max(worst, (o.norm() / n).item())
    assert worst <= tol, worst
    for b in range(0, V, 256):
        off = (gE[b:b + 256].to(f) - wE[b:b + 256]).norm() / wE[b:b + 256].norm()
        worst = max(worst, off.item())
    assert worst <= tol, worst
    return wE


@pytest.mark.parametrize("S,T,d,V,dtype", SIZES)
def test_cross_entropy_in_pieces(S, T, d, V, dtype):
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(S, T, d, V, dtype, dev)
    scale = 1.25
    loss, lse, *rest = dust.dust_head_loss(H, E, y, scale, changes=S > 1)
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl, scale)
    yl = y.long()

    def wanted(r):
        t = r % T
        q = torch.zeros((len(r), V), dtype=torch.float64, device=dev)
        have = yl[t] >= 0
        q[torch.nonzero(have)[:, 0], yl[t][have]] = 1.0
        return q, have.double()

    wE = _compare(H, E, scale, gl, wanted, gH, gE, TOL[dtype])
    assert (gH.reshape(S, T, d)[:, (y < 0).to(dev)] == 0).all()
    # Added to what is there, the same bits as alone but for the addition.
    into = torch.full_like(gE, 0.25)
    dust.dust_head_loss_grad(H, E, y, lse, gl, scale, flags=dust.ACCUMULATE, gE=into)
    assert torch.equal(into, gE + 0.25)
    if dtype == "bf16":
        _, short = dust.dust_head_loss_grad(H, E, y, lse, gl, scale, gE_dtype=torch.bfloat16)
        assert (short.double() - wE).norm() <= TOL[dtype] * wE.norm()


@pytest.mark.parametrize("K", [3, 300])
@pytest.mark.parametrize("S,T,d,V,dtype", SIZES)
def test_distillation_in_pieces(S, T, d, V, dtype, K):
    import torch
    dev = cuda()
    H, E, y, gl = _inputs(S, T, d, V, dtype, dev)
    g = torch.Generator().manual_seed(K)
    ids = torch.randint(0, V, (T, K), generator=g)
    # Runs of neighbouring ids about the ends of tiles in some rows.
    ids[::2] = (256 * torch.randint(0, V // 256 + 1, (T, 1), generator=g)[::2]
                + torch.arange(K) - K // 2).clamp(0, V - 1)
    ids[torch.rand((T, K), generator=g) < 0.1] = -1
    ids[7::13] = -1
    ids = ids.to(torch.int32).to(dev)
    z = torch.randn((T, K), generator=g).to(dev)
    scale = 0.75
    loss, lse, student = dust.dust_distill_loss(H, E, ids, z, scale)
    gH, gE = dust.dust_distill_loss_grad(H, E, ids, z, lse, student, gl, scale)
    have = ids >= 0
    q = torch.softmax((scale * z.double()).masked_fill(~have, -1e300), 1) * have
    part = have.any(1)

    def wanted(r):
        t = r % T
        out = torch.zeros((len(r), V), dtype=torch.float64, device=dev)
        out.scatter_add_(1, ids[t].long().clamp(min=0), q[t] * part[t, None])
        return out, part[t].double()

    _compare(H, E, scale, gl, wanted, gH, gE, TOL[dtype])
    assert (gH.reshape(S, T, d)[:, ~part] == 0).all()


def test_one_gradient_in_pieces():
    """gH alone and gE alone: the bits of the call for both."""
    import ctypes as C
    import torch
    dev = cuda()
    S, T, d, V, dtype = SIZES[0]
    H, E, y, gl = _inputs(S, T, d, V, dtype, dev)
    _, lse = dust.dust_head_loss(H, E, y)
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, gl)
    L, n = dust.lib(), C.c_size_t(0)
    assert L.dust_head_loss_grad_workspace(C.byref(n), S, T, d, V, dust.F32) == dust.OK
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    s = torch.cuda.current_stream().cuda_stream
    for which in range(2):
        h, e = torch.full_like(gH, 7.0), torch.full_like(gE, 7.0)
        st = L.dust_head_loss_grad(
            H.data_ptr(), d, E.data_ptr(), d, dust.F32, S, T, d, V, y.data_ptr(), 1.0,
            lse.data_ptr(), gl.data_ptr(), 0, h.data_ptr() if which == 0 else None, d,
            e.data_ptr() if which == 1 else None, dust.F32, ws.data_ptr(), n.value, s)
        assert st == dust.OK
        assert torch.equal(h, gH) if which == 0 else (h == 7.0).all()
        assert torch.equal(e, gE) if which == 1 else (e == 7.0).all()
