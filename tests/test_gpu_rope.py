"""GPU parity of the queries' and keys' norms with the rotation, and of their
gradients, against the formulas in 64 bits (numpy, on the CPU).

Tolerances. An output value is a few fp32 products (the root's relative error
is that of a sum of D squares, at most (8 + D / 32) 2^-24 in partial sums, and
halved): 2^-24 (16 + D / 32) of the values that are turned into it. bf16: one
rounding more, 2^-8 of the value. The gradients' weights are sums of fp32
terms over tokens and heads: 4e-6 of the sum of magnitudes, as for the layer
norm."""
import numpy as np
import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda

pytestmark = pytest.mark.gpu

LAYOUTS = {"halves": dust.ROPE_HALVES, "pairs": dust.ROPE_PAIRS}


def _np(t):
    return t.double().cpu().numpy()


def _tables(n, rot):
    import torch
    turns = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    angle = np.arange(n)[:, None] * turns[None]
    return (torch.tensor(np.cos(angle), dtype=torch.float32).cuda(),
            torch.tensor(np.sin(angle), dtype=torch.float32).cuda())


def _inputs(T, hq, hk, D, rot, dtype, dev, n_pos=64, pad=0.2, fused=False, seed=0):
    import torch
    g = torch.Generator().manual_seed(11 * T + 5 * D + hq + seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def heads(n, scale=1.0):
        return (torch.randn((T, n, D), generator=g) * scale).to(dt).to(dev)

    if fused:
        row = heads(hq + 2 * hk, 1.7)
        q, k = row[:, :hq], row[:, hq:hq + hk]
    else:
        q, k = heads(hq, 1.7), heads(hk, 0.6)
    wq = (1 + 0.2 * torch.randn(D, generator=g)).to(dev)
    wk = (1 + 0.2 * torch.randn(D, generator=g)).to(dev)
    pos = torch.randint(0, n_pos, (T,), generator=g, dtype=torch.int32)
    pos[torch.rand(T, generator=g) < pad] = -1
    return q, k, wq, wk, pos.to(dev), *_tables(n_pos, rot), heads(hq), heads(hk)


def turn64(m, pos, c, s, rot, layout, sign=1.0, sizes=False):
    """m turned; sizes: the sum of the magnitudes that each value is made of."""
    m = np.abs(m) if sizes else m.copy()
    c, s = (t[np.maximum(pos, 0)][:, None, :rot // 2] for t in (c, sign * s))
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "halves" else (
        slice(0, rot, 2), slice(1, rot, 2))
    x, y = m[..., a].copy(), m[..., b].copy()
    if sizes:
        c, s = np.abs(c), np.abs(s)
        m[..., a], m[..., b] = x * c + y * s, y * c + x * s
    else:
        m[..., a], m[..., b] = x * c - y * s, y * c + x * s
    return m


def reference(x, w, pos, c, s, rot, layout, eps, gy=None):
    x, pos = _np(x), pos.cpu().numpy()
    w = np.ones(x.shape[-1]) if w is None else _np(w)
    c, s = _np(c), _np(s)
    there = (pos >= 0)[:, None, None]
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * rstd
    if gy is None:
        y = turn64(n * w, pos, c, s, rot, layout)
        size = turn64(n * w, pos, c, s, rot, layout, sizes=True)
        return np.where(there, y, 0.0), np.where(there, size, 0.0)
    gm = np.where(there, turn64(_np(gy), pos, c, s, rot, layout, -1.0), 0.0)
    gn = gm * w
    dot = (gn * n).mean(-1, keepdims=True)
    gx = rstd * (gn - n * dot)
    sizes = turn64(_np(gy), pos, c, s, rot, layout, sizes=True)
    size = rstd * (sizes * np.abs(w) + np.abs(n) * (sizes * np.abs(w * n)).mean(-1, keepdims=True))
    return (np.where(there, gx, 0.0), np.where(there, size, 0.0), (gm * n).sum((0, 1)),
            np.where(there, sizes * np.abs(n), 0.0).sum((0, 1)))


def check(got, want, size, D, dtype):
    e = 2.0 ** -24 * (16 + D / 32) * size + 1e-37
    if dtype == "bf16":
        e = e + 2.0 ** -8 * (np.abs(want) + e)
    assert (np.abs(_np(got) - want) <= e).all()


SIZES = [(1, 8, 8, 64, 64), (1, 1, 0, 1, 0), (3, 2, 1, 2, 2), (5, 3, 1, 7, 6), (17, 4, 2, 32, 32),
         (33, 6, 3, 74, 36), (9, 5, 5, 80, 80), (9, 5, 5, 80, 40), (20, 8, 1, 128, 128),
         (64, 8, 4, 128, 64), (7, 32, 8, 96, 96), (13, 3, 3, 256, 256), (5, 2, 2, 512, 512),
         (6, 2, 1, 511, 100), (4, 1, 1, 513 - 2, 510), (40, 16, 2, 48, 24), (300, 2, 2, 16, 8),
         (11, 7, 3, 100, 0), (1000, 4, 4, 64, 64), (2, 40, 40, 12, 12), (50, 9, 3, 36, 20)]


# Sizes of every width of vectors and lanes, and so many tokens that warps take
# several, the last time fewer than they can. A warp's sums over its tokens (up to
# 16), a CTA's over 8 warps and the rows' (10 and 5 halvings) are below 40
# roundings: 40 * 2^-24 < 4e-6.
LONG = [(9001, 1, 1, 9, 4), (9001, 2, 2, 13, 12), (12000, 1, 1, 45, 44), (7000, 2, 1, 90, 90),
        (5000, 2, 1, 201, 200), (2500, 2, 1, 301, 300), (9001, 2, 1, 26, 26), (8000, 1, 1, 58, 20),
        (7000, 2, 1, 110, 110), (4000, 2, 2, 202, 200), (2500, 2, 1, 330, 64), (9001, 3, 1, 24, 8),
        (8000, 1, 1, 56, 24), (7000, 2, 1, 120, 120), (2500, 1, 1, 328, 200), (6000, 2, 1, 104, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("T,hq,hk,D,rot", SIZES + LONG)
def test_forward_and_gradients(T, hq, hk, D, rot, layout, dtype):
    dev = cuda()
    for fused in (False, True):
        q, k, wq, wk, pos, c, s, gyq, gyk = _inputs(T, hq, hk, D, rot, dtype, dev, fused=fused)
        eps = 1e-6
        yq, yk = dust.dust_qk_norm_rope(q, k, wq, wk, pos, c, s, eps, LAYOUTS[layout])
        for y, x, w in ((yq, q, wq), (yk, k, wk)):
            assert y.dtype == x.dtype and y.shape == x.shape
            check(y, *reference(x, w, pos, c, s, rot, layout, eps), D, dtype)
        gq, gk, gwq, gwk = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s, eps,
                                                       LAYOUTS[layout])
        for gx, gw, gy, x, w in ((gq, gwq, gyq, q, wq), (gk, gwk, gyk, k, wk)):
            want, size, gw64, gw_size = reference(x, w, pos, c, s, rot, layout, eps, gy)
            check(gx, want, size, 2 * D, dtype)
            assert (np.abs(_np(gw) - gw64) <= 4e-6 * gw_size + 1e-37).all()
        again = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s, eps, LAYOUTS[layout])
        assert all((a == b).all() for a, b in zip(again, (gq, gk, gwq, gwk)))
    assert dust.dust_last_error() == dust.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_and_without_weights_or_keys(dtype):
    import torch
    dev = cuda()
    T, hq, hk, D, rot = 50, 4, 2, 64, 64
    q, k, wq, wk, pos, c, s, gyq, gyk = _inputs(T, hq, hk, D, rot, dtype, dev, fused=True)
    yq, yk = dust.dust_qk_norm_rope(q, k, None, wk, pos, c, s)
    check(yq, *reference(q, None, pos, c, s, rot, "halves", 1e-6), D, dtype)
    only, none = dust.dust_qk_norm_rope(q, None, None, None, pos, c, s)
    assert none is None and (only == yq).all()
    plain, _ = dust.dust_qk_norm_rope(q, None, None, None, pos, None, None)
    check(plain, *reference(q, None, pos, c, s, 0, "halves", 1e-6), D, dtype)
    gq, gk, gwq, gwk = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, None, wk, pos, c, s)
    g1, g2, w1, w2 = dust.dust_qk_norm_rope_grad(gyq, None, q, None, None, None, pos, c, s)
    assert (g1 == gq).all() and g2 is None and w2 is None
    # The order of a weight's sum goes by the number of heads: each of the two is
    # within 4e-6 of the sum of magnitudes, as above.
    _, _, gw64, gw_size = reference(q, None, pos, c, s, rot, "halves", 1e-6, gyq)
    for w in (w1, gwq):
        assert (np.abs(_np(w) - gw64) <= 4e-6 * gw_size + 1e-37).all()
    a, b = gyq.clone(), gyk.clone()
    dust.dust_qk_norm_rope_grad(a, b, q, k, None, wk, pos, c, s, gq=a, gk=b)
    assert (a == gq).all() and (b == gk).all()
    row = torch.cat([q, k], 1).contiguous()
    dust.dust_qk_norm_rope(row[:, :hq], row[:, hq:], None, wk, pos, c, s, yq=row[:, :hq],
                           yk=row[:, hq:])
    assert (row[:, :hq] == yq).all() and (row[:, hq:] == yk).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("room", [1, 2, 4, 8])
def test_strides_and_alignment(room, dtype):
    """Heads with room between them, heads outside of tokens, rows off 16 bytes."""
    import torch
    dev = cuda()
    T, hq, hk, D, rot = 21, 3, 2, 64, 32
    q, k, wq, wk, pos, c, s, gyq, gyk = _inputs(T, hq, hk, D, rot, dtype, dev)
    want = dust.dust_qk_norm_rope(q, k, wq, wk, pos, c, s)
    wanted = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s)

    def spread(t):
        big = torch.full((t.shape[0], t.shape[1], D + room), 9.0, dtype=t.dtype, device=dev)
        big[..., :D] = t
        return big

    def outside(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    def off(t):
        flat = torch.empty(t.numel() + room, dtype=t.dtype, device=dev)
        view = flat[room:].view(t.shape)
        view.copy_(t)
        return view

    tol = 2.0 ** -7 if dtype == "bf16" else 1e-5  # other orders of summation, one rounding each
    for how in (lambda t: spread(t)[..., :D], outside, off):
        out = [how(torch.zeros_like(t)) for t in (q, k)]
        got = dust.dust_qk_norm_rope(how(q), how(k), wq, wk, pos, c, s, yq=out[0], yk=out[1])
        for a, b in zip(got, want):
            assert (a.float() - b.float()).abs().max() <= tol * b.float().abs().max()
        got = dust.dust_qk_norm_rope_grad(how(gyq), how(gyk), how(q), how(k), wq, wk, pos, c, s,
                                          gq=out[0], gk=out[1])
        for a, b in zip(got, wanted):
            assert (a.float() - b.float()).abs().max() <= tol * b.float().abs().max()
    big = spread(torch.zeros_like(q))
    dust.dust_qk_norm_rope(q, None, wq, None, pos, c, s, yq=big[..., :D])
    assert (big[..., D:] == 9.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk,D", [(0, 3, 64), (0, 1, 32), (5, 0, 64), (0, 2, 30), (13, 7, 16)])
def test_one_side_alone_and_odd_numbers_of_heads(hq, hk, D, dtype):
    import torch
    dev = cuda()
    T = 70
    q, k, wq, wk, pos, c, s, gyq, gyk = _inputs(T, max(hq, 1), max(hk, 1), D, D, dtype, dev)
    q, gyq, k, gyk = q[:, :hq], gyq[:, :hq], k[:, :hk], gyk[:, :hk]
    yq, yk = dust.dust_qk_norm_rope(q, k, wq, wk, pos, c, s)
    gq, gk, gwq, gwk = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s)
    for y, gx, gw, gy, x, w in ((yq, gq, gwq, gyq, q, wq), (yk, gk, gwk, gyk, k, wk)):
        if x.numel() == 0:
            assert y.numel() == 0 and (gw == 0).all()
            continue
        check(y, *reference(x, w, pos, c, s, D, "halves", 1e-6), D, dtype)
        want, size, gw64, gw_size = reference(x, w, pos, c, s, D, "halves", 1e-6, gy)
        check(gx, want, size, 2 * D, dtype)
        assert (np.abs(_np(gw) - gw64) <= 4e-6 * gw_size + 1e-37).all()


def test_padded_tokens_hide_what_they_hold():
    import torch
    dev = cuda()
    T, hq, hk, D, rot = 40, 4, 2, 64, 64
    q, k, wq, wk, pos, c, s, gyq, gyk = _inputs(T, hq, hk, D, rot, "bf16", dev)
    pos[5], pos[6], pos[39] = -1, -7, -1
    clean = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s)
    for t in (5, 6, 39):
        q[t], k[t], gyq[t], gyk[t] = float("nan"), float("inf"), float("inf"), float("nan")
    yq, yk = dust.dust_qk_norm_rope(q, k, wq, wk, pos, c, s)
    for t in (5, 6, 39):
        assert (yq[t] == 0).all() and (yk[t] == 0).all()
    grads = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s)
    assert all((a == b).all() for a, b in zip(grads, clean))
    pos.fill_(-1)
    gq, gk, gwq, gwk = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s)
    assert (gq == 0).all() and (gk == 0).all() and (gwq == 0).all() and (gwk == 0).all()
    assert dust.dust_last_error() == dust.OK
    pos[3] = c.shape[0]  # past the tables
    pos[4] = 2
    yq, _ = dust.dust_qk_norm_rope(q, k, wq, wk, pos, c, s)
    assert (yq[3] == 0).all() and yq[4].isfinite().all()
    assert dust.dust_last_error() == dust.ERR_INVALID_ARG
    assert dust.dust_last_error() == dust.OK


@pytest.mark.parametrize("D", [64, 30])
def test_tables_without_a_position(D):
    """No rows in the tables: every token that is no padding is past them."""
    import torch
    dev = cuda()
    q, k, wq, wk, pos, c, s, gyq, gyk = _inputs(9, 2, 1, D, D, "f32", dev)
    c, s = c[:0], s[:0]
    yq, yk = dust.dust_qk_norm_rope(q, k, wq, wk, pos, c, s)
    grads = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s)
    assert (yq == 0).all() and (yk == 0).all() and all((g == 0).all() for g in grads)
    assert dust.dust_last_error() == dust.ERR_INVALID_ARG


def test_accumulates_and_no_tokens():
    import torch
    dev = cuda()
    q, k, wq, wk, pos, c, s, gyq, gyk = _inputs(33, 4, 2, 48, 48, "f32", dev)
    _, _, gwq, gwk = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s)
    a, b = torch.full_like(gwq, 2.0), torch.full_like(gwk, -3.0)
    dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s, flags=dust.ACCUMULATE, gwq=a,
                                gwk=b)
    assert torch.allclose(a, gwq + 2.0, rtol=1e-6, atol=1e-6)
    assert torch.allclose(b, gwk - 3.0, rtol=1e-6, atol=1e-6)
    none = [t[:0] for t in (gyq, gyk, q, k)]
    gq, gk, w1, w2 = dust.dust_qk_norm_rope_grad(*none, wq, wk, pos[:0], c, s)
    assert gq.numel() == 0 and (w1 == 0).all() and (w2 == 0).all()
    dust.dust_qk_norm_rope_grad(*none, wq, wk, pos[:0], c, s, flags=dust.ACCUMULATE, gwq=a, gwk=b)
    assert torch.allclose(a, gwq + 2.0, rtol=1e-6, atol=1e-6)


def test_gradients_against_differences():
    """Central differences along random directions, fp32, as for the gated block."""
    import torch
    dev = cuda()
    for layout in LAYOUTS:
        q, k, wq, wk, pos, c, s, gyq, gyk = _inputs(19, 3, 2, 40, 24, "f32", dev)
        grads = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s,
                                            layout=LAYOUTS[layout])
        g = torch.Generator().manual_seed(5)
        dirs = [torch.randn(t.shape, generator=g).to(dev) for t in (q, k, wq, wk)]

        def value(e):
            at = [t + e * u for t, u in zip((q, k, wq, wk), dirs)]
            yq, yk = dust.dust_qk_norm_rope(*at, pos, c, s, layout=LAYOUTS[layout])
            return ((yq.double() * gyq.double()).sum() + (yk.double() * gyk.double()).sum()).item()

        e = 2.0 ** -8
        slope = (value(e) - value(-e)) / (2 * e)
        terms = [(a.double() * b.double()) for a, b in zip(grads, dirs)]
        assert abs(slope - sum(t.sum().item() for t in terms)) <= \
            2e-3 * sum(t.norm().item() for t in terms)


def test_on_another_stream_and_in_a_graph():
    import torch
    dev = cuda()
    q, k, wq, wk, pos, c, s, gyq, gyk = _inputs(100, 4, 2, 64, 64, "bf16", dev)
    want = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert all((a == b).all() for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = dust.dust_qk_norm_rope(q, k, wq, wk, pos, c, s)
        gs = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s)
    q.mul_(-0.5)
    graph.replay()
    for a, b in zip(ys, dust.dust_qk_norm_rope(q, k, wq, wk, pos, c, s)):
        assert (a == b).all()
    for a, b in zip(gs, dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, c, s)):
        assert (a == b).all()


def test_offsets_past_32_bits():
    """A strided operand whose last token lies beyond 2^31 elements."""
    import torch
    dev = cuda()
    T, D = 3, 64
    stride = (1 << 30) + 8
    big = torch.empty((T - 1) * stride + 2 * D, dtype=torch.bfloat16, device=dev)
    q = big.as_strided((T, 2, D), (stride, D, 1))
    src = torch.randn((T, 2, D), device=dev).to(torch.bfloat16)
    q.copy_(src)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    c, s = _tables(8, D)
    want, _ = dust.dust_qk_norm_rope(src, None, None, None, pos, c, s)
    got, _ = dust.dust_qk_norm_rope(q, None, None, None, pos, c, s)
    assert (got == want).all()
    dust.dust_qk_norm_rope(src, None, None, None, pos, c, s, yq=q)
    assert (q == want).all()


def test_any_position_without_tables():
    """Where nothing turns, the largest position is one like any other."""
    import torch
    dev = cuda()
    for dtype in ("bf16", "f32"):
        q, k, wq, wk, pos, c, s, gyq, gyk = _inputs(5, 3, 2, 32, 0, dtype, dev, pad=0.0)
        want = dust.dust_qk_norm_rope(q, k, wq, wk, pos, None, None)
        wanted = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, pos, None, None)
        far = torch.full_like(pos, 2 ** 31 - 1)
        for a, b in zip(dust.dust_qk_norm_rope(q, k, wq, wk, far, None, None), want):
            assert torch.equal(a, b)
        for a, b in zip(dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, far, None, None), wanted):
            assert torch.equal(a, b)
        far[1] = -1
        assert (dust.dust_qk_norm_rope(q, k, wq, wk, far, None, None)[0][1] == 0).all()
    assert dust.dust_last_error() == dust.OK
