"""GPU parity of the gradient norm and the clipping against 64 bits (numpy).

Tolerances. The norm's squares are summed 16 at a time in fp32 (at most 5
roundings of 2^-24 each, halved by the root), then in 64 bits, and the result is
rounded once: 4 x 2^-24. A scaled value has that of the factor and one rounding
of its own: 2^-24 x 2, bf16 2^-8 more."""
import ctypes as C

import numpy as np
import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda

class Grad(C.Structure):
    """dust_grad of include/dust.h."""
    _fields_ = [("g", C.c_void_p), ("out", C.c_void_p), ("n", C.c_int64), ("dtype", C.c_int32)]


pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


def _tensors(shapes, dtypes, dev, scale=1.0, seed=0):
    import torch
    g = torch.Generator().manual_seed(len(shapes) + seed)
    kinds = {"bf16": torch.bfloat16, "f32": torch.float32}
    return [(torch.randn(s, generator=g) * scale * (1 + i % 5)).to(kinds[dtypes[i % len(dtypes)]]).to(dev)
            for i, s in enumerate(shapes)]


def check(grads, max_norm, in_place=False):
    import torch
    want = [_np(t) for t in grads]
    norm64 = np.sqrt(sum((t * t).sum() for t in want))
    c = min(1.0, max_norm / norm64) if norm64 > 0 else 1.0
    out = None if in_place else [torch.full_like(t, 9.0) for t in grads]
    norm, got = dust.dust_clip_grads(grads, max_norm, out=out)
    assert abs(norm.item() - norm64) <= 4 * 2.0 ** -24 * norm64
    for a, b in zip(got, want):
        e = 2.0 ** -22 * np.abs(b * c) + 1e-44
        if a.dtype == torch.bfloat16:
            e = e + 2.0 ** -8 * np.abs(b * c)
        assert a.shape == b.shape and (np.abs(_np(a) - b * c) <= e).all()
    return norm


SHAPES = [[(1,)], [(5,), (1,), (8,)], [(0,), (17, 3), (0, 4)], [(4096,)], [(8192,), (8193,), (8191,)],
          [(1000, 33)] * 3, [(300, 500), (7,), (1 << 20,)], [(129,)] * 65, [(64, 64)] * 200,
          [(3,)] * 513, [(2,)] * 1100, [(1 << 22,), (5,), (123457,)]]


@pytest.mark.parametrize("dtypes", [["f32"], ["bf16"], ["f32", "bf16"]])
@pytest.mark.parametrize("shapes", SHAPES, ids=lambda v: "%d_%s" % (len(v), v[0]))
def test_norm_and_clipping(shapes, dtypes):
    import torch
    dev = cuda()
    grads = _tensors(shapes, dtypes, dev)
    first = check(grads, 0.7)
    assert torch.equal(first, check(grads, 1e9))
    check(grads, float("inf"))
    check([t.clone() for t in grads], 0.7, in_place=True)
    check([t.clone() for t in grads], 1e9, in_place=True)
    a = dust.dust_clip_grads(grads, 0.5, out=[torch.empty_like(t) for t in grads])
    b = dust.dust_clip_grads(grads, 0.5, out=[torch.empty_like(t) for t in grads])
    assert torch.equal(a[0], b[0]) and all(torch.equal(x, y) for x, y in zip(a[1], b[1]))


@pytest.mark.parametrize("off", [1, 2, 3, 5])
def test_views_off_16_bytes(off):
    import torch
    dev = cuda()
    for dt in (torch.float32, torch.bfloat16):
        flat = torch.randn(50000, device=dev).to(dt)
        grads = [flat[off:off + 20001], flat[20001 + off:20001 + off + 7], flat[30000:45000]]
        outs = torch.full((50000,), 9.0, device=dev, dtype=dt)
        want = [_np(t) for t in grads]
        norm64 = np.sqrt(sum((t * t).sum() for t in want))
        for o in (off, 4):
            outs.fill_(9.0)
            out = [outs[o:o + 20001], outs[20001 + o:20001 + o + 7], outs[30000:45000]]
            norm, got = dust.dust_clip_grads(grads, 2.0, out=out)
            for a, b in zip(got, want):
                assert (np.abs(_np(a) - b * 2.0 / norm64) <= 2.0 ** -7 * np.abs(b) * 2.0 / norm64).all()
            assert (outs[:o] == 9.0).all() and (outs[45000:] == 9.0).all()
            assert (outs[20008 + o:30000] == 9.0).all()


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e-3, 1e10, 1e19, 1e30])
def test_squares_past_the_range(scale):
    """Values whose squares overflow fp32, lose bits below it or vanish."""
    dev = cuda()
    check(_tensors([(3000,), (17,)], ["f32"], dev, scale), scale)
    check(_tensors([(3000,), (17,)], ["bf16"], dev, scale), scale * 1e3)


@pytest.mark.parametrize("max_norm", [1e3, 1.0, 1e-3, 1e-6, 1e-12, 1e-37, 1e-44])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("big", [500, 1 << 21])
def test_factors_below_fp32s_range(big, dtype, max_norm):
    """Gradients of 1e38 and of every size below it, scaled to a norm that is far from
    theirs: the factor is below fp32's normal numbers or all of its numbers, the
    scaled values are not. As in check(): the factor's rounding, two products'
    and bf16's; below 2^-126 of the result each of these is at most half of 2^-149
    (bf16 2^-133) instead, of which four fit into 2^-147 (2^-131)."""
    import torch
    dev = cuda()
    g = torch.Generator().manual_seed(big)
    a = torch.randn(big, generator=g).clamp(-3, 3) * 1e38
    a[1::2] *= 10.0 ** (-40 * torch.rand(big // 2, generator=g))
    a = a.to(torch.bfloat16 if dtype == "bf16" else torch.float32).to(dev)
    grads = [a, torch.ones(7, device=dev)]
    want = [_np(t) for t in grads]
    norm64 = np.sqrt(sum((t * t).sum() for t in want))
    c = float(np.float32(max_norm)) / norm64
    assert c < 2.0 ** -115 and norm64 > 3.4e38
    norm, got = dust.dust_clip_grads(grads, max_norm, out=[torch.empty_like(t) for t in grads])
    assert norm.item() == float("inf")
    for x, w in zip(got, want):
        e = 2.0 ** -22 * np.abs(w * c) + 2.0 ** -147
        if x.dtype == torch.bfloat16:
            e = e + 2.0 ** -8 * np.abs(w * c) + 2.0 ** -131
        assert (np.abs(_np(x) - w * c) <= e).all()
    assert max_norm < 1e-40 or (got[0] != 0).any()
    same, again = dust.dust_clip_grads(grads, max_norm)
    assert torch.equal(same, norm) and all(torch.equal(x, y) for x, y in zip(again, got))


def test_one_large_value_among_small_ones():
    import torch
    dev = cuda()
    t = torch.full((100000,), 1e-22, device=dev)
    t[777] = 3e20
    check([t, torch.ones(5, device=dev)], 1.0)
    z = torch.zeros(100000, device=dev)
    norm = check([z, z.clone()], 1.0)
    assert norm.item() == 0.0
    norm, out = dust.dust_clip_grads([z.clone()], 0.0)
    assert (out[0] == 0).all()
    norm, out = dust.dust_clip_grads([torch.ones(9, device=dev)], 0.0)
    assert norm.item() == 3.0 and (out[0] == 0).all()


def test_nan_and_infinity():
    import torch
    dev = cuda()
    for big in (10, 1 << 21):
        a, b = torch.ones(big, device=dev), torch.ones(40, device=dev, dtype=torch.bfloat16)
        a[3] = float("nan")
        norm, out = dust.dust_clip_grads([a.clone(), b.clone()], 1.0)
        assert norm.isnan().all() and out[0].isnan().all() and out[1].isnan().all()
        a[3] = -float("inf")
        norm, out = dust.dust_clip_grads([a.clone(), b.clone()], 1.0)
        assert norm.item() == float("inf") and out[0][3].isnan() and (out[1] == 0).all()
        assert (out[0][:3] == 0).all()
        norm, out = dust.dust_clip_grads([a.clone(), b.clone()], float("inf"))
        assert out[0][3] == -float("inf") and (out[1] == 1).all()


def test_norm_alone_and_no_tensors():
    import torch
    dev = cuda()
    norm, out = dust.dust_clip_grads([], 1.0)
    assert norm.item() == 0.0 and out == []
    g = torch.arange(1000, device=dev, dtype=torch.float32)
    arr = (Grad * 1)()
    arr[0].g, arr[0].n, arr[0].dtype = g.data_ptr(), 1000, dust.F32
    n = dust._query("dust_clip_grads_workspace", 1)
    ws, norm = torch.empty(n, dtype=torch.uint8, device=dev), torch.zeros(1, device=dev)
    st = dust.lib().dust_clip_grads(C.addressof(arr), 1, 1.0, norm.data_ptr(), ws.data_ptr(), n, None)
    want = np.sqrt((np.arange(1000.0) ** 2).sum())
    assert st == dust.OK and abs(norm.item() - want) <= 4 * 2.0 ** -24 * want
    assert torch.equal(g, torch.arange(1000, device=dev, dtype=torch.float32))


def test_overlaps_are_refused():
    import torch
    dev = cuda()
    t = torch.ones(1000, device=dev)
    for grads, out in (([t, t], None), ([t[:600], t[500:]], None), ([t[:500]], [t[1:501]]),
                       ([t[:500], t[500:]], [t[500:], t[:500]])):
        with pytest.raises(dust.DustError):
            dust.dust_clip_grads(grads, 1.0, out=out)
    assert (t == 1).all()
    # The same input twice with outputs apart, and neighbours in place, are fine.
    dust.dust_clip_grads([t, t], 1.0, out=[torch.empty_like(t), torch.empty_like(t)])
    dust.dust_clip_grads([t[:500], t[500:]], 1.0)


def test_on_another_stream_and_in_a_graph():
    import torch
    dev = cuda()
    for shapes in ([(100, 30), (7,)], [(1 << 21,), (513, 77)]):
        grads = _tensors(shapes, ["f32", "bf16"], dev)
        out = [torch.empty_like(t) for t in grads]
        want_norm, want = dust.dust_clip_grads(grads, 0.3, out=[torch.empty_like(t) for t in grads])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        norm, got = dust.dust_clip_grads(grads, 0.3, out=out, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(norm, want_norm) and all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm, got = dust.dust_clip_grads(grads, 0.3, out=out)
        for t in grads:
            t.mul_(2.0)
        for _ in range(2):
            graph.replay()
        again_norm, again = dust.dust_clip_grads(grads, 0.3, out=[torch.empty_like(t) for t in grads])
        assert torch.equal(norm, again_norm) and all(torch.equal(a, b) for a, b in zip(got, again))
