"""GPU parity of the policy loss and its gradient against the formulas in 64
bits (numpy, on the CPU).

Tolerances. A token's loss is a handful of fp32 roundings of its two terms, and
the exponentials' argument is the exact difference rounded once, which is
worth |difference| 2^-24: 2^-24 (8 + |old - nll| + |r|) of the sum of the terms'
magnitudes. The KL term itself comes from a series or from expm1 - r with |r|
above 0.5, whose cancellation costs at most a factor of 8. Means: 1e-6 of the
mean of magnitudes (fp32 sums of at most 4 values a thread, 32 lanes, 8 warps,
then 64 bits), and the weights' rounding."""
import numpy as np
import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda, offsets_from_lengths, random_lengths

pytestmark = pytest.mark.gpu

LOW, HIGH, BETA = 0.2, 0.28, 0.04


def _np(t):
    return t.double().cpu().numpy()


def _dev(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def _inputs(S, lengths, dev, before=0, behind=0, masked=0.3, per_token=False, seed=0):
    rng = np.random.default_rng(17 * S + len(lengths) + seed)
    T = before + int(np.sum(lengths)) + behind
    off = (before + offsets_from_lengths(lengths)).astype(np.int32)
    nll = -np.log(rng.uniform(1e-4, 1.0, T)) * 1.5
    old, ref = nll + 0.25 * rng.standard_normal(T), nll + 0.4 * rng.standard_normal(T)
    many = np.concatenate([nll[None], nll + 0.1 * rng.standard_normal((S - 1, T))])
    adv = rng.standard_normal(T if per_token else len(lengths))
    tg = np.where(rng.uniform(size=T) < masked, -1, rng.integers(0, 9, T)).astype(np.int32)
    f = np.float32
    return [_dev(a.astype(f), dev) for a in (many, old, ref, adv)] + [_dev(off, dev), _dev(tg, dev)]


def reference(nll, old, ref, adv, off, tg, beta, by_sequence, per_token, gtotal=None):
    nll, old, adv, off = _np(nll), _np(old), _np(adv), off.cpu().numpy()
    T = nll.shape[1]
    seq = np.searchsorted(off, np.arange(T), side="right") - 1
    inside = (seq >= 0) & (np.arange(T) < off[-1])
    scored = inside & (tg.cpu().numpy() >= 0 if tg is not None else True)
    seq = np.where(inside, seq, 0)
    A = adv if per_token else (adv[seq] if len(adv) else np.zeros(T))
    step = old - nll
    clipped = np.where(A > 0, step > np.log1p(HIGH),
                       (A < 0) & (step < np.log1p(-LOW)))
    bound = np.where(A > 0, 1 + HIGH, 1 - LOW)
    ratio = np.exp(step)
    first = -np.where(clipped, bound, ratio) * A
    r = nll - _np(ref) if ref is not None else np.zeros_like(nll)
    kl = np.expm1(r) - r
    b = np.float64(np.float32(beta))
    loss = np.where(scored, first + b * kl, 0.0)
    size = np.where(scored, (np.abs(first) + b * np.where(np.abs(r) > 0.5, np.exp(r) + np.abs(r), kl)) *
                    (8 + np.abs(step) + np.abs(r)), 0.0)
    count = np.bincount(seq[scored], minlength=max(len(off) - 1, 1))
    if by_sequence:
        w = np.where(scored, 1.0 / np.maximum(count[seq] * max((count > 0).sum(), 1), 1), 0.0)
    else:
        w = scored / max(scored.sum(), 1)
    kl, clipped = np.where(scored, kl, 0.0), clipped & scored
    if gtotal is None:
        return loss, size, [((w * v).sum(1), (w * np.abs(v)).sum(1)) for v in (loss, kl, clipped)]
    g = np.where(clipped, 0.0, ratio * A) + b * np.expm1(r)
    gs = (np.abs(np.where(clipped, 0.0, ratio * A)) + b * np.abs(np.expm1(r))) * (8 + np.abs(step) +
                                                                                   np.abs(r))
    gt = _np(gtotal)[:, None]
    return np.where(scored, gt * w * g, 0.0), np.where(scored, np.abs(gt) * w * gs, 0.0)


def check(S, lengths, dev, beta=BETA, by_sequence=True, use_ref=True, use_targets=True, **kw):
    import torch
    nll, old, ref, adv, off, tg = _inputs(S, lengths, dev, **kw)
    per_token = kw.get("per_token", False)
    ref, tg = ref if use_ref else None, tg if use_targets else None
    args = dict(ref=ref, targets=tg, clip_low=LOW, clip_high=HIGH, beta=beta, per_token=per_token,
                mean=dust.MEAN_SEQUENCE if by_sequence else dust.MEAN_TOKEN)
    out = dust.dust_policy_loss(nll, old, adv, off, changes=True, **args)
    loss, total, kl, clipped, delta = out
    want, size, means = reference(nll, old, ref, adv, off, tg, beta, by_sequence, per_token)
    e = 2.0 ** -24 * size + 1e-37
    assert (np.abs(_np(loss) - want) <= e).all()
    assert (np.abs(_np(delta) - (want[1:] - want[:1])) <=
            e[1:] + e[:1] + 2.0 ** -24 * np.abs(want[1:] - want[:1])).all()
    for got, (m, mag) in zip((total, kl, clipped), means):
        assert (np.abs(_np(got) - m) <= 4e-6 * mag + 1e-37).all()
    gtotal = torch.linspace(0.5, 1.5, S, device=dev)
    gnll = dust.dust_policy_loss_grad(nll, old, adv, off, gtotal, **args)
    g64, gsize = reference(nll, old, ref, adv, off, tg, beta, by_sequence, per_token, gtotal)
    assert (np.abs(_np(gnll) - g64) <= 2.0 ** -24 * gsize + 1e-37).all()
    again = dust.dust_policy_loss(nll, old, adv, off, changes=True, **args)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    return nll, old, ref, adv, off, tg, args


LENGTHS = [[1], [2], [300], [1, 1, 1], [5, 1, 40, 2], [1023], [1024], [1025], [700, 1, 2000, 33],
           [1] * 500, [40000, 3, 20000]]


@pytest.mark.parametrize("by_sequence", [False, True])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: "%dx%d" % (len(v), sum(v)))
@pytest.mark.parametrize("S", [1, 3, 9, 33])
def test_loss_and_gradient(S, lengths, by_sequence):
    dev = cuda()
    check(S, lengths, dev, by_sequence=by_sequence)
    check(S, lengths, dev, by_sequence=by_sequence, per_token=True, use_ref=False, beta=0.0)


@pytest.mark.parametrize("by_sequence", [False, True])
def test_ragged_batches(by_sequence):
    dev = cuda()
    rng = np.random.default_rng(3)
    for T, most in ((777, 50), (5000, 900), (70000, 30), (70000, 30000)):
        check(2, random_lengths(rng, T, most), dev, by_sequence=by_sequence)


@pytest.mark.parametrize("by_sequence", [False, True])
def test_tokens_outside_and_empty_sequences(by_sequence):
    dev = cuda()
    for lengths, before, behind in (([5, 0, 7], 3, 4), ([0], 2, 2), ([0, 0, 9, 0], 0, 1000),
                                    ([2000, 0, 0, 1], 1030, 1), ([0, 4], 0, 0)):
        check(3, lengths, dev, before=before, behind=behind, by_sequence=by_sequence)
        check(3, lengths, dev, before=before, behind=behind, by_sequence=by_sequence, masked=1.0)
        check(1, lengths, dev, before=before, behind=behind, by_sequence=by_sequence,
              use_targets=False)


@pytest.mark.parametrize("T", [40, 5000])
def test_unscored_tokens_hide_what_they_hold(T):
    import torch
    dev = cuda()
    nll, old, ref, adv, off, tg = _inputs(3, [T // 2, T - T // 2], dev, behind=5, per_token=True)
    args = dict(targets=tg, beta=BETA, mean=dust.MEAN_SEQUENCE, per_token=True)
    want = dust.dust_policy_loss(nll, old, adv, off, ref=ref, changes=True, **args)
    gt = torch.ones(3, device=dev)
    wanted = dust.dust_policy_loss_grad(nll, old, adv, off, gt, ref=ref, **args)
    off_now = tg < 0
    off_now[T:] = True
    for t, v in ((nll, float("nan")), (old, float("inf")), (ref, -float("inf")), (adv, float("nan"))):
        t[..., off_now] = v
    got = dust.dust_policy_loss(nll, old, adv, off, ref=ref, changes=True, **args)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = dust.dust_policy_loss_grad(nll, old, adv, off, gt, ref=ref, **args)
    assert torch.equal(g, wanted) and (g[:, off_now] == 0).all()


def test_borders_are_decided_exactly():
    """Ratios one fp32 step on either side of the bounds, both signs."""
    import torch
    dev = cuda()
    f = np.float32
    hi, lo = np.log1p(HIGH), np.log1p(-LOW)
    steps = []
    for b in (hi, lo):
        x = f(b)
        steps += [np.nextafter(x, f(-9)), x, np.nextafter(x, f(9))]
    steps = np.array(steps * 2, f)
    adv = np.array([1.0] * 6 + [-1.0] * 6, f)
    old = steps  # nll = 0: the difference is exact
    nll = torch.zeros(12, device=dev)
    off = torch.tensor([0, 12], dtype=torch.int32, device=dev)
    loss, total, kl, clipped = dust.dust_policy_loss(
        nll, _dev(old, dev), _dev(adv, dev), off, clip_low=LOW, clip_high=HIGH, per_token=True)
    want = np.where(adv > 0, steps.astype(np.float64) > hi, steps.astype(np.float64) < lo)
    assert abs(clipped.item() - want.mean()) < 1e-7
    g = dust.dust_policy_loss_grad(nll, _dev(old, dev), _dev(adv, dev), off,
                                   torch.ones((), device=dev), clip_low=LOW, clip_high=HIGH,
                                   per_token=True)
    assert ((_np(g) == 0) == want).all()


def test_bounds_at_their_ends():
    """clip_low 1 and an infinite clip_high: no ratio is clipped."""
    import torch
    dev = cuda()
    nll, old, ref, adv, off, tg = _inputs(2, [50, 60], dev, per_token=True)
    old = old * 20.0 - 10.0
    loss, total, kl, clipped = dust.dust_policy_loss(nll, old, adv, off, clip_low=1.0,
                                                     clip_high=float("inf"), per_token=True)
    assert (clipped == 0).all()
    # The exponent is rounded once, which is worth |step| 2^-24 of the ratio (steps
    # up to 140 here); past fp32's range the loss is infinite.
    step = old.double() - nll.double()

    def near(got, want):
        inside = want.abs() < 3.4e38
        assert (got[~inside] == want[~inside].sign().float() * float("inf")).all()
        off = (got.double() - want).abs()[inside]
        return bool((off <= 2.0 ** -24 * ((8 + step.abs()) * want.abs())[inside] + 1e-37).all())

    assert near(loss, -torch.exp(step) * adv.double())
    one = dust.dust_policy_loss(nll, old, adv, off, clip_low=0.0, clip_high=0.0, per_token=True)[0]
    assert near(one, -torch.minimum(torch.exp(step) * adv.double(), adv.double()))


def test_no_bound_takes_no_longer():
    """The documented calls without a bound on one side or both: few tokens may take
    the slow way, in 64 bits (which made them 1.9 times as long)."""
    import torch
    dev = cuda()
    S, T = 33, 65536
    g = torch.Generator().manual_seed(3)
    nll = torch.rand((S, T), generator=g).to(dev)
    old = nll[0] + 0.3 * torch.randn(T, generator=g).to(dev)
    adv = torch.randn(T, generator=g).to(dev)
    off = torch.tensor([0, T], dtype=torch.int32, device=dev)
    graphs = []
    for low, high in ((0.2, 0.28), (0.2, float("inf")), (1.0, 0.28), (1.0, float("inf"))):
        args = dict(ref=old, beta=BETA, per_token=True, clip_low=low, clip_high=high, changes=True)
        dust.dust_policy_loss(nll, old, adv, off, **args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(10):
                dust.dust_policy_loss(nll, old, adv, off, **args)
        graphs.append(graph)
    best = [float("inf")] * len(graphs)
    for _ in range(12):  # in turn, the shortest of each
        for i, graph in enumerate(graphs):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], a.elapsed_time(b))
    assert max(best[1:]) < 1.4 * best[0], best


@pytest.mark.parametrize("by_sequence", [False, True])
@pytest.mark.parametrize("S", [1, 2, 7])
@pytest.mark.parametrize("lengths", [[43], [7, 29, 7], [1531], [300, 25], [3, 4000, 900], [70001]],
                         ids=lambda v: "%dx%d" % (len(v), sum(v)))
def test_total_of_losses_that_cancel(lengths, S, by_sequence):
    """A ratio of 1 makes a token's loss the advantage, exactly, so that only the
    weights and sums can be off. Up to 2048 tokens of 4 slices those carry what
    their roundings lose along: below 2^7 roundings of 2^-48 of the magnitudes, and
    the result's own half step. Beyond, in either, a thread adds 4 tokens' terms in
    fp32: each of the 4 additions rounds by at most half a step of its running sum,
    that is of the thread's magnitudes, so that together they are off by at most
    4 * 2^-24 of all magnitudes; all else is in 64 bits or carried along."""
    import torch
    dev = cuda()
    rng = np.random.default_rng(5)
    T, f = sum(lengths), np.float32
    adv = rng.standard_normal(T).astype(f)
    adv[1::2] = -adv[:T - 1:2][:len(adv[1::2])] * f(1 + 1e-4)  # pairs of nearly opposite sign
    old = rng.uniform(0.1, 9.0, T).astype(f)
    off = offsets_from_lengths(lengths).astype(np.int32)
    loss, total = dust.dust_policy_loss(
        _dev(np.tile(old, (S, 1)), dev), _dev(old, dev), _dev(adv, dev), _dev(off, dev),
        clip_low=LOW, clip_high=HIGH, per_token=True,
        mean=dust.MEAN_SEQUENCE if by_sequence else dust.MEAN_TOKEN)[:2]
    assert torch.equal(loss, _dev(np.tile(-adv, (S, 1)), dev))
    n = np.repeat(lengths, lengths) * len(lengths) if by_sequence else np.full(T, T)
    terms = -adv.astype(np.float64) / n
    m, mag = terms.sum(), np.abs(terms).sum()
    tol = 2.0 ** -24 * abs(m) + (2.0 ** -41 if T <= 2048 and S <= 4 else 4 * 2.0 ** -24) * mag
    assert (np.abs(_np(total) - m) <= tol).all()


@pytest.mark.parametrize("S", [1, 7])
def test_weights_of_more_tokens_than_fp32_counts(S):
    """4097 sequences, one of them with 4099 scored tokens: their product is above
    2^24 and odd. All of its losses are 1 and all those of one with fewer tokens -1,
    so that the means cancel and the weights alone show; all others are 0.
    Each thread has one of these tokens, so that its term is exact; the terms are
    added in 64 bits. What a weight leaves is at most 3 * 2^-24 for the rounding of
    the counts and their product and 2^-24 for its own, 2^-22 of it in all: what is
    of second order below 2^-44, its computing and adding up (3 and 14 roundings)
    below 2^-41 with that. (A weight of the rounded product is 6e-8 off.)"""
    dev = cuda()
    f, ones, singles = np.float32, (16 * 1024 + 3, 15 * 1024 + 700), 4095
    lengths = list(ones) + [1] * singles
    off = offsets_from_lengths(lengths).astype(np.int32)
    T = int(off[-1])
    seq = np.repeat(np.arange(len(lengths)), lengths)
    scored = (np.arange(T) % 1024 < 256) | (seq > 1)
    count = np.bincount(seq[scored])
    assert count[0] == 4099 and len(count) * int(count[0]) > 2 ** 24 and (count > 0).all()
    w = f(1) / (f(len(count)) * count.astype(f))  # weights of the rounded products
    assert abs(w[0] * np.float64(count[0]) - w[1] * np.float64(count[1])) > 2.0 ** -26 / len(count)
    adv = np.zeros(len(lengths), f)
    adv[:2] = -1.0, 1.0
    old = np.random.default_rng(5).uniform(0.1, 9.0, T).astype(f)
    loss, total = dust.dust_policy_loss(
        _dev(np.tile(old, (S, 1)), dev), _dev(old, dev), _dev(adv, dev), _dev(off, dev),
        targets=_dev(np.where(scored, 1, -1).astype(np.int32), dev), clip_low=LOW, clip_high=HIGH,
        per_token=False, mean=dust.MEAN_SEQUENCE)[:2]
    assert (np.abs(_np(loss)).sum(1) == count[0] + count[1]).all()
    assert (np.abs(_np(total)) <= 2.0 ** -41 * 2.0 / len(count)).all()


@pytest.mark.parametrize("T", [1, 4, 64, 1000, 2048, 2049, 4096])
def test_infinite_losses_make_an_infinite_total(T):
    """One token whose ratio is above fp32's range: its loss is infinite, and the
    mean with it, in this slice alone; a NaN makes the mean a NaN."""
    import torch
    dev = cuda()
    for S, bad in ((1, 0), (3, 1), (33, 32)):
        nll = torch.ones(S, T, device=dev)
        old = torch.ones(T, device=dev)
        adv = torch.full((T,), -1.0, device=dev)
        off = torch.tensor([0, T], dtype=torch.int32, device=dev)
        t = T // 2
        nll[bad, t] = -100.0  # e^101 > 2^128
        for mean in (dust.MEAN_TOKEN, dust.MEAN_SEQUENCE):
            total = dust.dust_policy_loss(nll, old, adv, off, per_token=True, mean=mean)[1]
            want = torch.ones(S, device=dev)
            want[bad] = float("inf")
            assert torch.equal(total[want == 1], want[want == 1].double().to(total.dtype))
            assert total[bad] == float("inf")
            two = adv.clone()
            two[t] = float("nan")
            total = dust.dust_policy_loss(nll, old, two, off, per_token=True, mean=mean)[1]
            assert torch.isnan(total).all()


@pytest.mark.parametrize("T", [5, 3000])
def test_terms_of_no_weight_do_not_overflow(T):
    """Without advantage a ratio above fp32's range adds nothing to the loss, and
    without beta neither does such a KL term."""
    import torch
    dev = cuda()
    old = torch.full((T,), 200.0, device=dev)  # e^200 > 2^128
    nll = torch.zeros(2, T, device=dev)
    adv = torch.zeros(T, device=dev)
    ref = torch.full((T,), -100.0, device=dev)
    off = torch.tensor([0, T], dtype=torch.int32, device=dev)
    gt = torch.ones(2, device=dev)
    for kw in ({}, dict(ref=ref, beta=0.0)):
        loss, total, kl, clipped = dust.dust_policy_loss(nll, old, adv, off, per_token=True, **kw)
        assert (loss == 0).all() and (total == 0).all() and (clipped == 0).all()
        assert (kl == (float("inf") if kw else 0)).all()
        g = dust.dust_policy_loss_grad(nll, old, adv, off, gt, per_token=True, **kw)
        assert (g == 0).all()
    adv[T - 1] = float("nan")  # but no NaN is hidden
    assert torch.isnan(dust.dust_policy_loss(nll, old, adv, off, per_token=True)[0][:, -1]).all()
    adv[T - 1], old[T - 1] = 0, float("nan")
    assert torch.isnan(dust.dust_policy_loss(nll, old, adv, off, per_token=True)[0][:, -1]).all()


def test_gradient_against_differences():
    """Central differences of the total, where no ratio is near a bound."""
    import torch
    dev = cuda()
    nll, old, ref, adv, off, tg = _inputs(2, [60, 1, 90], dev)
    args = dict(ref=ref, targets=tg, clip_low=0.9, clip_high=9.0, beta=0.3, mean=dust.MEAN_SEQUENCE)
    gt = torch.tensor([0.7, 1.3], device=dev)
    g = dust.dust_policy_loss_grad(nll, old, adv, off, gt, **args)
    u = torch.randn(nll.shape, generator=torch.Generator().manual_seed(1)).to(dev)
    e = 2.0 ** -8

    def value(x):
        return (dust.dust_policy_loss(nll + x * u, old, adv, off, **args)[1].double() *
                gt.double()).sum().item()

    terms = g.double() * u.double()
    assert abs((value(e) - value(-e)) / (2 * e) - terms.sum().item()) <= 2e-3 * terms.norm().item()


def test_missing_outputs_one_dimension_and_in_place():
    import ctypes as C
    import torch
    dev = cuda()
    nll, old, ref, adv, off, tg = _inputs(1, [33, 50], dev)
    args = dict(ref=ref, targets=tg, beta=BETA)
    flat = dust.dust_policy_loss(nll[0], old, adv, off, **args)
    full = dust.dust_policy_loss(nll, old, adv, off, **args)
    assert flat[0].shape == nll[0].shape and flat[1].shape == ()
    assert all(torch.equal(a.reshape(-1), b.reshape(-1)) for a, b in zip(flat, full))
    g = dust.dust_policy_loss_grad(nll[0], old, adv, off, torch.ones((), device=dev), **args)
    mine = nll[0].clone()
    dust.dust_policy_loss_grad(mine, old, adv, off, torch.ones((), device=dev), gnll=mine, **args)
    assert torch.equal(mine, g)
    n = dust._query("dust_policy_loss_workspace", 1, 83, 2)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    kl = torch.zeros(1, device=dev)
    p = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    st = dust.lib().dust_policy_loss(p(nll), p(old), p(ref), p(adv), 0, p(off), 2, p(tg), 1, 83, 0.2,
                                     0.2, BETA, dust.MEAN_TOKEN, None, None, p(kl), None, None, p(ws),
                                     n, None)
    assert st == dust.OK and torch.equal(kl, full[2])
    none = dust.dust_policy_loss(nll[:, :0], old[:0], adv[:0], off[:1] * 0, per_token=False)
    assert none[0].numel() == 0 and (none[1] == 0).all()


def test_on_another_stream_and_in_a_graph():
    import torch
    dev = cuda()
    for lengths in ([100, 37], [3000, 9000]):
        nll, old, ref, adv, off, tg = _inputs(3, lengths, dev)
        args = dict(ref=ref, targets=tg, beta=BETA, mean=dust.MEAN_SEQUENCE)
        gt = torch.ones(3, device=dev)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        got = dust.dust_policy_loss(nll, old, adv, off, stream=st, changes=True, **args)
        torch.cuda.current_stream().wait_stream(st)
        want = dust.dust_policy_loss(nll, old, adv, off, changes=True, **args)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = dust.dust_policy_loss(nll, old, adv, off, changes=True, **args)
            g = dust.dust_policy_loss_grad(nll, old, adv, off, gt, **args)
        tg.copy_(torch.roll(tg, 7))
        nll.add_(0.01)
        for _ in range(2):
            graph.replay()
        want = dust.dust_policy_loss(nll, old, adv, off, changes=True, **args)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert torch.equal(g, dust.dust_policy_loss_grad(nll, old, adv, off, gt, **args))
