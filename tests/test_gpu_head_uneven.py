"""Rows of one warp that need different amounts of work in the same columns:
wanted logits and gradient entries crowded into a few columns in some rows,
spread out or missing in others. Each lane of the epilogue then goes through
its own entries as often as it has some before the warp reads on.

Tolerances, before the first run: a logit is an fp32 sum of d products of
values near 1, off by less than sqrt(d) 2^-24 of the sum of their magnitudes:
2e-5 absolute here (|x| < 20). fp32 gradients: a probability is off by that
much relative, normwise 2e-5; bf16: G and the result rounded, normwise 5e-3.
"""
import numpy as np
import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda, rel_fro

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


def _uneven(T, V, K):
    """Row t's entries: t mod (K + 1) of them, by turns in one block of 32
    columns, at its two edges, and over all columns."""
    rng = np.random.default_rng(5)
    ids = np.full((T, K), -1, np.int32)
    for t in range(T):
        n = t % (K + 1)
        block = 32 * int(rng.integers(0, V // 32))
        if t % 3 == 0:
            at = block + rng.permutation(32)[:min(n, 32)]
        elif t % 3 == 1:
            at = np.unique(np.clip([block - 1, block, block + 31, block + 32], 0, V - 1))[:n]
        else:
            at = rng.permutation(V)[:n]
        where = rng.permutation(K)[:len(at)]
        ids[t, where] = at
    return ids


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,V,K", [(260, 64, 1000, 40), (130, 1100, 333, 33)])
def test_entries_crowded_into_some_rows(T, d, V, K, dtype):
    import torch
    dev = cuda()
    g = torch.Generator().manual_seed(T + d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    H = torch.randn((T, d), generator=g).to(dt).to(dev)
    E = (torch.randn((V, d), generator=g) * (2.0 / d ** 0.5)).to(dt).to(dev)
    z = (torch.randn((T, K), generator=g) * 2).to(dev)
    idn = _uneven(T, V, K)
    ids = torch.from_numpy(idn).to(dev)
    loss, lse, student = dust.dust_distill_loss(H, E, ids, z)
    x = _np(H) @ _np(E).T
    want = np.where(idn >= 0, np.take_along_axis(x, np.maximum(idn, 0).astype(np.int64), 1), 0.0)
    assert np.abs(_np(student) - want).max() <= 2e-5
    m = x.max(1, keepdims=True)
    wl = (m + np.log(np.exp(x - m).sum(1, keepdims=True)))[:, 0]
    assert np.abs(_np(lse) - wl).max() <= 2e-5
    e = np.where(idn >= 0, np.exp(_np(z)), 0.0)
    q = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    G = np.exp(x - wl[:, None]) * (idn >= 0).any(1)[:, None]
    np.add.at(G, (np.arange(T)[:, None], np.maximum(idn, 0)), -q)
    gH, gE = dust.dust_distill_loss_grad(H, E, ids, z, lse, student, torch.ones(T, device=dev))
    tol = 2e-5 if dtype == "f32" else 5e-3
    assert rel_fro(_np(gH), G @ _np(E)) <= tol
    assert rel_fro(_np(gE), G.T @ _np(H)) <= tol


@pytest.mark.parametrize("every", [1, 7])
def test_targets_of_some_lanes_in_the_same_columns(every):
    """Every `every`-th row's target lies in the first 32 columns, the others
    have theirs elsewhere or none."""
    import torch
    dev = cuda()
    T, d, V = 200, 96, 700
    g = torch.Generator().manual_seed(every)
    H = torch.randn((T, d), generator=g).to(torch.bfloat16).to(dev)
    E = (torch.randn((V, d), generator=g) * (2.0 / d ** 0.5)).to(torch.bfloat16).to(dev)
    t = np.arange(T)
    yn = np.where(t % every == 0, t % 32, np.where(t % 2 == 0, -1, 32 + t * 3 % (V - 32)))
    y = torch.from_numpy(yn.astype(np.int32)).to(dev)
    loss, lse = dust.dust_head_loss(H, E, y)
    x = _np(H) @ _np(E).T
    m = x.max(1, keepdims=True)
    wl = (m + np.log(np.exp(x - m).sum(1, keepdims=True)))[:, 0]
    want = np.where(yn >= 0, wl - x[t, np.maximum(yn, 0)], 0.0)
    assert np.abs(_np(loss) - want).max() <= 4e-5
    G = np.exp(x - wl[:, None])
    G[t, np.maximum(yn, 0)] -= 1.0
    G *= (yn >= 0)[:, None]
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, torch.ones(T, device=dev))
    assert rel_fro(_np(gH), G @ _np(E)) <= 5e-3
    assert rel_fro(_np(gE), G.T @ _np(H)) <= 5e-3
