"""Gradients of tokens that the model is sure of: a loss near 1e-4, so that
the target's entry of G is -1e-4, the difference of a probability next to 1
and 1. An error in the target's logit that the log-sum does not share is an
error of that entry in full.

The logits are sums of d products of which the target's are all of one sign
(its vector lies along the token's), 30 in all, half of that shared by every
id; the reference takes the same bf16 values in 64 bits.

Tolerance, before the first run. With the forward's log-sum, the target's
entry is off by the rounding of the log-sum (2^-20, half a step at 30), of
its product with log2 e (half a step at 43, 2^-19 ln 2 in the exponent), of
the exponential and of the sum behind the log-sum (2^-22 each, twice):
3.3e-6 absolute at most, where logits of both passes are the same bits. G and
gH are rounded to bf16, 2^-9 each. A row of gH is the token's own part of its target's
vector times 1e-4 (the shared part cancels between the target and the rest,
but not its error: the error counts sqrt(2) of that): normwise by row
1.5 * 3.3e-6 / (1 - p) + 8e-3.
"""
import numpy as np
import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda

pytestmark = pytest.mark.gpu


def _sure(T, d, V, dev):
    """H, E bf16 and targets: logit 30 for the target, near 15 for the rest
    so that the loss is about 1e-4."""
    import torch
    g = torch.Generator().manual_seed(T + d + V)
    own = float(np.log(V / 1e-4))
    shared = 30.0 - own
    n = d // 2

    def size(*shape):  # magnitudes with all of bf16's bits
        return 0.75 + 0.5 * torch.rand(shape, generator=g)

    sign = torch.randint(0, 2, (V, n), generator=g) * 2.0 - 1.0
    # squares of these magnitudes are 1.02 on average
    vec = sign * size(V, n)
    common = size(n)
    E = torch.cat([common.expand(V, n) * (shared / (1.02 * n)), vec * (own / (1.02 * n))], 1)
    y = torch.randperm(V, generator=g)[:T].to(torch.int32)
    H = torch.cat([common.expand(T, n), vec[y.long()]], 1)
    return (H.to(torch.bfloat16).to(dev), E.to(torch.bfloat16).to(dev), y.to(dev))


def _np(t):
    return t.double().cpu().numpy()


# The tensor cores' tiles, sums in one run and in several; few rows, which the
# CUDA cores take.
@pytest.mark.parametrize("T,d,V", [(150, 512, 2000), (150, 1024, 1500), (150, 2048, 2000),
                                   (140, 8192, 1200), (260, 2056, 700), (1, 2048, 9000),
                                   (2, 1024, 3000), (4, 512, 4000), (5, 2048, 3000),
                                   (3, 2048, 9000), (4, 1024, 20000), (4, 4096, 2000)])
def test_gradients_of_sure_tokens(T, d, V):
    import torch
    dev = cuda()
    H, E, y = _sure(T, d, V, dev)
    loss, lse = dust.dust_head_loss(H, E, y)
    gH, gE = dust.dust_head_loss_grad(H, E, y, lse, torch.ones(T, device=dev))
    x = _np(H) @ _np(E).T
    m = x.max(1, keepdims=True)
    yn, r = y.cpu().numpy(), np.arange(T)
    e = np.exp(x - m)
    others = e.copy()
    others[r, yn] = 0.0
    e /= e.sum(1, keepdims=True)
    left = (others / (np.exp(x[r, yn] - m[:, 0])[:, None] + others.sum(1, keepdims=True))).sum(1)
    assert 1e-5 < left.min() and left.max() < 1e-3  # 1 - p of the target
    G = e
    G[r, yn] = -left
    want = G @ _np(E)
    off = np.linalg.norm(_np(gH) - want, axis=1) / np.linalg.norm(want, axis=1)
    tol = 1.5 * 3.3e-6 / left + 8e-3
    assert (off <= tol).all(), (off.max(), (off / tol).max())
    # Each id is the target of one token at most: its row of gE is that token's.
    wE = (G.T @ _np(H))[yn]
    offE = np.linalg.norm(_np(gE)[yn] - wE, axis=1) / np.linalg.norm(wE, axis=1)
    assert (offE <= tol).all(), (offE.max(), (offE / tol).max())
