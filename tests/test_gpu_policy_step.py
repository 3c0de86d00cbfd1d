"""A training step's operators together: examples/policy_step.py's gradients
against automatic differentiation of the same model in 64 bits.

fp32: every operator is within 2e-6 normwise of its formula and the matrix
products between them too; ten of them one after another, with gradients that
are up to ten times as sensitive: 2e-4. bf16: each of about twelve roundings
of the activations is worth 2^-9 rms or less (1.7e-3), independent of one
another, and the head's softmax and the rotations pass them on unamplified:
sqrt(12) x 1.7e-3 x 5 for the products' sensitivity = 3e-2."""
import os
import sys

import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def reference(w, b, nll0):
    """The objective's gradients in 64 bits, the samples' losses as given."""
    import torch
    import policy_step as ex
    w = {k: t.double().requires_grad_() for k, t in w.items()}
    x, hq, hk = b["x"].double(), b["heads"], b["kv_heads"]
    T, d = x.shape
    D = d // hq

    def ln(t):
        return torch.nn.functional.layer_norm(t, (d,), eps=1e-5)

    def rope(t, weight):
        m = torch.nn.functional.rms_norm(t, (D,), weight, 1e-6)
        p = b["positions"].long()
        c, s = b["cosine"].double()[p][:, None], b["sine"].double()[p][:, None]
        u, v = m[..., :D // 2], m[..., D // 2:]
        return torch.cat([u * c - v * s, v * c + u * s], -1)

    qkv = (ln(x) @ w["Wqkv"].t()).view(T, hq + 2 * hk, D)
    a = ex.attention(rope(qkv[:, :hq], w["wq"]), rope(qkv[:, hq:hq + hk], w["wk"]), qkv[:, hq + hk:], b)
    x1 = x + a @ w["Wo"].t()
    x2 = ln(x1)
    h = torch.nn.functional.silu(x2 @ w["Wg"].t()) * (x2 @ w["Wu"].t())
    H = ln(x1 + h @ w["Wd"].t())
    logp = (H @ w["E"].t()).log_softmax(-1)
    y = b["targets"].long()
    nll = torch.where(y >= 0, -logp.gather(1, y.clamp(min=0)[:, None])[:, 0], torch.zeros(T).to(x))
    old, ref = (nll0.double() + 0.2 * n.double() for n in b["noise"])
    ends = b["seq_offsets"].long()
    seq = torch.repeat_interleave(torch.arange(len(b["lengths"]), device=x.device), ends.diff())
    adv = b["advantages"].double()[seq]
    ratio = (old - nll).exp()
    r = nll - ref
    loss = -torch.minimum(ratio * adv, ratio.clamp(1 - ex.CLIP, 1 + ex.CLIP) * adv) + ex.BETA * (
        r.expm1() - r)
    scored = (y >= 0).double()
    count = torch.zeros(len(b["lengths"])).to(x).index_add(0, seq, scored)
    weight = scored / (count.clamp(min=1) * (count > 0).sum())[seq]
    total = (weight * loss).sum()
    total.backward()
    return total.detach(), nll.detach(), {k: t.grad for k, t in w.items()}


def check(dtype, tol, **sizes):
    import torch
    import policy_step as ex
    cuda()
    w, b = ex.make(dtype=dtype, **sizes)
    r = ex.step(w, b)
    torch.cuda.synchronize()
    assert dust.dust_last_error() == dust.OK
    total, nll, want = reference(w, b, r["nll"][0])
    assert ((r["nll"][0].double() - nll).norm() / nll.norm()).item() <= tol
    for k, g in r["grads"].items():
        assert ((g.double() - want[k]).norm() / want[k].norm()).item() <= tol, k
    norm = torch.sqrt(sum((g.double() ** 2).sum() for g in r["grads"].values()))
    assert abs(r["norm"].item() - norm.item()) <= 4 * 2.0 ** -24 * norm.item()
    c = min(1.0, 0.1 / norm.item())
    for k, g in r["clipped_grads"].items():
        assert torch.allclose(g.double(), r["grads"][k].double() * c, rtol=1e-6, atol=0)


def test_gradients_of_the_step_fp32():
    import torch
    check(torch.float32, 2e-4)
    check(torch.float32, 2e-4, lengths=(1, 2, 1), d=72, heads=3, kv_heads=1, f=101, V=97)


def test_gradients_of_the_step_bf16():
    import torch
    check(torch.bfloat16, 3e-2, lengths=(300, 1, 40, 700))


def test_estimate_beside_the_exact_gradient():
    """The estimate of the down projection's gradient from the policy's loss
    changes points the exact gradient's way: its expected cosine is about
    sqrt(K / (K + d)) = 0.7; half of that is far from chance (1 / sqrt(d f))."""
    import torch
    import policy_step as ex
    cuda()
    r = ex.step(*ex.make(d=64, heads=2, f=96, lengths=(500, 300, 224)), 64)
    assert dust.dust_last_error() == dust.OK
    cosine = torch.nn.functional.cosine_similarity(r["estimate"].flatten(),
                                                   r["grads"]["Wd"].flatten(), dim=0)
    assert cosine.item() >= 0.3
    assert r["estimate"].shape == r["grads"]["Wd"].shape and r["objective"].shape == (65,)
