"""One training step of a small model on rewards: a block with attention and a
gated feed-forward part, the head, a clipped policy loss, exact gradients, the
estimate of one layer's gradient from jittered forwards, and clipping.

    x -> norm -> queries, keys, values -> norms and rotation -> attention -> + x
      -> norm -> gated projections -> down projection (jittered) -> + x
      -> norm -> head -> per-token losses -> policy loss

1. `dust_layer_norm`, `dust_qk_norm_rope` on the fused projection's rows, and
   attention over each sequence (PyTorch's operators).
2. `dust_gated_up`, then the down projection: clean and, in bf16, jittered by
   `dust_forward_jitter`.
3. `dust_head_loss` of every slice, and `dust_policy_loss` on those losses: the
   objective and each draw's loss changes, from which `dust_estimate_gW`
   estimates the down projection's gradient.
4. The exact gradients, back through each of them: `dust_policy_loss_grad` gives
   the `gloss` of `dust_head_loss_grad`, and so on down to the projections.
5. `dust_clip_grads` over all weights' gradients.

    python examples/policy_step.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import token_perturbation_estimator_gb300 as dust

CLIP, BETA, SIGMA = 0.2, 0.05, 0.05


def make(lengths=(200, 1, 55), d=128, heads=4, kv_heads=2, f=352, V=1000, dtype=torch.bfloat16,
         device="cuda", seed=0):
    """Weights and a batch of sampled sequences."""
    g = torch.Generator(device=device).manual_seed(seed)
    T, D = sum(lengths), d // heads

    def weight(n, m):
        return (torch.randn(n, m, generator=g, device=device) / m ** 0.5).to(dtype)

    w = {"Wqkv": weight((heads + 2 * kv_heads) * D, d), "Wo": weight(d, d), "Wg": weight(f, d),
         "Wu": weight(f, d), "Wd": weight(d, f), "E": weight(V, d)}
    w["wq"], w["wk"] = torch.ones(D, device=device), torch.ones(D, device=device)
    angle = torch.arange(max(lengths), device=device)[:, None] * 10000.0 ** (
        -torch.arange(0, D, 2, device=device) / D)
    ends = torch.tensor([0, *lengths], device=device).cumsum(0).to(torch.int32)
    targets = torch.randint(0, V, (T,), generator=g, dtype=torch.int32, device=device)
    targets[::5] = -1  # the prompts' tokens
    return w, {
        "x": torch.randn(T, d, generator=g, device=device).to(dtype), "targets": targets,
        "lengths": lengths, "heads": heads, "kv_heads": kv_heads, "seq_offsets": ends,
        "positions": torch.cat([torch.arange(n, device=device) for n in lengths]).to(torch.int32),
        "cosine": angle.cos(), "sine": angle.sin(),
        "advantages": torch.randn(len(lengths), generator=g, device=device),
        "noise": torch.randn(2, T, generator=g, device=device)}


def attention(q, k, v, b):
    """Causal, each sequence by itself, keys and values shared by groups of heads."""
    out, at = [], 0
    for n in b["lengths"]:
        qs, ks, vs = (t[at:at + n].transpose(0, 1) for t in (q, k, v))
        ks, vs = (t.repeat_interleave(b["heads"] // b["kv_heads"], 0) for t in (ks, vs))
        s = (qs @ ks.transpose(1, 2)) / q.shape[-1] ** 0.5
        s = s.masked_fill(torch.ones(n, n, device=q.device).triu(1) > 0, -float("inf"))
        out.append((s.softmax(-1) @ vs).transpose(0, 1))
        at += n
    return torch.cat(out).flatten(1)


def step(w, b, K=0, max_norm=0.1):
    x, hq, hk = b["x"], b["heads"], b["kv_heads"]
    T, d = x.shape
    D, dt = d // hq, x.dtype
    turn = (b["positions"], b["cosine"], b["sine"])

    # Forward.
    x0, mean0, rstd0 = dust.dust_layer_norm(x)
    qkv = (x0 @ w["Wqkv"].t()).view(T, hq + 2 * hk, D)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    yq, yk = dust.dust_qk_norm_rope(q, k, w["wq"], w["wk"], *turn)
    leaves = [t.detach().float().requires_grad_() for t in (yq, yk, v)]
    a32 = attention(*leaves, b)
    a = a32.detach().to(dt)
    x1 = x + a @ w["Wo"].t()
    x2, mean2, rstd2 = dust.dust_layer_norm(x1)
    h = dust.dust_gated_up(x2, w["Wg"], w["Wu"], dust.SILU)
    if K:
        Y = dust.dust_forward_jitter(h, w["Wd"], 7, dust.GAUSSIAN, 0, K, SIGMA, clean=True)
    else:
        Y = (h @ w["Wd"].t())[None]
    x3 = x1 + Y
    H, mean4, rstd4 = dust.dust_layer_norm(x3.view(-1, d))
    H = H.view(1 + K, T, d)
    nll, lse = dust.dust_head_loss(H, w["E"], b["targets"])
    # The policy that drew the samples and the reference, not far from this one.
    old, ref = nll[0] + 0.2 * b["noise"][0], nll[0] + 0.2 * b["noise"][1]
    args = (old, b["advantages"], b["seq_offsets"])
    rest = dict(ref=ref, targets=b["targets"], clip_low=CLIP, clip_high=CLIP, beta=BETA,
                mean=dust.MEAN_SEQUENCE, per_token=False)
    out = dust.dust_policy_loss(nll, *args, changes=K > 0, **rest)
    res = {"objective": out[1], "kl": out[2], "clipped": out[3], "nll": nll, "old": old, "ref": ref}
    if K:
        res["estimate"] = dust.dust_estimate_gW(h, out[4], d, b["seq_offsets"], 7, dust.GAUSSIAN, 0,
                                                SIGMA, 0.0, 1.0 / T, dust.CENTER)

    # Backward, of the clean slice.
    gloss = dust.dust_policy_loss_grad(nll[0], *args, torch.ones((), device=x.device), **rest)
    gH, gE = dust.dust_head_loss_grad(H[0], w["E"], b["targets"], lse[0], gloss)
    g3, _, _ = dust.dust_layer_norm_grad(gH, x3[0], mean4[:T], rstd4[:T])
    gh = g3 @ w["Wd"]
    g2, gWg, gWu = dust.dust_gated_up_grad(gh, x2, w["Wg"], w["Wu"], dust.SILU)
    g1 = g3 + dust.dust_layer_norm_grad(g2, x1, mean2, rstd2)[0]
    a32.backward((g1 @ w["Wo"]).float())
    gyq, gyk, gv = (t.grad.to(dt) for t in leaves)
    gqkv = torch.empty_like(qkv)  # the gradients take the projection's layout
    gqkv[:, hq + hk:] = gv
    _, _, gwq, gwk = dust.dust_qk_norm_rope_grad(gyq, gyk, q, k, w["wq"], w["wk"], *turn,
                                                 gq=gqkv[:, :hq], gk=gqkv[:, hq:hq + hk])
    f32 = torch.float32
    grads = {"Wqkv": gqkv.view(T, -1).to(f32).t() @ x0.to(f32), "Wo": g1.to(f32).t() @ a.to(f32),
             "Wg": gWg, "Wu": gWu, "Wd": g3.to(f32).t() @ h.to(f32), "E": gE, "wq": gwq, "wk": gwk}
    res["grads"] = grads
    res["norm"], clipped = dust.dust_clip_grads(list(grads.values()), max_norm,
                                                out=[torch.empty_like(t) for t in grads.values()])
    res["clipped_grads"] = dict(zip(grads, clipped))
    return res


if __name__ == "__main__":
    K = 64
    weights, batch = make()
    r = step(weights, batch, K)
    torch.cuda.synchronize()
    status = dust.dust_last_error()
    if status != dust.OK:
        raise RuntimeError("device status: " + dust.status_string(status))
    cosine = torch.nn.functional.cosine_similarity(r["estimate"].flatten(), r["grads"]["Wd"].flatten(),
                                                   dim=0)
    print("objective %.4f, KL %.4f, clipped %.3f, gradient norm %.4f"
          % (r["objective"][0], r["kl"][0], r["clipped"][0], r["norm"]))
    print("cosine of Wd's estimate (%d draws) to its gradient %.3f" % (K, cosine))
