"""One step of a model's last layers, forwards only where the estimator works
and with exact gradients where nothing stands between a layer and the loss.

    x -> norm -> linear layer W, jittered -> norm -> head E -> per-token loss

1. `dust_layer_norm` gives the layer's input X.
2. `dust_forward_jitter` runs the layer once for the clean pass and K draws.
3. `dust_layer_norm` over all slices, then `dust_head_loss`: the losses of the
   clean pass and each draw's loss changes, without any logits in memory.
4. `dust_estimate_gW` turns the loss changes into W's gradient estimate.
5. `dust_head_loss_grad` and `dust_layer_norm_grad` give the head's and the
   final norm's exact gradients, and the exact error at the layer's output,
   next to which the estimate of W's gradient is shown.
6. `dust_distill_loss` and its gradient: the same head, against a teacher's
   stored top logits.

    python examples/last_layers.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import token_perturbation_estimator_gb300 as dust


def step(T=4096, d=512, V=4096, K=64, sigma=0.05, teacher_k=32, device="cuda"):
    g = torch.Generator(device=device).manual_seed(0)
    bf16 = torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=device)

    x = normal(T, d).to(bf16)
    W = (normal(d, d) / d ** 0.5).to(bf16)
    E = (normal(V, d) * (2.0 / d ** 0.5)).to(bf16)
    weight, bias = torch.ones(d, device=device), torch.zeros(d, device=device)
    targets = torch.randint(0, V, (T,), generator=g, dtype=torch.int32, device=device)
    targets[::7] = -1  # padding
    seq = torch.tensor([0, T // 2, T], dtype=torch.int32, device=device)

    X, _, _ = dust.dust_layer_norm(x, weight, bias)
    Y = dust.dust_forward_jitter(X, W, 1, dust.GAUSSIAN, 0, K, sigma, clean=True)
    S = K + 1
    H, mean, rstd = dust.dust_layer_norm(Y.view(S * T, d), weight, bias)
    H = H.view(S, T, d)
    loss, lse, delta = dust.dust_head_loss(H, E, targets, changes=True)
    gW = dust.dust_estimate_gW(X, delta, d, seq, 1, dust.GAUSSIAN, 0, sigma, 0.0, 1.0 / T,
                               dust.CENTER)

    live = (targets >= 0).sum()
    gloss = (targets >= 0).float() / live
    gH, gE = dust.dust_head_loss_grad(H[0], E, targets, lse[0], gloss)
    gY, gweight, gbias = dust.dust_layer_norm_grad(gH, Y[0], mean[:T], rstd[:T], weight)
    exact = gY.float().t() @ X.float()  # W's gradient, through the exact error

    logits = H[0].float() @ E.float().t()
    top = (logits + 0.3 * normal(T, V)).topk(teacher_k, dim=-1)
    ids = top.indices.to(torch.int32)
    dloss, dlse, student = dust.dust_distill_loss(H[0], E, ids, top.values.contiguous(), 0.5)
    dH, dE = dust.dust_distill_loss_grad(H[0], E, ids, top.values.contiguous(), dlse, student,
                                         torch.full((T,), 1.0 / T, device=device), 0.5)
    torch.cuda.synchronize()
    status = dust.dust_last_error()
    if status != dust.OK:
        raise RuntimeError("device status: " + dust.status_string(status))
    cosine = torch.nn.functional.cosine_similarity(gW.flatten(), exact.flatten(), dim=0)
    return {"loss": (loss[0].sum() / live).item(), "cosine": cosine.item(),
            "expected_cosine": (K / (K + d)) ** 0.5, "distillation": dloss.mean().item(),
            "gE": gE, "gweight": gweight, "gbias": gbias, "dH": dH, "dE": dE}


if __name__ == "__main__":
    out = step()
    print("mean loss %.4f, distillation loss %.4f" % (out["loss"], out["distillation"]))
    print("cosine of W's estimate to its gradient %.3f (sqrt(K / (K + d)) = %.3f)"
          % (out["cosine"], out["expected_cosine"]))
