"""The language-model operators beside the estimator, as cases to be measured.

Three operators, each forward and backward: layer norm, the head's softmax
cross entropy over the vocabulary, and distillation from a teacher's top
logits through the same head. `run` computes a case once, in elementary torch
operations in 32 bits (`own` false) or through the library (`own` true);
`exact` computes the same outputs from the definitions in 64 bits.

A case's fields: op ("ln", "loss", "distill"), back (backward pass), dtype
("bf16" or "f32") and sizes: T tokens, d width, V vocabulary, S slices of the
T tokens (draws of a jittered forward, the first one clean), k teacher logits
a token, ignored (the share of tokens without a target).
"""
import math

import torch

own = False

EPS = 1e-5
TEMPER = 0.5  # the distillation's inverse temperature


def listed():
    return [
        # The final norm of one generated token: all latency.
        dict(name="ln_token", op="ln", back=False, dtype="bf16", T=1, d=512),
        # Norm before the down-projection of the 64 x 1024-token sweep: past L2.
        dict(name="ln_wide", op="ln", back=False, dtype="bf16", T=65536, d=2048),
        # Backward of the residual stream's norm over the same tokens.
        dict(name="ln_back_sweep", op="ln", back=True, dtype="bf16", T=65536, d=512),
        # A ragged fp32 batch of odd width, backward.
        dict(name="ln_back_odd", op="ln", back=True, dtype="f32", T=9973, d=1531),
        # Scoring four single tokens against a 4096-token vocabulary.
        dict(name="loss_tokens", op="loss", back=False, dtype="bf16", S=1, T=4, d=512, V=4096,
             ignored=0.0),
        # Loss changes of eight jittered draws beside the clean pass, one 2048-token sequence.
        dict(name="loss_draws", op="loss", back=False, dtype="bf16", S=9, T=2048, d=512, V=4096,
             ignored=0.0),
        # Gradients of the base model's head, a batch of 8 x 2048 tokens.
        dict(name="loss_back_base", op="loss", back=True, dtype="bf16", S=1, T=16384, d=512,
             V=4096, ignored=0.0),
        # A wide model with a large vocabulary of odd size, a sixth of the tokens masked.
        dict(name="loss_back_large", op="loss", back=True, dtype="bf16", S=1, T=8192, d=2048,
             V=50257, ignored=0.17),
        # fp32 gradients of a small ragged batch, odd in every size.
        dict(name="loss_back_odd", op="loss", back=True, dtype="f32", S=1, T=777, d=301, V=5003,
             ignored=0.1),
        # Distilling from 64 stored logits a token, 32k vocabulary: the loss ...
        dict(name="distill_64", op="distill", back=False, dtype="bf16", S=1, T=4096, d=1024,
             V=32768, k=64),
        # ... and the gradients.
        dict(name="distill_back_64", op="distill", back=True, dtype="bf16", S=1, T=4096, d=1024,
             V=32768, k=64),
        # A short fp32 distillation, odd in every size.
        dict(name="distill_back_odd", op="distill", back=True, dtype="f32", S=1, T=65, d=129,
             V=1003, k=5),
    ]


MOST_NORM = 65536 * 2048        # elements of the largest listed norm
MOST_HEAD = 8192 * 50257 * 2048  # products of the largest listed head


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["ln", "loss", "distill"])
    back = rng.random() < 0.5
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "ln":
        d = _spread(rng, 32, 8192)
        if rng.random() < 0.5:
            d = (d + 7) // 8 * 8
        T = _spread(rng, 1, min(65536, MOST_NORM // d))
        return dict(op=op, back=back, dtype=dtype, T=T, d=d)
    d = _spread(rng, 32, 2048)
    if rng.random() < 0.7:
        d = min(2048, (d + 7) // 8 * 8)
    V = _spread(rng, 256, 50257)
    S = rng.choice([1, 1, 1, 3, 9]) if op == "loss" and not back else 1
    most = (MOST_HEAD // 8 if dtype == "f32" else MOST_HEAD) // 2
    T = _spread(rng, 1, max(1, min(16384 // S, most // (d * V * S))))
    if op == "loss":
        return dict(op=op, back=back, dtype=dtype, S=S, T=T, d=d, V=V,
                    ignored=rng.choice([0.0, 0.0, 0.1, 0.5]))
    return dict(op=op, back=back, dtype=dtype, S=1, T=T, d=d, V=V, k=min(V, _spread(rng, 1, 128)))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    T, d = case["T"], case["d"]
    if case["op"] == "ln":
        if case["back"]:  # gy, x, weight, mean, rstd in; gx, gweight, gbias out
            return {"bytes": 3 * e * T * d + 8 * T + 12 * d, "flops": 11 * T * d}
        return {"bytes": 2 * e * T * d + 8 * T + 8 * d, "flops": 8 * T * d}
    R, V = case["S"] * T, case["V"]
    side = 4 * T if case["op"] == "loss" else 8 * T * case["k"] + 4 * R * case["k"]
    inputs = e * (R * d + V * d) + side
    if case["back"]:  # the logits again, then each factor's gradient
        return {"bytes": inputs + 8 * R + e * (R * d + V * d), "flops": 6 * R * V * d}
    changes = 4 * (R - T)
    return {"bytes": inputs + 8 * R + changes, "flops": 2 * R * V * d}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    T, d = case["T"], case["d"]
    s = dict(case)
    if case["op"] == "ln":
        # A residual stream: rows of different scale, off zero, some channels larger.
        scale = torch.exp(0.3 * normal(T, 1)) * torch.exp(0.3 * normal(d))
        s["x"] = (normal(T, d) * scale + 0.5).to(dt)
        s["weight"] = 1.0 + 0.1 * normal(d)
        s["bias"] = 0.1 * normal(d)
        if case["back"]:
            s["gy"] = (normal(T, d) / math.sqrt(d)).to(dt)
            _, s["mean"], s["rstd"] = _plain_norm(s["x"], s["weight"], s["bias"])
        return s
    S, V = case["S"], case["V"]
    H = normal(1, T, d)
    if S > 1:  # the clean pass, then draws that jitter it
        H = torch.cat([H, H + 0.2 * normal(S - 1, T, d)])
    s["H"] = H.to(dt)[0] if S == 1 else H.to(dt)
    s["E"] = (normal(V, d) * (2.0 / math.sqrt(d))).to(dt)
    if case["op"] == "loss":
        # Frequent tokens have low ids.
        u = torch.rand(T, generator=g, device="cuda")
        s["targets"] = (V * u ** 3).to(torch.int32).clamp_(0, V - 1)
        skip = torch.rand(T, generator=g, device="cuda") < case["ignored"]
        s["targets"] = torch.where(skip, torch.full_like(s["targets"], -1), s["targets"])
        if case["back"]:
            valid = s["targets"] >= 0
            s["gloss"] = valid.float() / valid.sum().clamp(min=1)
            s["lse"] = _logits(s["H"], s["E"], 1.0).logsumexp(-1)
        return s
    # A teacher that saw a little more: its largest logits, sorted; some rows
    # were cut short (a nucleus), some are padding.
    k = case["k"]
    z = (s["H"].float() + 0.5 * normal(T, d)) @ s["E"].float().t()
    top = z.topk(k, dim=-1)
    count = torch.randint(1, k + 1, (T, 1), generator=g, device="cuda")
    whole = torch.rand(T, 1, generator=g, device="cuda")
    count = torch.where(whole < 0.7, torch.full_like(count, k), count)
    count = torch.where(whole > 0.95, torch.zeros_like(count), count)
    have = torch.arange(k, device="cuda") < count
    s["ids"] = torch.where(have, top.indices, torch.full_like(top.indices, -1)).to(torch.int32)
    s["teacher"] = top.values.contiguous()
    if case["back"]:
        x = _logits(s["H"], s["E"], TEMPER)
        s["lse"] = x.logsumexp(-1)
        s["student"] = x.gather(-1, s["ids"].long().clamp(min=0)) * have
        s["gloss"] = torch.full((T,), 1.0 / T, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _logits(H, E, scale):
    return (H.float() @ E.float().t()) * scale


def _plain_norm(x, weight, bias):
    v = x.float()
    mean = v.sum(-1) / v.shape[-1]
    c = v - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).sum(-1) / v.shape[-1] + EPS)
    return (c * rstd[:, None] * weight + bias).to(x.dtype), mean, rstd


def _plain_norm_back(s):
    x, gy, d = s["x"].float(), s["gy"].float(), s["d"]
    n = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gn = gy * s["weight"]
    a = gn.sum(-1, keepdim=True) / d
    b = (gn * n).sum(-1, keepdim=True) / d
    gx = (gn - a - n * b) * s["rstd"][:, None]
    return {"gx": gx.to(s["x"].dtype), "gweight": (gy * n).sum(0), "gbias": gy.sum(0)}


def _plain_lse(x):
    m = x.max(-1).values
    return m + (x - m[..., None]).exp().sum(-1).log()


def _plain_loss(s):
    x = _logits(s["H"], s["E"], 1.0)
    lse = _plain_lse(x)
    at = s["targets"].long().clamp(min=0).expand(x.shape[:-1])[..., None]
    loss = torch.where(s["targets"] >= 0, lse - x.gather(-1, at)[..., 0], torch.zeros_like(lse))
    out = {"loss": loss, "lse": lse}
    if s["S"] > 1:
        out["delta"] = loss[1:] - loss[0]
    return out


def _plain_factors(s, P, scale):
    """The head's gradients from those of its scaled logits."""
    P = P * scale
    return {"gH": (P @ s["E"].float()).to(s["H"].dtype),
            "gE": (P.t() @ s["H"].float()).to(s["E"].dtype)}


def _plain_loss_back(s):
    P = (_logits(s["H"], s["E"], 1.0) - s["lse"][:, None]).exp()
    rows = torch.arange(s["T"], device=P.device)
    P[rows, s["targets"].long().clamp(min=0)] -= 1.0
    w = torch.where(s["targets"] >= 0, s["gloss"], torch.zeros_like(s["gloss"]))
    return _plain_factors(s, P * w[:, None], 1.0)


def _teacher(s):
    """(which entries are there, the teacher's logarithms of them, its probabilities)"""
    have = s["ids"] >= 0
    z = torch.where(have, s["teacher"] * TEMPER, torch.full_like(s["teacher"], -1e30))
    m = z.max(-1, keepdim=True).values
    logq = z - m - torch.where(have, (z - m).exp(), torch.zeros_like(z)).sum(
        -1, keepdim=True).clamp(min=1e-30).log()
    return have, logq, torch.where(have, logq.exp(), torch.zeros_like(z))


def _plain_distill(s):
    x = _logits(s["H"], s["E"], TEMPER)
    lse = _plain_lse(x)
    have, logq, q = _teacher(s)
    student = torch.where(have, x.gather(-1, s["ids"].long().clamp(min=0)), torch.zeros_like(q))
    terms = torch.where(have, q * (logq - (student - lse[:, None])), torch.zeros_like(q))
    return {"loss": terms.sum(-1), "lse": lse, "student": student}


def _plain_distill_back(s):
    have, _, q = _teacher(s)
    P = (_logits(s["H"], s["E"], TEMPER) - s["lse"][:, None]).exp()
    P = torch.where(have.any(-1, keepdim=True), P, torch.zeros_like(P))
    P.scatter_add_(-1, s["ids"].long().clamp(min=0), -q)
    return _plain_factors(s, P * s["gloss"][:, None], TEMPER)


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "ln":
        if s["back"]:
            return _plain_norm_back(s)
        y, mean, rstd = _plain_norm(s["x"], s["weight"], s["bias"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if s["op"] == "loss":
        return _plain_loss_back(s) if s["back"] else _plain_loss(s)
    return _plain_distill_back(s) if s["back"] else _plain_distill(s)


def _run_own(s):
    import token_perturbation_estimator_gb300 as dust
    if s["op"] == "ln":
        if s["back"]:
            gx, gw, gb = dust.dust_layer_norm_grad(s["gy"], s["x"], s["mean"], s["rstd"],
                                                   s["weight"])
            return {"gx": gx, "gweight": gw, "gbias": gb}
        y, mean, rstd = dust.dust_layer_norm(s["x"], s["weight"], s["bias"], EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if s["op"] == "loss":
        if s["back"]:
            gH, gE = dust.dust_head_loss_grad(s["H"], s["E"], s["targets"], s["lse"], s["gloss"],
                                              gE_dtype=s["E"].dtype)
            return {"gH": gH, "gE": gE}
        if s["S"] > 1:
            loss, lse, delta = dust.dust_head_loss(s["H"], s["E"], s["targets"], changes=True)
            return {"loss": loss, "lse": lse, "delta": delta}
        loss, lse = dust.dust_head_loss(s["H"], s["E"], s["targets"])
        return {"loss": loss, "lse": lse}
    if s["back"]:
        gH, gE = dust.dust_distill_loss_grad(s["H"], s["E"], s["ids"], s["teacher"], s["lse"],
                                             s["student"], s["gloss"], TEMPER,
                                             gE_dtype=s["E"].dtype)
        return {"gH": gH, "gE": gE}
    loss, lse, student = dust.dust_distill_loss(s["H"], s["E"], s["ids"], s["teacher"], TEMPER)
    return {"loss": loss, "lse": lse, "student": student}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "ln":
        if not case["back"]:
            return _exact_norm(s)
        x, gy, w = s["x"].to(f), s["gy"].to(f), s["weight"].to(f)
        mean, rstd = s["mean"].to(f).unsqueeze(1), s["rstd"].to(f).unsqueeze(1)
        n = (x - mean) * rstd
        gn = gy * w
        # The Jacobian's projections: off the ones, off the normalised row.
        gx = gn - gn.mean(1, keepdim=True)
        gx = rstd * (gx - n * (gn * n).mean(1, keepdim=True))
        return {"gx": gx, "gweight": torch.einsum("td,td->d", gy, n), "gbias": gy.sum(0)}
    scale = TEMPER if case["op"] == "distill" else 1.0
    H = s["H"].to(f).reshape(-1, case["d"])
    E = s["E"].to(f)
    R, V = H.shape[0], case["V"]
    if case["op"] == "distill":
        q = torch.softmax((s["teacher"].to(f) * scale).masked_fill(s["ids"] < 0, -math.inf), 1)
        q = torch.nan_to_num(q, nan=0.0)  # a row without entries
    parts, gE = [], torch.zeros_like(E)
    step = max(1, (1 << 28) // V)
    for r0 in range(0, R, step):
        r1 = min(R, r0 + step)
        at = torch.arange(r0, r1, device=E.device) % case["T"]
        logp = scale * torch.einsum("rd,vd->rv", H[r0:r1], E)
        lse = torch.logsumexp(logp, 1)
        if case["op"] == "loss":
            y = s["targets"][at].long()
            want = torch.zeros(r1 - r0, V, dtype=f, device=E.device)
            want[y >= 0, y[y >= 0]] = 1.0
        else:
            want = torch.zeros(r1 - r0, V + 1, dtype=f, device=E.device)
            want.scatter_add_(1, s["ids"][at].long() % (V + 1), q[at])
            want = want[:, :V]
        if case["back"]:
            logp -= s["lse"][r0:r1].to(f)[:, None]
            G = (logp.exp_() * want.sum(1, keepdim=True) - want)
            G *= scale * s["gloss"][r0:r1].to(f)[:, None]
            gE += G.t() @ H[r0:r1]
            parts.append((G @ E,))
        elif case["op"] == "loss":
            parts.append((((lse[:, None] - logp) * want).sum(1), lse))
        else:
            t, ids = q[at], s["ids"][at]
            x = logp.gather(1, ids.long().clamp(min=0))
            x[ids < 0] = 0.0
            parts.append(((torch.xlogy(t, t) - t * (x - lse[:, None])).sum(1), lse, x))
    out = [torch.cat(p) for p in zip(*parts)]
    if case["back"]:
        return {"gH": out[0], "gE": gE}
    if case["op"] == "distill":
        return {"loss": out[0], "lse": out[1], "student": out[2]}
    shape = s["H"].shape[:-1]
    loss, lse = out[0].reshape(shape), out[1].reshape(shape)
    return {"loss": loss, "lse": lse, **({"delta": loss[1:] - loss[:1]} if case["S"] > 1 else {})}


def _exact_norm(s):
    x = s["x"].to(torch.float64)
    var, mean = torch.var_mean(x, dim=1, unbiased=False)
    rstd = torch.rsqrt(var + EPS)
    y = (x - mean[:, None]) * rstd[:, None] * s["weight"].double() + s["bias"].double()
    return {"y": y, "mean": mean, "rstd": rstd}
