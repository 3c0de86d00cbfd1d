"""The operators of a training step around the estimator and the head, as cases
to be measured.

Four operators: the gated feed-forward block ("gated": both projections, the
activation and the product; forward and backward), the norms of queries and
keys for each head with the position rotation ("rope"; forward and backward),
the clipped policy loss with a KL term on the head's per-token losses
("policy"; forward and backward), and clipping by the global gradient norm
("clip"). `run` computes a case once, in elementary torch operations (`own`
false) or through the library (`own` true); `exact` computes the same outputs
from the definitions in 64 bits.

A case's fields: op, back (backward pass), dtype ("bf16" or "f32") and sizes.
  gated   T tokens, d width, f hidden units, act ("silu", "gelu", "relu2")
  rope    T tokens, hq and hk heads of D values, rot of them rotated, layout
          ("halves": value i with i + rot / 2, "pairs": 2i with 2i + 1),
          fused (queries, keys and values lie in one row of the projection),
          padded (the share of tokens without a position)
  policy  S slices (the clean pass, then draws) of T tokens in n sequences,
          mean ("token": over all tokens, "sequence": of the sequences' means),
          per_token (advantages of tokens, or one for each sequence), ref (with
          the KL term), masked (the share of tokens that are not scored)
  clip    model: "sweep" (the 48 linear layers of the 12-layer sweep), or n
          tensors of about `size` values
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0           # of the rotation's wavelengths
LOW, HIGH, BETA = 0.2, 0.28, 0.04


def listed():
    return [
        # The block of one generated token: all latency and weights.
        dict(name="gated_token", op="gated", back=False, dtype="bf16", T=1, d=512, f=2048,
             act="silu"),
        # The up-projection of the 64 x 1024-token sweep, gated.
        dict(name="gated_sweep", op="gated", back=False, dtype="bf16", T=65536, d=512, f=2048,
             act="silu"),
        # Gradients of a wide model's block, 8 x 1024 tokens.
        dict(name="gated_back_wide", op="gated", back=True, dtype="bf16", T=8192, d=2048, f=8192,
             act="gelu"),
        # fp32 gradients of a small ragged batch, odd in every size.
        dict(name="gated_back_odd", op="gated", back=True, dtype="f32", T=777, d=301, f=1003,
             act="relu2"),
        # Queries and keys of one generated token.
        dict(name="rope_token", op="rope", back=False, dtype="bf16", T=1, hq=8, hk=8, D=64, rot=64,
             layout="halves", fused=True, padded=0.0),
        # Those of the sweep's 65536 tokens, as the 512 -> 1536 projection leaves them.
        dict(name="rope_sweep", op="rope", back=False, dtype="bf16", T=65536, hq=8, hk=8, D=64,
             rot=64, layout="halves", fused=True, padded=0.0),
        # Backward at width 4096 with shared keys, some padding.
        dict(name="rope_back_wide", op="rope", back=True, dtype="bf16", T=16384, hq=32, hk=8, D=128,
             rot=128, layout="halves", fused=False, padded=0.1),
        # fp32, odd sizes, neighbouring values rotated, half of each head left as it is.
        dict(name="rope_back_odd", op="rope", back=True, dtype="f32", T=1531, hq=6, hk=3, D=74,
             rot=36, layout="pairs", fused=False, padded=0.0),
        # Loss changes of the sweep's 32 draws beside the clean pass, 64 ragged sequences.
        dict(name="policy_draws", op="policy", back=False, dtype="f32", S=33, T=65536, n=64,
             mean="sequence", per_token=False, ref=True, masked=0.3),
        # Gradients of a short batch: a few sequences of a few hundred tokens, some of one.
        dict(name="policy_back_short", op="policy", back=True, dtype="f32", S=1, T=1531, n=7,
             mean="token", per_token=True, ref=True, masked=0.1),
        # All weight gradients of one pass over the 12-layer sweep.
        dict(name="clip_sweep", op="clip", back=False, dtype="f32", model="sweep"),
        # A few odd bf16 tensors.
        dict(name="clip_odd", op="clip", back=False, dtype="bf16", model="odd", n=5, size=30011),
    ]


MOST_GATED = 8192 * 2048 * 8192   # products of the largest listed block
MOST_ROPE = 16384 * 40 * 128      # values of the largest listed rotation
MOST_POLICY = 33 * 65536
MOST_CLIP = 12 * (512 * 1536 + 512 * 512 + 2 * 512 * 2048)


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "rope", "rope", "policy", "clip"])
    back = rng.random() < 0.5
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "gated":
        d, f = _spread(rng, 32, 4096), _spread(rng, 64, 8192)
        if rng.random() < 0.7:
            d, f = (d + 7) // 8 * 8, (f + 7) // 8 * 8
        most = MOST_GATED // (16 if dtype == "f32" else 2)
        T = _spread(rng, 1, max(1, min(65536, most // (d * f))))
        return dict(op=op, back=back, dtype=dtype, T=T, d=d, f=f,
                    act=rng.choice(["silu", "gelu", "relu2"]))
    if op == "rope":
        hk = rng.choice([1, 2, 3, 4, 8])
        hq = hk * rng.choice([1, 2, 4])
        D = rng.choice([32, 64, 64, 80, 128, 128, 256, _spread(rng, 8, 256)])
        rot = rng.choice([D // 2 * 2, D // 2 * 2, D // 4 * 2])
        most = MOST_ROPE // (2 if dtype == "f32" else 1)
        T = _spread(rng, 1, min(65536, most // ((hq + hk) * D)))
        return dict(op=op, back=back, dtype=dtype, T=T, hq=hq, hk=hk, D=D, rot=rot,
                    layout=rng.choice(["halves", "halves", "pairs"]), fused=rng.random() < 0.5,
                    padded=rng.choice([0.0, 0.1]))
    if op == "policy":
        S = 1 if back else rng.choice([1, 3, 9, 33])
        T = _spread(rng, 1, MOST_POLICY // max(S, 8))
        return dict(op=op, back=back, dtype="f32", S=S, T=T, n=_spread(rng, 1, max(1, T // 2)),
                    mean=rng.choice(["token", "sequence"]), per_token=rng.random() < 0.5,
                    ref=rng.random() < 0.7, masked=rng.choice([0.0, 0.1, 0.5]))
    n = _spread(rng, 1, 200)
    return dict(op=op, back=False, dtype=dtype, model="odd", n=n,
                size=_spread(rng, 1, min(MOST_CLIP // (2 * n), 1 << 24)))


def _layers(case):
    """The shapes of the tensors that are clipped."""
    if case["model"] == "sweep":
        return [(1536, 512), (512, 512), (2048, 512), (512, 2048)] * 12
    # Sizes around the case's, the first one as it is.
    return [(case["size"] if i == 0 else 1 + case["size"] * ((7 * i) % 11 + 3) // 10,)
            for i in range(case["n"])]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "gated":
        T, d, f = case["T"], case["d"], case["f"]
        if case["back"]:  # gh, X, Wg, Wu in; gX, gWg, gWu out; g and u once more
            return {"bytes": e * (T * f + 2 * T * d + 4 * f * d), "flops": 12 * T * d * f}
        return {"bytes": e * (T * d + 2 * f * d + T * f), "flops": 4 * T * d * f}
    if case["op"] == "rope":
        n = case["T"] * (case["hq"] + case["hk"]) * case["D"]
        side = case["T"] * (4 + 4 * case["rot"]) + 8 * case["D"]
        if case["back"]:  # gradients and inputs in, gradients and the weights' out
            return {"bytes": 3 * e * n + side + 8 * case["D"], "flops": 14 * n}
        return {"bytes": 2 * e * n + side, "flops": 8 * n}
    if case["op"] == "policy":
        R, T = case["S"] * case["T"], case["T"]
        inputs = 4 * (R + 2 * T) + (4 * T if case["ref"] else 0) + 4 * (
            T if case["per_token"] else case["n"])
        if case["back"]:
            return {"bytes": inputs + 4 * R, "flops": 20 * R}
        return {"bytes": inputs + 4 * R + 4 * (R - T), "flops": 20 * R}
    n = sum(math.prod(s) for s in _layers(case))
    return {"bytes": 2 * e * n, "flops": 3 * n}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case)
    if case["op"] == "gated":
        T, d, f = case["T"], case["d"], case["f"]
        # Normalised rows; weights as they are after some training.
        s["X"] = normal(T, d).to(dt)
        s["Wg"] = (normal(f, d) * (1.2 / math.sqrt(d))).to(dt)
        s["Wu"] = (normal(f, d) / math.sqrt(d)).to(dt)
        if case["back"]:
            s["gh"] = (normal(T, f) / math.sqrt(f)).to(dt)
        return s
    if case["op"] == "rope":
        T, hq, hk, D, rot = case["T"], case["hq"], case["hk"], case["D"], case["rot"]
        # Heads of different scale; in the projection's row the values follow the keys.
        if case["fused"]:
            row = (normal(T, hq + 2 * hk, D) * torch.exp(0.5 * normal(hq + 2 * hk, 1))).to(dt)
            s["q"], s["k"] = row[:, :hq], row[:, hq:hq + hk]
        else:
            s["q"] = (normal(T, hq, D) * torch.exp(0.5 * normal(hq, 1))).to(dt)
            s["k"] = (normal(T, hk, D) * torch.exp(0.5 * normal(hk, 1))).to(dt)
        s["wq"], s["wk"] = 1.0 + 0.2 * normal(D), 1.0 + 0.2 * normal(D)
        # Sequences of 1024 tokens, or one generated token somewhere in one.
        at = torch.arange(T, device="cuda") % 1024
        if T == 1:
            at = torch.randint(0, 1024, (1,), generator=g, device="cuda")
        pad = uniform(T) < case["padded"]
        s["positions"] = torch.where(pad, torch.full_like(at, -1), at).to(torch.int32)
        turns = BASE ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1))
        angle = torch.arange(1024, device="cuda", dtype=torch.float64)[:, None] * turns
        s["cosine"], s["sine"] = angle.cos().float(), angle.sin().float()
        if case["back"]:
            s["gyq"], s["gyk"] = normal(T, hq, D).to(dt), normal(T, hk, D).to(dt)
        return s
    if case["op"] == "policy":
        S, T, n = case["S"], case["T"], case["n"]
        # Lengths of every scale: borders at random, each sequence of one token at least.
        cuts = 1 + torch.randperm(max(T - 1, 1), generator=g, device="cuda")[:n - 1].sort().values
        ends = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)])
        s["seq_offsets"] = ends.to(torch.int32)
        nll = -torch.log(uniform(T).clamp(min=1e-4)) * 1.5
        # Samples of an earlier policy, scored by it and by the first one.
        s["old"] = (nll + 0.25 * normal(T)).contiguous()
        s["nll"] = torch.cat([nll[None], nll + 0.1 * normal(S - 1, T)]) if S > 1 else nll[None]
        s["ref"] = nll + 0.3 * normal(T) if case["ref"] else None
        s["beta"] = BETA if case["ref"] else 0.0
        s["advantages"] = normal(T if case["per_token"] else n)
        scored = uniform(T) >= case["masked"]
        s["targets"] = torch.where(scored, torch.randint(0, 4096, (T,), generator=g, device="cuda"),
                                   torch.full((T,), -1, device="cuda")).to(torch.int32)
        if case["back"]:
            s["gtotal"] = 0.5 + uniform(S)
        return s
    # Layers whose gradients differ in scale, and the buffers that the optimiser reads.
    s["grads"] = [(normal(*shape) * math.exp(0.7 * math.sin(i))).to(dt)
                  for i, shape in enumerate(_layers(case))]
    s["out"] = [torch.empty_like(t) for t in s["grads"]]
    s["max_norm"] = 1.0
    return s


# ---------------------------------------------------------------- plain forms

def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


GELU = 2.0 * math.sqrt(2.0 / math.pi)


def _act(x, act):
    if act == "relu2":
        r = x.clamp(min=0.0)
        return r * r
    return x * _sigmoid(x if act == "silu" else GELU * (x + 0.044715 * x * x * x))


def _act_slope(x, act):
    if act == "relu2":
        return 2.0 * x.clamp(min=0.0)
    if act == "silu":
        p = _sigmoid(x)
        return p * (1.0 + x * (1.0 - p))
    p = _sigmoid(GELU * (x + 0.044715 * x * x * x))
    return p + x * p * (1.0 - p) * GELU * (1.0 + 3 * 0.044715 * x * x)


def _plain_gated(s):
    X, Wg, Wu = s["X"].float(), s["Wg"].float(), s["Wu"].float()
    gate, up = X @ Wg.t(), X @ Wu.t()
    if not s["back"]:
        return {"h": (_act(gate, s["act"]) * up).to(s["X"].dtype)}
    gh = s["gh"].float()
    dG, dU = gh * up * _act_slope(gate, s["act"]), gh * _act(gate, s["act"])
    dt = s["X"].dtype
    return {"gX": (dG @ Wg + dU @ Wu).to(dt), "gWg": (dG.t() @ X).to(dt),
            "gWu": (dU.t() @ X).to(dt)}


def _rotate(m, s, sign):
    """The first `rot` values of each head turned by the token's angles."""
    rot = s["rot"]
    at = s["positions"].long().clamp(min=0)
    c, n = s["cosine"][at][:, None], sign * s["sine"][at][:, None]
    a, b = (m[..., :rot // 2], m[..., rot // 2:rot]) if s["layout"] == "halves" else (
        m[..., 0:rot:2], m[..., 1:rot:2])
    x, y = a * c - b * n, b * c + a * n
    turned = torch.cat([x, y], -1) if s["layout"] == "halves" else torch.stack([x, y], -1).flatten(-2)
    return torch.cat([turned, m[..., rot:]], -1)


def _unit(x):
    x = x.float()
    rstd = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    return x * rstd, rstd


def _plain_rope(x, w, s):
    n, _ = _unit(x)
    y = _rotate(n * w, s, 1.0)
    there = (s["positions"] >= 0)[:, None, None]
    return torch.where(there, y, torch.zeros_like(y)).to(x.dtype)


def _plain_rope_back(gy, x, w, s):
    n, rstd = _unit(x)
    gm = _rotate(gy.float(), s, -1.0)
    there = (s["positions"] >= 0)[:, None, None]
    gm = torch.where(there, gm, torch.zeros_like(gm))
    gn = gm * w
    gx = rstd * (gn - n * (gn * n).sum(-1, keepdim=True) / x.shape[-1])
    return gx.to(x.dtype), (gm * n).sum((0, 1))


def _policy_terms(s):
    """Per token: its weight in the mean, the ratio, whether it is clipped, its
    advantage, and how far it is from the reference. What decides whether a
    ratio is beyond its border, and the KL term's differences, in 64 bits."""
    T = s["T"]
    sizes = s["seq_offsets"].long().diff()
    seq = torch.repeat_interleave(torch.arange(s["n"], device=sizes.device), sizes, output_size=T)
    scored = s["targets"] >= 0
    adv = s["advantages"] if s["per_token"] else s["advantages"][seq]
    if s["mean"] == "token":
        weight = scored.double() / scored.sum().clamp(min=1)
    else:
        count = torch.zeros(s["n"], dtype=torch.float64, device=seq.device).index_add_(
            0, seq, scored.double())
        weight = scored / (count.clamp(min=1) * (count > 0).sum().clamp(min=1))[seq]
    step = s["old"].double() - s["nll"].double()
    clipped = torch.where(adv > 0, step > math.log1p(HIGH), (adv < 0) & (step < math.log1p(-LOW)))
    far = s["nll"].double() - s["ref"].double() if s["ref"] is not None else None
    return weight, scored, adv, step, clipped & scored, far


def _plain_policy(s):
    weight, scored, adv, step, clipped, far = _policy_terms(s)
    bound = torch.where(adv > 0, 1.0 + HIGH, 1.0 - LOW).float()
    loss = -torch.where(clipped, bound, step.float().exp()) * adv
    kl = torch.zeros_like(loss)
    if far is not None:
        kl = torch.where(scored, (far.expm1() - far).float(), kl)
        loss = loss + s["beta"] * kl
    loss = torch.where(scored, loss, torch.zeros_like(loss))
    out = {"loss": loss, "total": (weight * loss).sum(-1).float(),
           "kl": (weight * kl).sum(-1).float(), "clipped": (weight * clipped).sum(-1).float()}
    if s["S"] > 1:
        out["delta"] = loss[1:] - loss[0]
    return out


def _plain_policy_back(s):
    weight, scored, adv, step, clipped, far = _policy_terms(s)
    slope = torch.where(clipped, torch.zeros_like(adv), step.float().exp() * adv)
    if far is not None:
        slope = slope + s["beta"] * far.expm1().float()
    slope = torch.where(scored, slope, torch.zeros_like(slope))
    return {"gnll": s["gtotal"][:, None] * (weight.float() * slope)}


def _plain_clip(s):
    squares = torch.stack([t.double().square().sum() for t in s["grads"]])
    norm = squares.sum().sqrt()
    c = (s["max_norm"] / norm).clamp(max=1.0).float()
    return {"norm": norm.float().reshape(1), "out": [(t.float() * c).to(t.dtype) for t in s["grads"]]}


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "gated":
        return _plain_gated(s)
    if s["op"] == "rope":
        if not s["back"]:
            return {"yq": _plain_rope(s["q"], s["wq"], s), "yk": _plain_rope(s["k"], s["wk"], s)}
        gq, gwq = _plain_rope_back(s["gyq"], s["q"], s["wq"], s)
        gk, gwk = _plain_rope_back(s["gyk"], s["k"], s["wk"], s)
        return {"gq": gq, "gk": gk, "gwq": gwq, "gwk": gwk}
    if s["op"] == "policy":
        return _plain_policy_back(s) if s["back"] else _plain_policy(s)
    return _plain_clip(s)


def _run_own(s):
    import token_perturbation_estimator_gb300 as dust
    if s["op"] == "gated":
        act = {"silu": dust.SILU, "gelu": dust.GELU, "relu2": dust.RELU2}[s["act"]]
        if not s["back"]:
            return {"h": dust.dust_gated_up(s["X"], s["Wg"], s["Wu"], act)}
        gX, gWg, gWu = dust.dust_gated_up_grad(s["gh"], s["X"], s["Wg"], s["Wu"], act,
                                               gW_dtype=s["X"].dtype)
        return {"gX": gX, "gWg": gWg, "gWu": gWu}
    if s["op"] == "rope":
        layout = dust.ROPE_HALVES if s["layout"] == "halves" else dust.ROPE_PAIRS
        turn = (s["positions"], s["cosine"], s["sine"], EPS, layout)
        if not s["back"]:
            yq, yk = dust.dust_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], *turn)
            return {"yq": yq, "yk": yk}
        gq, gk, gwq, gwk = dust.dust_qk_norm_rope_grad(s["gyq"], s["gyk"], s["q"], s["k"], s["wq"],
                                                       s["wk"], *turn)
        return {"gq": gq, "gk": gk, "gwq": gwq, "gwk": gwk}
    if s["op"] == "policy":
        mean = dust.MEAN_TOKEN if s["mean"] == "token" else dust.MEAN_SEQUENCE
        rest = dict(ref=s["ref"], targets=s["targets"], clip_low=LOW, clip_high=HIGH,
                    beta=s["beta"], mean=mean)
        if s["back"]:
            return {"gnll": dust.dust_policy_loss_grad(s["nll"], s["old"], s["advantages"],
                                                       s["seq_offsets"], s["gtotal"], **rest)}
        out = dust.dust_policy_loss(s["nll"], s["old"], s["advantages"], s["seq_offsets"],
                                    changes=s["S"] > 1, **rest)
        return dict(zip(("loss", "total", "kl", "clipped", "delta"), out))
    norm, out = dust.dust_clip_grads(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, "out": out}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _exact_gated, "rope": _exact_rope, "policy": _exact_policy,
            "clip": _exact_clip}[case["op"]](s)


def _exact_gated(s):
    """Forward in 64 bits, the gradients by automatic differentiation, some rows
    at a time."""
    f64 = torch.float64
    Wg, Wu = s["Wg"].to(f64).requires_grad_(), s["Wu"].to(f64).requires_grad_()
    rows, parts = max(1, (1 << 28) // s["f"]), []
    for r in range(0, s["T"], rows):
        X = s["X"][r:r + rows].to(f64).requires_grad_()
        gate = torch.einsum("td,fd->tf", X, Wg)
        if s["act"] == "silu":
            a = torch.nn.functional.silu(gate)
        elif s["act"] == "gelu":
            a = torch.nn.functional.gelu(gate, approximate="tanh")
        else:
            a = torch.relu(gate) ** 2
        h = a * torch.einsum("td,fd->tf", X, Wu)
        if s["back"]:
            h.backward(s["gh"][r:r + rows].to(f64))
            parts.append(X.grad)
        else:
            parts.append(h.detach())
    if s["back"]:
        return {"gX": torch.cat(parts), "gWg": Wg.grad, "gWu": Wu.grad}
    return {"h": torch.cat(parts)}


def _exact_rope(s):
    """The rotation as a product of complex numbers, the gradients by automatic
    differentiation."""
    f64, rot = torch.float64, s["rot"]
    at = s["positions"].long()
    phase = torch.complex(s["cosine"].to(f64), s["sine"].to(f64))[at.clamp(min=0)][:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].to(f64).requires_grad_()
        w = s["w" + name].to(f64).requires_grad_()
        m = torch.nn.functional.rms_norm(x, (s["D"],), w, EPS)
        if s["layout"] == "halves":
            z = torch.complex(m[..., :rot // 2], m[..., rot // 2:rot]) * phase
            turned = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.complex(m[..., 0:rot:2], m[..., 1:rot:2]) * phase
            turned = torch.view_as_real(z).flatten(-2)
        y = torch.cat([turned, m[..., rot:]], -1) * (at >= 0)[:, None, None]
        if s["back"]:
            y.backward(s["gy" + name].to(f64))
            out["g" + name], out["gw" + name] = x.grad, w.grad
        else:
            out["y" + name] = y.detach()
    return {k: out[k] for k in (("gq", "gk", "gwq", "gwk") if s["back"] else ("yq", "yk"))}


def _exact_policy(s):
    f64 = torch.float64
    T = s["T"]
    nll = s["nll"].to(f64).requires_grad_()
    seq = torch.searchsorted(s["seq_offsets"][1:].long(), torch.arange(T, device=nll.device),
                             right=True)
    scored = (s["targets"] >= 0).to(f64)
    adv = (s["advantages"] if s["per_token"] else s["advantages"][seq]).to(f64)
    ratio = torch.exp(s["old"].to(f64) - nll)
    free, held = ratio * adv, ratio.clamp(1.0 - LOW, 1.0 + HIGH) * adv
    loss = torch.maximum(-free, -held)
    kl = torch.zeros_like(loss)
    if s["ref"] is not None:
        r = nll - s["ref"].to(f64)
        kl = torch.special.expm1(r) - r
        loss = loss + s["beta"] * kl
    loss, kl = loss * scored, kl * scored
    count = torch.bincount(seq, weights=scored, minlength=s["n"])

    def mean(v):
        if s["mean"] == "token":
            return v.sum(-1) / scored.sum().clamp(min=1.0)
        sums = torch.zeros(v.shape[0], s["n"], dtype=f64, device=v.device).index_add(1, seq, v)
        return (sums / count.clamp(min=1.0)).sum(-1) / (count > 0).sum().clamp(min=1)

    total = mean(loss)
    if s["back"]:
        total.backward(s["gtotal"].to(f64))
        return {"gnll": nll.grad}
    out = {"loss": loss.detach(), "total": total.detach(), "kl": mean(kl).detach(),
           "clipped": mean((free > held).to(f64) * scored).detach()}
    if s["S"] > 1:
        out["delta"] = out["loss"][1:] - out["loss"][:1]
    return out


def _exact_clip(s):
    norm = torch.sqrt(sum(torch.linalg.vector_norm(t.to(torch.float64)) ** 2 for t in s["grads"]))
    c = torch.clamp(s["max_norm"] / norm, max=1.0)
    return {"norm": norm.reshape(1), "out": [t.to(torch.float64) * c for t in s["grads"]]}
