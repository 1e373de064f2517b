"""Workloads of the training losses over label scores, and their plain forms.

The operators, each a loss with its gradient over rows of label scores
(logits [B, T, V]; position t of sequence b counts when t < lengths[b] and its
label is not negative):

  label_logprob    log-probabilities of given labels under a softmax per position
  policy_loss      clipped policy loss with a KL term on those log-probabilities
  policy_scores    the same, one ratio for each sampled segmentation (float64 scores)
  preference_loss  logistic loss on paired log-ratios of whole sequences
  preference_scores  the same on path scores (float64)
  distill_loss     KL divergence from a teacher's top labels

`run` computes them with elementary torch operations in float32 (per-position
scalars in float64) or, with `own`, through the library's entry points.
"""

from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_CLIP_LOW, _CLIP_HIGH, _KL = 0.2, 0.25, 0.05
_BETA, _MARGIN, _SMOOTH = 0.1, 0.05, 0.05


# ------------------------------------------------------------------- the cases
def _c(name, op, **kw):
    base = dict(name=name, op=op, B=1, T=1, V=1, dtype="f32", ragged=False, prompt=0, k=0,
                temperature=1.0, grad=True, per_token=False, lse=False, average=False)
    base.update(kw)
    return base


def listed():
    return [
        # per-position label scores of the speech batch: 39 labels, ragged lengths
        _c("logprob labels speech", "logprob", B=32, T=800, V=39, ragged=True),
        # scoring a batch with the reference model: no gradient, a large vocabulary
        _c("logprob scoring", "logprob", B=4, T=2048, V=131072, dtype="bf16", grad=False),
        # one new token a sequence: the smallest step, where latency counts
        _c("policy one token", "policy", B=16, T=1, V=32768, dtype="bf16"),
        # a ragged batch with prompts, token advantages, a vocabulary that is odd
        _c("policy ragged odd", "policy", B=16, T=512, V=50021, dtype="bf16", ragged=True,
           prompt=64, per_token=True),
        # the largest step: 8192 positions over a large vocabulary
        _c("policy largest", "policy", B=4, T=2048, V=131072, dtype="bf16"),
        # sampled segmentations of a batch: one score each
        _c("policy paths", "policy_paths", B=512),
        # two short pairs, half precision
        _c("preference small", "preference", B=4, T=96, V=16384, dtype="f16", ragged=True),
        # an ordinary batch of pairs
        _c("preference pairs", "preference", B=8, T=1024, V=65536, dtype="bf16", ragged=True,
           prompt=128),
        # pairs of segmentations by their path scores
        _c("preference paths", "preference_paths", B=4096),
        # the large-label batch: emissions learn from a teacher's eight best labels
        _c("distill labels large", "distill", B=8, T=10_000, V=128, k=8, temperature=2.0),
        # an ordinary distillation step
        _c("distill tokens", "distill", B=8, T=512, V=32768, dtype="bf16", k=64,
           temperature=1.5, ragged=True),
        # float32 logits, an odd vocabulary, long teacher lists with their true mass
        _c("distill f32 odd", "distill", B=2, T=1024, V=100003, k=128, lse=True),
    ]


def draw(rng):
    op = rng.choice(["logprob", "logprob", "policy", "policy", "policy", "preference", "preference",
                     "preference", "distill", "distill", "distill", "policy_paths",
                     "preference_paths"])
    if op in ("policy_paths", "preference_paths"):
        c = _c("", op, B=int(math.exp(rng.uniform(math.log(16), math.log(500_000)))))
        del c["name"]
        return c
    V = int(math.exp(rng.uniform(math.log(6), math.log(131072))))
    elements = math.exp(rng.uniform(math.log(2e5), math.log(3e8)))
    rows = max(2, min(200_000, int(elements / V)))
    B = int(math.exp(rng.uniform(0.0, math.log(min(64, rows)))))
    if op == "preference":
        B = max(2, B - B % 2)
    T = max(1, rows // B)
    c = _c("", op, B=B, T=T, V=V, dtype=rng.choice(["f32", "bf16", "bf16", "f16"]),
           ragged=rng.random() < 0.6, temperature=rng.choice([1.0, 1.0, 0.7, 2.0]),
           grad=op != "logprob" or rng.random() < 0.6, per_token=rng.random() < 0.5,
           prompt=rng.choice([0, 0, T // 4]), average=op == "preference" and rng.random() < 0.3)
    if op == "distill":
        c["k"] = int(math.exp(rng.uniform(0.0, math.log(min(V, 256)))))
        c["lse"] = rng.random() < 0.4
        c["prompt"] = 0
    del c["name"]
    return c


def _lengths(case):
    """Lengths of the case's sequences: T, or spread over (T/3, T] where ragged."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    span = T - T // 3
    return [T - (b * 7919 + 3 * (b % 5)) % span for b in range(B)]


def _counted(case):
    return sum(max(0, n - case["prompt"]) if n > case["prompt"] else 0 for n in _lengths(case))


def work(case):
    op, B = case["op"], case["B"]
    if op == "policy_paths":    # logp, old, ref, adv -> loss, kl, grad
        return {"bytes": 7 * 8 * B, "flops": 20 * B}
    if op == "preference_paths":  # four scores -> loss, two gradients
        return {"bytes": 7 * 8 * B, "flops": 20 * B}
    T, V, es = case["T"], case["V"], 4 if case["dtype"] == "f32" else 2
    rows = _counted(case)
    small = 4 * B * T * (2 if op == "logprob" else 4)
    if op == "distill":
        small = 4 * B * T + rows * (8 * case["k"] + (4 if case["lse"] else 0))
    return {"bytes": rows * V * es + (B * T * V * es if case["grad"] else 0) + small,
            "flops": rows * V * (8 if case["grad"] else 4)}


# ------------------------------------------------------------------ the inputs
def _rand(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * (int(seed) + 1))
    return g


def _off_corners(delta):
    """Log-ratios moved off the two corners of the clip, where the gradient of
    the loss has two values."""
    for corner in (math.log(1 - _CLIP_LOW), math.log(1 + _CLIP_HIGH)):
        near = (delta - corner).abs() < 2e-3
        delta = torch.where(near, torch.full_like(delta, corner + 4e-3), delta)
    return delta


def prepare(case, seed):
    g = _rand(seed)
    B, op = case["B"], case["op"]
    s = dict(case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    if op == "policy_paths":
        logp = -20.0 + 6.0 * normal(B, dtype=torch.float64)
        s["logp"] = logp
        s["old"] = logp - _off_corners(0.2 * normal(B, dtype=torch.float64))
        s["ref"] = logp + 0.3 * normal(B, dtype=torch.float64)
        s["adv"] = normal(B, dtype=torch.float64)
        s["out"] = {}
        return s
    if op == "preference_paths":
        s["chosen"] = 300.0 + 20.0 * normal(B, dtype=torch.float64)
        s["rejected"] = s["chosen"] - 4.0 + 8.0 * normal(B, dtype=torch.float64)
        s["ref_chosen"] = s["chosen"] + 3.0 * normal(B, dtype=torch.float64)
        s["ref_rejected"] = s["rejected"] + 3.0 * normal(B, dtype=torch.float64)
        s["out"] = {}
        return s
    T, V = case["T"], case["V"]
    dt = _DTYPES[case["dtype"]]
    lens = torch.tensor(_lengths(case), dtype=torch.int32)
    s["lengths"] = lens.cuda()
    small = V < 1024
    logits = normal(B, T, V, dtype=dt)
    if not small:
        logits *= 2.5
    s["logits"] = logits
    at = torch.arange(T, device="cuda")[None, :]
    counts = (at < s["lengths"][:, None].long()) & (at >= case["prompt"])
    labels = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int64)
    # the label that was drawn is a likely one
    lift = torch.full((B, T, 1), 1.5 if small else 9.0, device="cuda", dtype=dt)
    logits.scatter_add_(2, labels[..., None], lift)
    s["labels"] = torch.where(counts, labels, torch.full_like(labels, -1)).int()
    s["weight"] = torch.full((B // 2 if op == "preference" else B,), 1.0 / max(1, _counted(case)),
                             dtype=torch.float64, device="cuda")
    if op == "preference":
        s["weight"].fill_(2.0 / B)
    if dt is torch.float16:  # a scaled loss keeps small gradients inside the type's range
        s["weight"].fill_(16.0)
    if op == "logprob":
        s["grad_logp"] = -torch.rand((B, T), generator=g, device="cuda")
    elif op in ("policy", "preference"):
        now = torch.stack([torch.gather(logits[b], 1, labels[b][:, None])[:, 0].double()
                           / case["temperature"]
                           - torch.cat([(c.float() / case["temperature"]).logsumexp(-1).double()
                                        for c in logits[b].split(256)]) for b in range(B)])
        drift = torch.zeros(B, 1, dtype=torch.float64, device="cuda")
        if op == "preference":  # training has lifted the chosen labels and lowered the others
            drift[:B // 2], drift[B // 2:] = -0.3, 0.3
        s["ref"] = (now + drift + 0.2 * normal(B, T)).float()
        if op == "policy":
            s["old"] = (now - _off_corners(0.15 * normal(B, T))).float()
            s["adv"] = normal(B, T) if case["per_token"] else normal(B)
    elif op == "distill":
        k = case["k"]
        t_logits, ids, lse = [], [], []
        for b in range(B):
            for c in logits[b].split(max(1, 2 ** 25 // V)):
                t = 0.8 * c.float() + (0.5 if small else 1.0) * normal(*c.shape)
                top = t.topk(k, dim=-1)
                t_logits.append(top.values)
                ids.append(top.indices)
                lse.append((t / case["temperature"]).logsumexp(-1))
        s["teacher_logits"] = torch.cat(t_logits).view(B, T, k).contiguous()
        ids = torch.cat(ids).view(B, T, k)
        # lists are ragged: between half and all of the entries are used
        used = torch.randint((k + 1) // 2, k + 1, (B, T, 1), generator=g, device="cuda")
        s["teacher_ids"] = torch.where(torch.arange(k, device="cuda") < used, ids,
                                       torch.full_like(ids, -1)).int()
        s["teacher_lse"] = torch.cat(lse).view(B, T).contiguous() if case["lse"] else None
    s["out"] = {}
    return s


# -------------------------------------------------------------- the plain forms
def _softmax_parts(logits, temperature):
    """exp(z - max), its sum (float64) and the log-sum-exp (float64) of the rows."""
    z = logits.float() if temperature == 1.0 else logits.float() / temperature
    m = z.amax(-1, keepdim=True)
    e = (z - m).exp_()
    total = e.sum(-1).double()
    return z, e, total, m[..., 0].double() + total.log()


def _label_terms(s):
    labels = s["labels"].long()
    counts = labels >= 0
    y = labels.clamp_min(0)[..., None]
    z, e, total, lse = _softmax_parts(s["logits"], s["temperature"])
    logp = torch.where(counts, z.gather(-1, y)[..., 0].double() - lse, torch.zeros_like(lse))
    return counts, y, e, total, logp


def _label_gradient(s, e, total, y, counts, a):
    """a ([v = y] - q_v) / temperature, zero where the position does not count."""
    a = torch.where(counts, a, torch.zeros_like(a)) / s["temperature"]
    grad = e.mul_((-a / total).float()[..., None])
    grad.scatter_add_(-1, y, a.float()[..., None])
    return torch.where(counts[..., None], grad, torch.zeros_like(grad)).to(s["logits"].dtype)


def _plain_logprob(s):
    counts, y, e, total, logp = _label_terms(s)
    out = {"logp": logp.float(), "score": logp.sum(-1).float()}
    if s["grad"]:
        out["grad_logits"] = _label_gradient(s, e, total, y, counts, s["grad_logp"].double())
    return out


def _policy_terms(logp, old, ref, adv):
    r = (logp - old).exp()
    clipped = ((adv > 0) & (r > 1 + _CLIP_HIGH)) | ((adv < 0) & (r < 1 - _CLIP_LOW))
    d = ref - logp
    kl = d.exp() - d - 1
    pg = -torch.minimum(r * adv, r.clamp(1 - _CLIP_LOW, 1 + _CLIP_HIGH) * adv)
    slope = torch.where(clipped, torch.zeros_like(r), -adv * r) + _KL * (1 - d.exp())
    return pg + _KL * kl, kl, clipped, slope


def _plain_policy(s):
    counts, y, e, total, logp = _label_terms(s)
    adv = s["adv"].double() if s["per_token"] else s["adv"].double()[:, None]
    loss, kl, clipped, slope = _policy_terms(logp, s["old"].double(), s["ref"].double(), adv)
    zero = torch.zeros_like(loss)
    return {"loss": torch.where(counts, loss, zero).sum(-1).float(),
            "kl": torch.where(counts, kl, zero).sum(-1).float(),
            "clipped": (clipped & counts).sum(-1).int(),
            "logp": logp.float(),
            "grad_logits": _label_gradient(s, e, total, y, counts, slope * s["weight"][:, None])}


def _preference_terms(u):
    soft = lambda v: v.clamp_max(0).neg() + (-v.abs()).exp().log1p()  # -log sigma(v)
    loss = (1 - _SMOOTH) * soft(u) + _SMOOTH * soft(-u)
    slope = -(1 - _SMOOTH) / (1 + u.exp()) + _SMOOTH / (1 + (-u).exp())
    return loss, slope


def _plain_preference(s):
    counts, y, e, total, logp = _label_terms(s)
    ratio = torch.where(counts, logp - s["ref"].double(), torch.zeros_like(logp)).sum(-1)
    n = counts.sum(-1).clamp_min(1).double() if s["average"] else torch.ones_like(ratio)
    reward = _BETA * ratio / n
    P = s["B"] // 2
    loss, slope = _preference_terms(reward[:P] - reward[P:] - _MARGIN)
    w = _BETA * torch.cat([slope * s["weight"], -slope * s["weight"]]) / n
    return {"loss": loss.float(), "reward": reward.float(), "logp": logp.float(),
            "grad_logits": _label_gradient(s, e, total, y, counts, w[:, None].expand_as(logp))}


def _plain_distill(s):
    tau = s["temperature"]
    inside = torch.arange(s["T"], device="cuda")[None, :] < s["lengths"][:, None].long()
    ids = s["teacher_ids"].long()
    used = (ids >= 0) & inside[..., None]
    at = ids.clamp_min(0)
    z, e, total, lse = _softmax_parts(s["logits"], tau)
    logq = z.gather(-1, at).double() - lse[..., None]
    t = torch.where(used, s["teacher_logits"].double() / tau, torch.full_like(logq, -math.inf))
    if s["teacher_lse"] is not None:
        logt = t - s["teacher_lse"].double()[..., None]
    else:
        top = t.amax(-1, keepdim=True)
        top = torch.where(top > -math.inf, top, torch.zeros_like(top))
        logt = t - top - (t - top).exp().sum(-1, keepdim=True).log()
    p = torch.where(used, logt.exp(), torch.zeros_like(logt))
    terms = torch.where(p > 0, p * (logt - logq), torch.zeros_like(p))
    token = tau * tau * terms.sum(-1)
    w = torch.where(inside, tau * s["weight"][:, None], torch.zeros_like(token))
    grad = e.mul_((w * p.sum(-1) / total).float()[..., None])
    grad.scatter_add_(-1, at, (-w[..., None] * p).float())
    grad = torch.where(inside[..., None], grad, torch.zeros_like(grad))
    return {"loss": token.sum(-1).float(), "token_loss": token.float(),
            "grad_logits": grad.to(s["logits"].dtype)}


def _plain_policy_paths(s):
    loss, kl, clipped, slope = _policy_terms(s["logp"], s["old"], s["ref"], s["adv"])
    return {"loss": loss, "kl": kl, "grad_logp": slope}


def _plain_preference_paths(s):
    u = _BETA * ((s["chosen"] - s["rejected"]) - (s["ref_chosen"] - s["ref_rejected"])) - _MARGIN
    loss, slope = _preference_terms(u)
    return {"loss": loss, "grad_chosen": _BETA * slope, "grad_rejected": -_BETA * slope}


# ------------------------------------------------------- the library's own calls
def _own(s):
    from semi_markov_crf_b200 import semicrf
    op = s["op"]
    if op == "policy_paths":
        return semicrf.policy_scores(s["logp"], s["old"], s["adv"], ref_logp=s["ref"],
                                     clip_low=_CLIP_LOW, clip_high=_CLIP_HIGH, kl_coef=_KL,
                                     out=s["out"])
    if op == "preference_paths":
        return semicrf.preference_scores(s["chosen"], s["rejected"], s["ref_chosen"],
                                         s["ref_rejected"], beta=_BETA, margin=_MARGIN,
                                         smoothing=_SMOOTH, out=s["out"])
    if "ws" not in s:
        s["ws"] = semicrf.LossWorkspace(s["B"], s["T"], s["logits"].device)
    common = dict(temperature=s["temperature"], ws=s["ws"], out=s["out"])
    if op == "logprob":
        return semicrf.label_logprob(s["logits"], s["lengths"], s["labels"],
                                     grad_logp=s["grad_logp"] if s["grad"] else None,
                                     grad=s["grad"], **common)
    if op == "policy":
        return semicrf.policy_loss(s["logits"], s["lengths"], s["labels"], s["old"], s["adv"],
                                   ref_logp=s["ref"], clip_low=_CLIP_LOW, clip_high=_CLIP_HIGH,
                                   kl_coef=_KL, grad_loss=s["weight"], **common)
    if op == "preference":
        return semicrf.preference_loss(s["logits"], s["lengths"], s["labels"], ref_logp=s["ref"],
                                       beta=_BETA, margin=_MARGIN, smoothing=_SMOOTH,
                                       average=s["average"], grad_loss=s["weight"], **common)
    return semicrf.distill_loss(s["logits"], s["lengths"], s["teacher_ids"], s["teacher_logits"],
                                teacher_lse=s["teacher_lse"], grad_loss=s["weight"], **common)


def run(state):
    if own:
        return _own(state)
    return {"logprob": _plain_logprob, "policy": _plain_policy,
            "policy_paths": _plain_policy_paths, "preference": _plain_preference,
            "preference_paths": _plain_preference_paths,
            "distill": _plain_distill}[state["op"]](state)


# ----------------------------------------------- the definitions, in 64 bits
def _pair_loss(u):
    sig = torch.nn.functional.logsigmoid
    return -(1 - _SMOOTH) * sig(u) - _SMOOTH * sig(-u)


def _clip_loss(logp, old, ref, adv):
    r = torch.exp(logp - old)
    kl = torch.expm1(ref - logp) - (ref - logp)
    gain = torch.minimum(r * adv, torch.clamp(r, 1 - _CLIP_LOW, 1 + _CLIP_HIGH) * adv)
    return _KL * kl - gain, kl, gain


def exact(case, seed):
    """The losses from their definitions in float64, the gradients by automatic
    differentiation of those."""
    s = prepare(case, seed)
    op, B = case["op"], case["B"]
    if op == "policy_paths":
        x = s["logp"].clone().requires_grad_()
        loss, kl, _ = _clip_loss(x, s["old"], s["ref"], s["adv"])
        (grad,) = torch.autograd.grad(loss.sum(), x)
        return {"loss": loss.detach(), "kl": kl.detach(), "grad_logp": grad}
    if op == "preference_paths":
        c, r = (s[n].clone().requires_grad_() for n in ("chosen", "rejected"))
        loss = _pair_loss(_BETA * (c - r - s["ref_chosen"] + s["ref_rejected"]) - _MARGIN)
        gc, gr = torch.autograd.grad(loss.sum(), (c, r))
        return {"loss": loss.detach(), "grad_chosen": gc, "grad_rejected": gr}
    T, V, tau = case["T"], case["V"], case["temperature"]
    lens = _lengths(case)
    step = max(1, 2 ** 26 // V)
    grad = torch.zeros((B, T, V), dtype=torch.float64, device="cuda") if case["grad"] else None
    logp = torch.zeros((B, T), dtype=torch.float64, device="cuda")

    def spans():
        for b in range(B):
            for t0 in range(min(case["prompt"], lens[b]), lens[b], step):
                yield b, slice(t0, min(t0 + step, lens[b]))

    def log_q(b, at):
        x = s["logits"][b, at].double().requires_grad_()
        return x, torch.log_softmax(x / tau, -1)

    if op == "distill":
        token = torch.zeros_like(logp)
        for b, at in spans():
            x, lq = log_q(b, at)
            ids, t = s["teacher_ids"][b, at].long(), s["teacher_logits"][b, at].double() / tau
            t = t.masked_fill(ids < 0, -math.inf)
            whole = torch.logsumexp(t, -1) if s["teacher_lse"] is None else \
                s["teacher_lse"][b, at].double()
            p = torch.exp(t - whole[:, None])
            part = tau ** 2 * (torch.special.xlogy(p, p)
                               - p * lq.gather(-1, ids.clamp_min(0))).sum(-1)
            token[b, at] = part.detach()
            (grad[b, at],) = torch.autograd.grad((part * s["weight"][b]).sum(), x)
        return {"loss": token.sum(-1), "token_loss": token, "grad_logits": grad}

    def label_logp(b, at):
        x, lq = log_q(b, at)
        return x, lq.gather(-1, s["labels"][b, at].long()[:, None])[:, 0]

    out = {}
    if op == "preference":
        for b, at in spans():
            logp[b, at] = label_logp(b, at)[1].detach()
        rows = torch.stack([torch.zeros(2, dtype=torch.float64, device="cuda")] * B)
        for b, at in spans():
            rows[b, 0] += (logp[b, at] - s["ref"][b, at].double()).sum()
            rows[b, 1] += at.stop - at.start
        ratio = rows[:, 0].clone().requires_grad_()
        n = rows[:, 1].clamp_min(1) if case["average"] else torch.ones_like(ratio)
        reward = _BETA * ratio / n
        loss = _pair_loss(reward[:B // 2] - reward[B // 2:] - _MARGIN)
        (w,) = torch.autograd.grad((loss * s["weight"]).sum(), ratio)
        out.update(loss=loss.detach(), reward=reward.detach())
        for b, at in spans():
            x, lp = label_logp(b, at)
            (grad[b, at],) = torch.autograd.grad(lp.sum() * w[b], x)
    elif op == "policy":
        loss, kl = torch.zeros_like(logp), torch.zeros_like(logp)
        hit = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        for b, at in spans():
            x, lp = label_logp(b, at)
            adv = s["adv"][b, at].double() if case["per_token"] else s["adv"][b].double()
            part, k3, gain = _clip_loss(lp, s["old"][b, at].double(), s["ref"][b, at].double(), adv)
            (grad[b, at],) = torch.autograd.grad((part * s["weight"][b]).sum(), x)
            logp[b, at], loss[b, at], kl[b, at] = lp.detach(), part.detach(), k3.detach()
            free = torch.exp(lp - s["old"][b, at].double()) * adv
            hit[b, at] = (gain < free).int()
        out.update(loss=loss.sum(-1), kl=kl.sum(-1), clipped=hit.sum(-1).int())
    else:
        for b, at in spans():
            x, lp = label_logp(b, at)
            logp[b, at] = lp.detach()
            if case["grad"]:
                (grad[b, at],) = torch.autograd.grad((lp * s["grad_logp"][b, at].double()).sum(), x)
        out["score"] = logp.sum(-1)
    out["logp"] = logp
    if case["grad"]:
        out["grad_logits"] = grad
    return out
