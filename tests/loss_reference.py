"""Plain float64 statements of the training losses over label scores, on the
CPU, one position at a time in the order of their definitions.  Nothing of the
package is used."""

import math

import torch


def _counted(lengths, labels, b, t):
    return t < int(lengths[b]) and (labels is None or int(labels[b, t]) >= 0)


def _row(logits, b, t, tau):
    x = logits[b, t].double()
    z = (x - x.max()) / tau  # only differences of z are used: none is lost at the type's lowest value
    lse = z.exp().sum().log()
    return z, lse, (z - lse).exp()


def _label_rows(logits, lengths, labels, tau):
    B, T, V = logits.shape
    logp = torch.zeros(B, T, dtype=torch.float64)
    base = torch.zeros(B, T, V, dtype=torch.float64)  # d logp / d logits
    for b in range(B):
        for t in range(T):
            if _counted(lengths, labels, b, t):
                z, lse, q = _row(logits, b, t, tau)
                y = int(labels[b, t])
                logp[b, t] = z[y] - lse
                base[b, t] = -q / tau
                base[b, t, y] += 1.0 / tau
    return logp, base


def label_logprob(logits, lengths, labels, tau=1.0, grad_logp=None):
    logp, base = _label_rows(logits, lengths, labels, tau)
    a = torch.ones_like(logp) if grad_logp is None else grad_logp.double()
    return {"logp": logp, "score": logp.sum(1), "grad_logits": a[..., None] * base,
            "slope": a}


def policy_term(logp, old, adv, ref, lo, hi, c):
    r = math.exp(logp - old)
    free, cut = r * adv, min(max(r, 1 - lo), 1 + hi) * adv
    loss, slope = -min(free, cut), 0.0 if cut < free else -free
    kl = 0.0
    if ref is not None:
        d = ref - logp
        kl = math.expm1(d) - d
        loss += c * kl
        slope -= c * math.expm1(d)
    return loss, kl, slope, cut < free


def policy_loss(logits, lengths, labels, old, adv, ref=None, lo=0.2, hi=0.2, c=0.0, tau=1.0,
                w=None):
    B, T, _ = logits.shape
    logp, base = _label_rows(logits, lengths, labels, tau)
    loss, kl = torch.zeros(B, dtype=torch.float64), torch.zeros(B, dtype=torch.float64)
    clipped = torch.zeros(B, dtype=torch.int32)
    slope = torch.zeros(B, T, dtype=torch.float64)
    for b in range(B):
        for t in range(T):
            if _counted(lengths, labels, b, t):
                a = float(adv[b, t] if adv.dim() == 2 else adv[b])
                l, k, s, hit = policy_term(float(logp[b, t]), float(old[b, t]), a,
                                           None if ref is None else float(ref[b, t]), lo, hi, c)
                loss[b] += l
                kl[b] += k
                clipped[b] += hit
                slope[b, t] = s * (1.0 if w is None else float(w[b]))
    return {"loss": loss, "kl": kl, "clipped": clipped, "logp": logp, "slope": slope,
            "grad_logits": slope[..., None] * base}


def preference_term(u, smoothing):
    soft = lambda v: max(-v, 0.0) + math.log1p(math.exp(-abs(v)))  # -log sigmoid(v)
    sig = lambda v: 1 / (1 + math.exp(-v)) if v >= 0 else math.exp(v) / (1 + math.exp(v))
    return ((1 - smoothing) * soft(u) + smoothing * soft(-u),
            -(1 - smoothing) * sig(-u) + smoothing * sig(u))


def preference_loss(logits, lengths, labels, ref=None, beta=0.1, margin=0.0, smoothing=0.0,
                    average=False, tau=1.0, w=None):
    B, T, _ = logits.shape
    logp, base = _label_rows(logits, lengths, labels, tau)
    reward = torch.zeros(B, dtype=torch.float64)
    n = torch.ones(B, dtype=torch.float64)
    for b in range(B):
        at = [t for t in range(T) if _counted(lengths, labels, b, t)]
        total = sum((float(logp[b, t]) - (0.0 if ref is None else float(ref[b, t])) for t in at), 0.0)
        if average:
            n[b] = max(1, len(at))
        reward[b] = beta * total / n[b]
    P = B // 2
    loss = torch.zeros(P, dtype=torch.float64)
    slope = torch.zeros(B, T, dtype=torch.float64)
    for i in range(P):
        loss[i], s = preference_term(float(reward[i] - reward[P + i]) - margin, smoothing)
        s *= beta * (1.0 if w is None else float(w[i]))
        slope[i] = s / n[i]
        slope[P + i] = -s / n[P + i]
    return {"loss": loss, "reward": reward, "logp": logp, "slope": slope,
            "grad_logits": slope[..., None] * base}


def distill_loss(logits, lengths, ids, teacher, lse=None, tau=1.0, w=None):
    B, T, V = logits.shape
    token = torch.zeros(B, T, dtype=torch.float64)
    grad = torch.zeros(B, T, V, dtype=torch.float64)
    slope = torch.zeros(B, T, dtype=torch.float64)
    for b in range(B):
        for t in range(T):
            if not _counted(lengths, None, b, t):
                continue
            z, zlse, q = _row(logits, b, t, tau)
            use = [j for j in range(ids.shape[2])
                   if int(ids[b, t, j]) >= 0 and float(teacher[b, t, j]) > -math.inf]
            if not use:
                continue
            tz = torch.tensor([float(teacher[b, t, j]) / tau for j in use], dtype=torch.float64)
            top = tz.max()
            whole = float(lse[b, t]) if lse is not None else top + (tz - top).exp().sum().log()
            logt = tz - whole
            p = logt.exp()
            wb = 1.0 if w is None else float(w[b])
            for j, lt, pj in zip(use, logt, p):
                y = int(ids[b, t, j])
                if pj > 0:
                    token[b, t] += tau ** 2 * pj * (lt - (z[y] - zlse))
                grad[b, t, y] -= wb * tau * pj
            grad[b, t] += wb * tau * p.sum() * q
            slope[b, t] = wb * tau * tau * p.sum()
    return {"loss": token.sum(1), "token_loss": token, "grad_logits": grad, "slope": slope}
