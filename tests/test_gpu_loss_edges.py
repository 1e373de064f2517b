"""GPU tests of the training losses over label scores where their inputs or
sizes go wrong: masks of finite values, scores that are not numbers, positions
without a teacher's entries, ratios far from 1, the limits of the temperature,
calls without a gradient, very wide rows entry by entry.

Tolerances (u = 2^-24), entry by entry, against float64 statements on the GPU.
 * An exponential of the row: 2^-22 = 4 u for ex2, u |gap| each for the rounded
   argument and for the rounded factor log2(e) / temperature, gap the entry's
   distance from the row's maximum (natural logarithms).  Terms that matter in
   a sum have gap <= 22: 48 u.
 * The sum over a row: no term goes through more than V / 512 + 64 roundings
   (a thread's running sum over its share of a row, then the joins).  So a
   sum's relative error, the absolute one of its logarithm, is E(V) = (48 +
   V / 512 + 64 + 4) u, the 4 u for the logarithm itself.
 * A softmax entry q: E(V) + (4 + 2 gap) u, and 8 u for the factor, its
   division and the product: (E(V) + (12 + 2 gap) u) q.  Below 2^-126 of the
   maximum an exponential is 0.
 * log-probabilities: E(V), and u |logp| for the output's rounding.
 * Policy: with r the ratio and d = ref - logp, a term moves by |A| r (E + 12 u)
   and c |e^d - 1| (E + 8 u) <= 2 c (E + 8 u) for the d here.
 * Distillation: log p - log q is a difference of differences, 4 u of each
   (|t - t_max| + |x - x_max|) / temperature and of itself; p carries
   (2 |log p| + 28 + k / 32) u.
 * One rounding to the output's type: half a step of it, and half a subnormal
   step for float16.
"""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
# a width for each row kernel: lane groups, a CTA a row, rings, a cluster's
# rings, and beyond them
WIDTHS = [39, 1500, 5000, 40000, 140001, 600001]


def sum_error(V):
    return (48 + V / 512 + 64 + 4) * U


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _near(name, got, want, tol):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, name
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    off = ~same & ~((got - want).abs() <= tol)
    assert not bool(off.any()), (
        f"{name}: {int(off.sum())} of {off.numel()} off, first {got[off][0].item()} "
        f"for {want[off][0].item()}, tolerance {torch.as_tensor(tol, device=got.device).expand_as(got)[off][0].item():.3e}")


def _scores(B, T, V, dtype, seed, pad=0, scale=2.5):
    x = torch.full((B, T, V + pad), math.nan, dtype=dtype, device="cuda")[..., :V]
    x.copy_(scale * torch.randn(B, T, V, generator=_gen(seed), device="cuda"))
    return x


class Problem:
    """Scores [B, T, V] with everything that the four losses take beside them,
    their calls and their float64 statements."""

    lo, hi, c, beta = 0.2, 0.3, 0.1, 0.3

    def __init__(self, x, lens, tau=1.0, seed=0, k=20, lse=False, average=False, labels=None):
        self.x, self.tau, self.lens, self.average = x, tau, list(lens), average
        B, T, V = x.shape
        self.B, self.T, self.V, self.k = B, T, V, min(k, V)
        g = _gen(seed + 77)
        self.lengths = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.inside = torch.arange(T, device="cuda")[None] < self.lengths[:, None]
        if labels is None:
            labels = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32)
            if T > 2:
                labels[:, 1] = -1
        self.y = labels
        self.counts = self.inside & (labels >= 0)
        z = x.double()  # differences first: none is lost where a mask's value is all there is
        z = (z - z.amax(-1, keepdim=True)) / tau
        self.logq = torch.log_softmax(z, -1)
        self.gap = -z
        self.logp = torch.where(self.counts, self.logq.gather(-1, self.at())[..., 0],
                                torch.zeros((), dtype=torch.float64, device="cuda"))
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)
        delta = 0.3 * rnd(B, T)
        for corner in (math.log(1 - self.lo), math.log(1 + self.hi)):
            delta = torch.where((delta - corner).abs() < 2e-3, delta + 5e-3, delta)
        self.old = (self.logp - delta).float()
        self.ref = (self.logp + 0.2 * rnd(B, T)).float()
        self.adv = rnd(B, T).clamp(-2, 2).float()
        self.w = torch.rand(B, generator=g, device="cuda", dtype=torch.float64) + 0.5
        t = 0.8 * x.float() + tau * torch.randn(B, T, V, generator=g, device="cuda")
        top = torch.nan_to_num(t).topk(self.k, -1)
        self.ids, self.teacher = top.indices.int(), top.values.contiguous()
        self.ids[..., -1] = self.ids[..., 0]  # one label comes twice
        self.lse = None
        if lse:
            self.lse = ((self.teacher.double() / tau).logsumexp(-1) + 0.3).float()

    def at(self):
        return self.y.clamp_min(0).long()[..., None]

    def call(self, op, grad=True, accumulate=False, pad=0, fill=math.nan, **kw):
        from semi_markov_crf_b200 import semicrf
        if grad:
            buf = torch.full((self.B, self.T, self.V + pad), fill, dtype=self.x.dtype, device="cuda")
            buf = buf[..., :self.V]
            if accumulate:
                buf.copy_(torch.randn(buf.shape, generator=_gen(5), device="cuda"))
                self.start = buf.double()
            kw["out"] = {"grad_logits": buf}
        kw.update(temperature=self.tau, grad=grad, accumulate=accumulate)
        if op == "logprob":
            return semicrf.label_logprob(self.x, self.lengths, self.y,
                                         grad_logp=self.adv if grad else None, **kw)
        if op == "policy":
            return semicrf.policy_loss(self.x, self.lengths, self.y, self.old, self.adv,
                                       ref_logp=self.ref, clip_low=self.lo, clip_high=self.hi,
                                       kl_coef=self.c, grad_loss=self.w, **kw)
        if op == "preference":
            return semicrf.preference_loss(self.x, self.lengths, self.y, self.ref, beta=self.beta,
                                           margin=0.1, smoothing=0.1, average=self.average,
                                           grad_loss=self.w[:self.B // 2].contiguous(), **kw)
        return semicrf.distill_loss(self.x, self.lengths, self.ids, self.teacher,
                                    teacher_lse=self.lse, grad_loss=self.w, **kw)

    def check(self, op, out, accumulated=False, where=None):
        """Every output against its statement; `where` [B, T]: only these rows'
        gradients."""
        V, B, tau, E = self.V, self.B, self.tau, sum_error(self.V)
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        live = lambda v: torch.where(self.counts, v, zero)
        if op != "distill":
            _near("logp", out["logp"], self.logp, E + U * self.logp.abs())
        points = self.at()
        if op == "logprob":
            e = live(E + U * self.logp.abs())
            s = self.logp.sum(1)
            _near("score", out["score"], s, e.sum(1) + U * s.abs())
            a = live(self.adv.double())
            err, p = a.abs() * 2 * U, torch.ones_like(points, dtype=torch.float64)
        elif op == "policy":
            A, old, ref = self.adv.double(), self.old.double(), self.ref.double()
            r, d = (self.logp - old).exp(), ref - self.logp
            kl = live(torch.expm1(d) - d)
            free, cut = r * A, r.clamp(1 - self.lo, 1 + self.hi) * A
            term = live(-torch.minimum(free, cut)) + self.c * kl
            held = (cut < free) & self.counts
            ekl = live(2 * (E + 8 * U) + U * kl)
            e = live(A.abs() * r * (E + 12 * U)) + self.c * ekl + U * term.abs()
            _near("loss", out["loss"], term.sum(1), e.sum(1) + U * term.sum(1).abs())
            _near("kl", out["kl"], kl.sum(1), ekl.sum(1) + U * kl.sum(1))
            assert torch.equal(out["clipped"], held.sum(1).int())
            w = self.w[:, None]
            a = w * live(torch.where(held, zero, -free) - self.c * torch.expm1(d))
            err = w * (live(A.abs() * r * (E + 12 * U)) + self.c * live(2 * (E + 8 * U) + zero)) \
                + 2 * U * a.abs()
            p = torch.ones_like(points, dtype=torch.float64)
        elif op == "preference":
            ratio = live(self.logp - self.ref.double())
            n = self.counts.sum(1).clamp_min(1).double() if self.average else torch.ones(B).cuda()
            reward = self.beta * ratio.sum(1) / n
            e = self.beta * (live(E + U * ratio.abs())).sum(1) / n + U * reward.abs()
            _near("reward", out["reward"], reward, e + U * reward.abs())
            P = B // 2
            u = reward[:P] - reward[P:] - 0.1
            sig = torch.nn.functional.logsigmoid
            loss = -0.9 * sig(u) - 0.1 * sig(-u)
            eu = e[:P] + e[P:]
            _near("loss", out["loss"], loss, eu + U * loss.abs())
            slope = (-0.9 * torch.sigmoid(-u) + 0.1 * torch.sigmoid(u)) * self.beta * self.w[:P]
            a = live(torch.cat([slope, -slope])[:, None] / n[:, None])
            err = live((torch.cat([eu, eu]) * 0.25 * self.beta * torch.cat([self.w[:P]] * 2)
                        / n)[:, None] + zero) + 2 * U * a.abs()
            p = torch.ones_like(points, dtype=torch.float64)
        else:
            t = self.teacher.double() / tau
            if self.lse is None:
                logt = torch.log_softmax(t - t.amax(-1, keepdim=True), -1)
            else:
                logt = t - self.lse.double()[..., None]
            p, i = logt.exp(), self.ids.long()
            points = i
            gap = logt - self.logq.gather(-1, i)
            inside = lambda v: torch.where(self.inside, v, zero)
            token = inside(tau ** 2 * (p * gap).sum(-1))
            dt = t.amax(-1, keepdim=True) - t
            ep = (2 * dt + 28 + self.k / 32) * U
            e = p * (E + 4 * U * (dt + self.gap.gather(-1, i) + gap.abs())) + p * gap.abs() * ep
            e = inside(tau ** 2 * (e.sum(-1) + 40 * U)) + U * token.abs()
            _near("token_loss", out["token_loss"], token, e)
            _near("loss", out["loss"], token.sum(1), e.sum(1) + U * token.sum(1).abs())
            a = inside(-tau * tau * self.w[:, None] + 0 * token)  # over temperature, below
            err, p = a.abs() * 60 * U, p
        if "grad_logits" not in out:
            return
        dtype = self.x.dtype
        rows = (a != 0 if where is None else where & (a != 0)).nonzero()
        got = out["grad_logits"]
        for b, t in rows.tolist():
            q = self.logq[b, t].exp()
            f = a[b, t] / tau
            total = p[b, t].sum() if op == "distill" else 1.0
            # equal labels add up
            hot = torch.zeros_like(q).scatter_add_(0, points[b, t], p[b, t])
            want = f * (hot - total * q)
            tol = (f.abs() * total * q * (E + (12 + 2 * self.gap[b, t]) * U)
                   + f.abs() * hot * (80 + self.k / 32) * U
                   + err[b, t] / tau * (q * total + hot) + f.abs() * 2.0 ** -120)
            if op == "distill":
                dt = (self.teacher[b, t].amax() - self.teacher[b, t]).double() / tau
                tol += f.abs() * torch.zeros_like(q).scatter_add_(0, points[b, t],
                                                                  p[b, t] * 2 * dt * U)
            if accumulated:
                want = want + self.start[b, t]
                tol += 3 * U * (self.start[b, t].abs() + want.abs())
            _near(f"gradient of row {b}, {t}", got[b, t], want,
                  tol + HALF[dtype] * want.abs() + TINY[dtype])
        rest = (a == 0 if where is None else where & (a == 0)).nonzero()
        for b, t in rest.tolist():
            want = self.start[b, t] if accumulated else torch.zeros(V, dtype=torch.float64).cuda()
            _near(f"gradient of row {b}, {t}", got[b, t], want, 0.0)


OPS = ["logprob", "policy", "preference", "distill"]


MASKS = {torch.float32: [-1e9, -1e10, -1e30, torch.finfo(torch.float32).min],
         torch.bfloat16: [-1e10, -1e30, torch.finfo(torch.bfloat16).min],
         torch.float16: [-65504.0]}


@pytest.mark.parametrize("dtype", list(MASKS), ids=str)
@pytest.mark.parametrize("tau", [1.0, 2.0, 0.5, 1e-3, 1e3])
@pytest.mark.parametrize("V", WIDTHS)
def test_masks_of_finite_values(V, tau, dtype):
    """Masks of any finite value: labels of probability zero beside ordinary
    scores, wherever in the row they are; a row of nothing but the mask's value,
    however large, is uniform."""
    B, T = 2, 4
    labels = torch.tensor([[V - 1, 0, V // 2, V - 2], [V // 3, 1, V // 2, 0]], dtype=torch.int32).cuda()
    for value in MASKS[dtype]:
        x = _scores(B, T, V, dtype, V)
        x[0, 0, :V // 2] = value           # the first half
        x[0, 1, V // 2:] = value           # the last half
        x[0, 2, :V // 2] = value           # all but one
        x[0, 2, V // 2 + 1:] = value
        x[0, 3] = value                    # all of them
        x[1, 0] = -value                   # a uniform row far up
        x[1, 1, ::2] = value               # every second
        x[1, 2] += value / 4               # a common offset
        p = Problem(x, [T, T], tau=tau, seed=V, labels=labels, k=9)
        p.w *= 0.5
        for op in OPS:
            p.check(op, p.call(op))
        for op in OPS:
            p.check(op, p.call(op, grad=False))


@pytest.mark.parametrize("lse", [-math.inf, -100.0, math.nan, 3.0, None], ids=str)
@pytest.mark.parametrize("V", WIDTHS)
def test_positions_without_teacher_entries(V, lse):
    """No loss and no gradient where a position has no entry of positive
    probability, whatever the teacher's log-sum-exp and the scores are there; the
    other positions have theirs."""
    x = _scores(2, 4, V, torch.float32, V)
    x[1, 1, V // 2] = math.nan
    x[1, 2] = -math.inf
    empty = torch.tensor([[1, 1, 0, 1], [0, 1, 1, 0]], dtype=torch.bool, device="cuda")
    p = Problem(torch.nan_to_num(x), [4, 3], tau=1.5, seed=V, lse=lse is not None)
    p.x = x
    p.ids[0, 0] = -1
    p.teacher[0, 1] = -math.inf
    p.ids[0, 3, ::2] = -5
    p.teacher[0, 3, 1::2] = -math.inf
    p.teacher[0, 3, ::2] = math.nan     # behind an unused entry
    p.ids[1, 1:3] = -1
    if lse is not None:
        p.lse[empty] = lse
    for accumulate in (False, True):
        out = p.call("distill", accumulate=accumulate)
        assert bool((out["token_loss"][empty] == 0).all())
        start = p.start if accumulate else torch.zeros_like(out["grad_logits"]).double()
        assert torch.equal(out["grad_logits"][empty].double(), start[empty])
        assert torch.isfinite(out["loss"]).all()
        q = Problem(torch.nan_to_num(x), [4, 3], tau=1.5, seed=V, lse=lse is not None)
        want = q.call("distill", accumulate=accumulate)
        full = ~empty
        assert torch.equal(out["token_loss"][full], want["token_loss"][full])
        assert torch.equal(out["grad_logits"][full], want["grad_logits"][full])
    out = p.call("distill", grad=False)
    assert bool((out["token_loss"][empty] == 0).all())
    assert torch.isfinite(out["loss"]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("V", WIDTHS)
def test_scores_that_are_not_numbers(V, dtype):
    """A row that holds NaN or +inf, or nothing but -inf, makes its loss and its
    gradient row NaN, so that a step that looks for them sees them: for a pair
    the rows of both its sequences that count.  Other sequences and pairs keep
    theirs."""
    B, T = 6, 3
    clean = _scores(B, T, V, dtype, V)
    for value in ("nan", "inf", "none"):
        p = Problem(clean, [3, 2, 3, 3, 2, 3], seed=V)
        x = clean.clone()
        if value == "none":
            x[1, 0] = -math.inf
        else:
            x[1, 0, V // 3] = float(value)
        p.x = x
        for op in ("logprob", "policy", "distill"):
            out = p.call(op)
            g = out["grad_logits"]
            assert bool(torch.isnan(g[1, 0]).all()), (value, op)
            loss = out["score" if op == "logprob" else "loss"]
            assert torch.isnan(loss).tolist() == [False, True] + [False] * 4, (value, op)
            keep = torch.ones(B, T, dtype=torch.bool, device="cuda")
            keep[1, 0] = False
            assert torch.isfinite(g[keep]).all(), (value, op)
            bare = p.call(op, grad=False)
            assert torch.isnan(bare["score" if op == "logprob" else "loss"]).tolist() \
                == torch.isnan(loss).tolist(), (value, op)
        out = p.call("preference")
        assert torch.isnan(out["loss"]).tolist() == [False, True, False], value
        assert torch.isnan(out["reward"]).tolist() == [False, True] + [False] * 4, value
        g = out["grad_logits"]
        for b in (1, 4):
            for t in range(T):
                if bool(p.counts[b, t]):
                    assert bool(torch.isnan(g[b, t]).all()), (value, b, t)
                else:
                    assert not bool(g[b, t].any()), (value, b, t)
        for b in (0, 2, 3, 5):
            assert torch.isfinite(g[b]).all(), (value, b)
        # a malformed label takes the pair's gradient away all the same
        p.y = p.y.clone()
        p.y[4, 0] = V
        out = p.call("preference")
        assert torch.isnan(out["loss"]).tolist() == [False, True, False], value
        assert not bool(out["grad_logits"][[1, 4]].any()), value
        assert bool(out["grad_logits"][[0, 2]].any())


def test_a_reference_that_is_not_a_number():
    """A NaN in ref_logp reaches its pair's loss and gradient."""
    p = Problem(_scores(4, 3, 50, torch.float32, 1), [3, 3, 3, 3])
    p.ref[0, 0] = math.nan
    out = p.call("preference")
    assert torch.isnan(out["loss"]).tolist() == [True, False]
    g = out["grad_logits"]
    assert bool(torch.isnan(g[[0, 2]][:, [0, 2]]).all()) and torch.isfinite(g[[1, 3]]).all()
    p.ref[0, 1] = math.nan     # a position that does not count is not read
    p.ref[0, 0] = -1.0
    out = p.call("preference")
    assert torch.isfinite(out["loss"]).all() and torch.isfinite(out["grad_logits"]).all()


@pytest.mark.parametrize("V", [39, 1500, 5000, 40000, 140001])
def test_ratios_far_from_one(V):
    """Log-ratios beyond float32's exponentials: an advantage of 0 has no loss
    and no gradient, one that the clip holds the clip's loss, and a small one a
    finite product, as in 64 bits.  r A = e^D A with D known to E (logp's
    error): relative error E, and its rounding (by 2^-149 where the value is
    smaller than float32 holds)."""
    from semi_markov_crf_b200 import semicrf
    B, T = 6, 2
    x = _scores(B, T, V, torch.float32, V)
    p = Problem(x, [T] * B, seed=V)
    gap = torch.tensor([100.0, 500.0, 100.0, 95.0, -120.0, 80.0], device="cuda")[:, None]
    old = (p.logp - gap).float()
    adv = torch.tensor([0.0, 0.0, 1.0, -1e-20, 1.0, -1e-3], device="cuda")
    for hi in (0.3, math.inf):
        out = semicrf.policy_loss(x, p.lengths, p.y, old, adv, clip_low=0.2, clip_high=hi)
        r, A = (p.logp - old.double()).exp(), adv.double()[:, None]
        free, cut = r * A, r.clamp(0.8, 1 + hi) * A
        want = -torch.minimum(free, cut)
        if hi < math.inf:
            _near("loss", out["loss"].double(), want.sum(1),
                  (want.abs() * (sum_error(V) + 4 * U)).sum(1) + U * want.sum(1).abs() + 2.0 ** -149)
        else:
            keep = [0, 1, 3, 4, 5]   # e^100 is no float32
            _near("loss", out["loss"].double()[keep], want.sum(1)[keep],
                  ((want.abs() * (sum_error(V) + 4 * U)).sum(1) + U * want.sum(1).abs()
                   + 2.0 ** -149)[keep])
            assert out["loss"][2].item() == -math.inf
        held = cut < free
        assert torch.equal(out["clipped"], held.sum(1).int())
        slope = torch.where(held, torch.zeros_like(r), -free)
        q = p.logq.exp()
        hot = torch.zeros_like(q).scatter_(2, p.at(), 1.0)
        for b in (0, 1, 3, 4, 5) + ((2,) if hi < math.inf else ()):
            a = slope[b][:, None]
            w = a * (hot[b] - q[b])
            tol = a.abs() * (q[b] * (E2(V) + 2 * U * p.gap[b]) + hot[b] * E2(V)) + U * w.abs()
            _near(f"gradient {b}", out["grad_logits"][b], w, tol + 2.0 ** -120)


def E2(V):
    """A gradient entry's error relative to its softmax, its factor's with it."""
    return 2 * sum_error(V) + 24 * U


def test_path_ratios_far_from_one():
    """The same in float64, on paths."""
    from semi_markov_crf_b200 import semicrf
    t = lambda *v: torch.tensor(v, dtype=torch.float64).cuda()
    logp = t(-10.0, -10.0, -10.0, -10.0)
    old = t(-900.0, -900.0, -900.0, 900.0)
    out = semicrf.policy_scores(logp, old, t(0.0, 1.0, -0.0, 0.0))
    assert out["loss"].tolist() == [0.0, -1.2, 0.0, 0.0]
    assert out["grad_logp"].tolist() == [0.0, 0.0, 0.0, 0.0]
    out = semicrf.policy_scores(logp, old, t(0.0, 0.0, 0.0, 0.0), clip_high=math.inf)
    assert out["loss"].tolist() == [0.0] * 4 and out["grad_logp"].tolist() == [0.0] * 4
    out = semicrf.policy_scores(t(math.nan), t(-1.0), t(0.0))
    assert math.isnan(out["loss"][0]) and math.isnan(out["grad_logp"][0])


def test_preferences_of_impossible_labels():
    """A labelling of probability zero: u = -inf, where a smoothing of 1 leaves
    -log sigma(-u) = 0 alone, and u = +inf, where a smoothing of 0 leaves
    -log sigma(u) = 0; nothing is multiplied by a weight of 0."""
    from semi_markov_crf_b200 import semicrf
    inf = math.inf
    c = torch.tensor([-inf, inf, -inf, inf, -inf, inf], dtype=torch.float64).cuda()
    r = torch.zeros(6, dtype=torch.float64).cuda()
    for smoothing, loss, grad in ((1.0, [0.0, inf], [0.0, 1.0]), (0.0, [inf, 0.0], [-1.0, 0.0]),
                                  (0.5, [inf, inf], [-0.5, 0.5])):
        out = semicrf.preference_scores(c, r, beta=1.0, smoothing=smoothing)
        assert out["loss"].tolist() == loss * 3, smoothing
        assert out["grad_chosen"].tolist() == grad * 3, smoothing
    x = torch.zeros(2, 1, 10, device="cuda")
    x[0, 0, 3] = -inf
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    y = torch.full((2, 1), 3, dtype=torch.int32, device="cuda")
    out = semicrf.preference_loss(x, n, y, beta=1.0, smoothing=1.0)
    assert out["loss"].tolist() == [0.0] and not bool(out["grad_logits"].any())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("pads", [(0, 0), (1, 1), (0, 3)], ids=str)
def test_every_shape_of_short_rows(dtype, pads):
    """Every number of lanes, elements and kept teacher's entries is compiled and
    right: a row's log-probability within E + u |logp|, and its gradient, whose
    entries sum to 0: each is rounded by half a step of its size and the softmax's
    parts by E and 12 u, so that the sum is off by at most (half a step + E + 12 u)
    times the sum of their sizes, 2 at most (float16: V halves of a subnormal step
    more)."""
    from semi_markov_crf_b200 import semicrf
    n = torch.full((2,), 2, dtype=torch.int32, device="cuda")
    y = torch.tensor([[0, 1], [2, 0]], dtype=torch.int32, device="cuda")
    g = _gen(1)
    noise = torch.randn(2, 2, 2060, generator=g, device="cuda")
    teacher = torch.randn(2, 2, 300, generator=g, device="cuda")
    for V in list(range(3, 280)) + list(range(280, 2049, 17)) + [511, 512, 513, 1023, 1024, 1025, 1032, 2047, 2048]:
        x = torch.full((2, 2, V + pads[0]), math.nan, dtype=dtype, device="cuda")[..., :V]
        x.copy_(noise[..., :V])
        logq = torch.log_softmax(x.double(), -1)
        logp = logq.gather(-1, y.long()[..., None])[..., 0]
        E = sum_error(V)
        near = lambda o: bool(((o["logp"] - logp).abs() <= E + U * logp.abs()).all())
        buf = torch.empty(2, 2, V + pads[1], dtype=dtype, device="cuda")[..., :V]
        tol = 2 * (HALF[dtype] + E + 12 * U) + V * TINY[dtype]
        zero = lambda o: bool((o["grad_logits"].double().sum(-1).abs() <= tol).all())
        assert near(semicrf.label_logprob(x, n, y)), V
        pairs = semicrf.preference_loss(x, n, y, grad=False)
        assert near(pairs), V
        for call in (lambda o: semicrf.label_logprob(x, n, y, grad=True, out=o),
                     lambda o: semicrf.policy_loss(x, n, y, logp.float(), noise[:, 0, 0].clamp(-1, 1), out=o),
                     lambda o: semicrf.preference_loss(x, n, y, beta=1.0, out=o)):
            out = call({"grad_logits": buf.fill_(math.nan)})
            assert near(out) and zero(out), V
        for k in (1, 3, 5, 9, 17, 33, 65, 128, 129, 300):
            ids = (torch.arange(k, device="cuda", dtype=torch.int32) * 7 % V).expand(2, 2, k).contiguous()
            t = teacher[..., :k].contiguous()
            assert zero(semicrf.distill_loss(x, n, ids, t, out={"grad_logits": buf.fill_(math.nan)})), (V, k)
            bare = semicrf.distill_loss(x, n, ids, t, grad=False)["token_loss"].double()
            p = torch.softmax(t.double(), -1)
            gap = p.log() - logq.gather(-1, ids.long())
            want = (p * gap).sum(-1)
            e = E + ((28 + k / 32 + 12) * U * (1 + gap.abs()) * p * (1 + gap.abs())).sum(-1)
            assert bool(((bare - want).abs() <= e + 40 * U + U * want.abs()).all()), (V, k)


@pytest.mark.parametrize("V", [39, 5000, 40000])
def test_divergence_from_an_impossible_label(V):
    """A label of probability zero that the reference allows: the KL term is
    infinite, and without its weight the loss and the gradient are finite; one that
    only the reference excludes has an infinite term too."""
    from semi_markov_crf_b200 import semicrf
    x = _scores(3, 1, V, torch.float32, V)
    x[0, 0, 2] = -math.inf
    n = torch.ones(3, dtype=torch.int32, device="cuda")
    y = torch.full((3, 1), 2, dtype=torch.int32, device="cuda")
    old = torch.full((3, 1), -3.0, device="cuda")
    ref = torch.tensor([[-2.0], [-math.inf], [-3.0]], device="cuda")
    adv = torch.ones(3, device="cuda")
    for c in (0.0, 0.1):
        out = semicrf.policy_loss(x, n, y, old, adv, ref_logp=ref, kl_coef=c)
        assert out["kl"][:2].tolist() == [math.inf] * 2 and math.isfinite(out["kl"][2])
        assert out["logp"][0, 0].item() == -math.inf
        assert [math.isfinite(v) for v in out["loss"].tolist()] == [c == 0.0, c == 0.0, True]
        assert not torch.isnan(out["loss"]).any()
        if c == 0.0:
            assert torch.isfinite(out["grad_logits"]).all()
            assert not bool(out["grad_logits"][0].any())
    t = lambda *v: torch.tensor(v, dtype=torch.float64).cuda()
    inf = math.inf
    out = semicrf.policy_scores(t(-inf, -5.0, -2000.0), t(-3.0, -5.0, -2000.0), t(1.0, 1.0, 1.0),
                                t(-2.0, -inf, 0.0), kl_coef=0.5)
    assert out["kl"].tolist() == [inf, inf, inf] and out["loss"].tolist() == [inf, inf, inf]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("op", OPS)
def test_every_gradient_entry(op, dtype):
    """Each entry of the gradient, written over NaN, at a width of every kernel:
    the relative error of its softmax, not only that of its row's weight."""
    for V, pad in ((39, 0), (150, 1), (1000, 0), (1999, 1), (2048, 8), (3001, 3), (8192, 0), (9001, 5),
                   (20000, 0), (33001, 0), (131072, 0), (140000, 3), (300001, 0), (600001, 0),
                   (900001, 1)):
        p = Problem(_scores(4, 3, V, dtype, V, pad), [3, 0, 1, 3], tau=1.25, seed=V, k=40,
                    lse=V % 2 == 1, average=V % 3 == 0)
        p.check(op, p.call(op, pad=pad))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("V", [150, 3001, 40000, 140001, 600001])
def test_gradient_rows_on_other_boundaries(V, op):
    """Scores and gradient rows that lie differently in their 16-byte vectors."""
    for dtype in (torch.float32, torch.bfloat16):
        p = Problem(_scores(2, 3, V, dtype, V, 3), [3, 2], seed=V)
        p.check(op, p.call(op, pad=2))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("V", [39, 1500, 5000, 8200, 40000, 140001, 600001])
def test_accumulated_entries(V, op):
    p = Problem(_scores(4, 3, V, torch.float32, V), [3, 0, 2, 3], tau=0.8, seed=V)
    p.check(op, p.call(op, accumulate=True), accumulated=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("op", OPS)
def test_losses_without_a_gradient(op, dtype):
    for B, T in ((4, 3), (4, 1), (2, 300)):
        for V, pad in ((6, 0), (39, 1), (128, 0), (777, 0), (2048, 0), (2049, 0), (5000, 3), (12000, 0),
                       (40000, 1), (131072, 0), (300001, 0), (600001, 0)):
            if T == 300 and V > 12000:
                continue
            lens = [T, T // 2, T, T - 1][:B]
            p = Problem(_scores(B, T, V, dtype, V, pad), lens, tau=1.25, seed=V, k=30, lse=V % 2 == 1)
            out = p.call(op, grad=False)
            assert "grad_logits" not in out
            p.check(op, out)


@pytest.mark.parametrize("tau", [1e-3, 0.02, 50.0, 1e3])
@pytest.mark.parametrize("op", OPS)
def test_temperatures_to_their_limits(op, tau):
    """Scores whose differences matter at the temperature, and scores of
    ordinary size."""
    for V in (39, 1500, 5000, 40000, 140001, 600001):
        for dtype in (torch.float32, torch.bfloat16):
            for scale in (2.5, 2.5 * tau):
                p = Problem(_scores(2, 3, V, dtype, V, scale=scale), [3, 2], tau=tau, seed=V)
                p.check(op, p.call(op))
                p.check(op, p.call(op, grad=False))
