"""GPU tests of the training losses over label scores (label_logprob,
policy_loss, preference_loss, distill_loss and the path forms) against plain
float64 statements of the same formulas.

Tolerances, from the arithmetic (u = 2^-24, half a step of float32).
 * An exponential ex2(fma(x, sl, -m sl)): 2^-22 for ex2 and u |argument| ln 2
   for the rounded argument; terms that matter have |argument| <= 32: 2^-22 +
   22 u = 26 u.  A row's sum: at most V / 32 + 15 rounded additions per term
   for the sizes here (each <= u), so (26 + V / 32 + 15) u relative, which is
   the absolute error of the log-sum-exp; the factor log2(e) / temperature is
   rounded once, u |z - m| <= 40 u more.  LSE(V) = (81 + V / 32) u.
 * logp: LSE(V) + u |logp| for its own rounding.
 * A gradient entry a ([v = y] - q): |a| (2 LSE(V) + 8 u) for q, its factor
   and the subtraction, half a step of the output type relative to the entry,
   and a's own error: exponential of a difference of log-probabilities, which
   adds |a| (LSE(V) + 4 u), times (1 + c e^|d|) <= 4 for the policy's terms.
 * A sum over n positions of terms with error e: n e + u |sum|.
"""

import math
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import loss_reference as ref
import oracle
from semi_markov_crf_b200 import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # half a subnormal step
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def lse_tol(V):
    return (81 + V / 32) * U


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _logits(B, T, V, dtype, seed, pad=0, scale=2.5):
    """[B, T, V] scores on the CPU and their device copy, rows V + pad apart
    and the padding NaN."""
    x = (scale * torch.randn(B, T, V, generator=_gen(seed))).to(dtype)
    d = torch.full((B, T, V + pad), float("nan"), dtype=dtype, device="cuda")[..., :V]
    d.copy_(x)
    return x, d


def _labels(B, T, V, lengths, seed, holes=True):
    y = torch.randint(0, V, (B, T), generator=_gen(seed + 1), dtype=torch.int32)
    if holes and T > 2:
        y[:, ::3] = torch.where(torch.rand(B, (T + 2) // 3, generator=_gen(seed + 2)) < 0.5,
                                torch.full_like(y[:, ::3], -1), y[:, ::3])
    for b in range(B):
        y[b, lengths[b]:] = 10 ** 9  # never read
    return y


def _check(name, got, want, tol):
    got = got.double().cpu()
    want = want.double()
    assert got.shape == want.shape, name
    assert torch.equal(torch.isnan(got), torch.isnan(want)), name
    same = got == want  # infinities
    err = torch.where(same | torch.isnan(want), torch.zeros_like(got), (got - want).abs())
    tol = torch.as_tensor(tol, dtype=torch.float64).expand_as(err)
    over = (err > 0) & ~(err <= tol)
    assert not over.any(), (f"{name}: {int(over.sum())} values off, error {err[over].max().item():.3e} "
                            f"against {tol[over].min().item():.3e}")


def _check_grad(got, want, slope, dtype, V, tau, factor=1.0):
    a = slope.abs()[..., None] / tau
    tol = a * (factor * (3 * lse_tol(V) + 12 * U)) + HALF[dtype] * want.abs() + TINY[dtype]
    _check("grad_logits", got, want, tol)


def _case(B, T):
    lengths = [T, 0, 1, max(1, T - 2), T // 2, T][:B]
    return lengths, torch.tensor(lengths, dtype=torch.int32)


SIZES = [(3, 7, 1), (4, 5, 2), (5, 9, 6), (4, 6, 39), (4, 5, 64), (4, 5, 128), (4, 5, 129),
         (5, 3, 257), (4, 3, 1000), (4, 3, 1024), (4, 3, 2049), (4, 2, 4096), (4, 2, 8191),
         (2, 2, 20001), (2, 1, 32768), (2, 1, 65537), (2, 1, 131072), (2, 1, 300001)]
LAYOUTS = [(torch.float32, 0), (torch.bfloat16, 0), (torch.float16, 0), (torch.float32, 3),
           (torch.bfloat16, 5)]


@pytest.mark.parametrize("dtype,pad", LAYOUTS, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("B,T,V", SIZES)
def test_label_logprob(B, T, V, dtype, pad):
    from semi_markov_crf_b200 import semicrf
    lens, lengths = _case(B, T)
    tau = 0.7 if V % 2 else 1.0
    x, d = _logits(B, T, V, dtype, V, pad)
    y = _labels(B, T, V, lens, V)
    a = torch.randn(B, T, generator=_gen(3))
    want = ref.label_logprob(x, lens, y, tau, a)
    ws = semicrf.LossWorkspace(B, T)
    out = semicrf.label_logprob(d, lengths.cuda(), y.cuda(), tau, a.cuda(), grad=True, ws=ws)
    assert semicrf.get_status(ws) == 0
    _check("logp", out["logp"], want["logp"], lse_tol(V) + U * want["logp"].abs())
    _check("score", out["score"], want["score"],
           T * lse_tol(V) + 2 * U * want["logp"].abs().sum(1))
    _check_grad(out["grad_logits"], want["grad_logits"], want["slope"], dtype, V, tau)
    alone = semicrf.label_logprob(d, lengths.cuda(), y.cuda(), tau)
    assert "grad_logits" not in alone
    _check("logp without a gradient", alone["logp"], want["logp"],
           lse_tol(V) + U * want["logp"].abs())


def _policy_inputs(logits, lens, y, tau, seed, spread=0.3):
    g = _gen(seed)
    B, T, _ = logits.shape
    now, _ = ref._label_rows(logits, lens, y, tau)
    delta = spread * torch.randn(B, T, generator=g, dtype=torch.float64)
    for corner in (math.log(0.8), math.log(1.3)):  # off the corners of the clip
        delta = torch.where((delta - corner).abs() < 1e-3, delta + 3e-3, delta)
    old = (now - delta).float()
    return old, (now + 0.2 * torch.randn(B, T, generator=g, dtype=torch.float64)).float()


def _policy_tolerances(out, want, lens, V, adv_max, c):
    n = torch.tensor([max(1, v) for v in lens], dtype=torch.float64)
    # term: r A + c k; r <= 4 here, d(term) <= (4 |A| + 4 c) d(logp), and roundings of the parts
    e = (4 * adv_max + 4 * abs(c)) * (lse_tol(V) + 6 * U)
    _check("logp", out["logp"], want["logp"], lse_tol(V) + U * want["logp"].abs())
    _check("loss", out["loss"], want["loss"], n * e + U * want["loss"].abs())
    _check("kl", out["kl"], want["kl"], n * 4 * (lse_tol(V) + 4 * U) + U * want["kl"].abs())
    assert torch.equal(out["clipped"].cpu(), want["clipped"])


@pytest.mark.parametrize("dtype,pad", LAYOUTS, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("B,T,V", SIZES)
def test_policy_loss(B, T, V, dtype, pad):
    from semi_markov_crf_b200 import semicrf
    lens, lengths = _case(B, T)
    tau = 1.0 if V % 2 else 1.3
    x, d = _logits(B, T, V, dtype, V + 1, pad)
    y = _labels(B, T, V, lens, V + 5)
    old, reference = _policy_inputs(x, lens, y, tau, V)
    per_token = V % 3 == 0
    adv = torch.randn((B, T) if per_token else (B,), generator=_gen(9)).clamp(-2, 2)
    w = torch.rand(B, generator=_gen(10), dtype=torch.float64) + 0.5
    want = ref.policy_loss(x, lens, y, old, adv, reference, 0.2, 0.3, 0.1, tau, w)
    ws = semicrf.LossWorkspace(B, T)
    out = semicrf.policy_loss(d, lengths.cuda(), y.cuda(), old.cuda(), adv.cuda(),
                              ref_logp=reference.cuda(), clip_low=0.2, clip_high=0.3, kl_coef=0.1,
                              temperature=tau, grad_loss=w.cuda(), ws=ws)
    assert semicrf.get_status(ws) == 0
    _policy_tolerances(out, want, lens, V, 2.0, 0.1)
    # the slope's own scale: |A| r + c |1 - e^d|, not the slope after cancellation
    scale = w[:, None] * (2 * (want["logp"] - old.double()).exp() + 0.1) * (want["slope"] != 0)
    _check_grad(out["grad_logits"], want["grad_logits"], scale, dtype, V, tau, 2.0)


@pytest.mark.parametrize("kind", ["no_reference", "no_kl_weight", "open_clip", "closed_clip"])
def test_policy_loss_forms(kind):
    from semi_markov_crf_b200 import semicrf
    B, T, V = 4, 9, 77
    lens, lengths = _case(B, T)
    x, d = _logits(B, T, V, torch.float32, 5)
    y = _labels(B, T, V, lens, 6)
    old, reference = _policy_inputs(x, lens, y, 1.0, 7)
    adv = torch.tensor([1.0, -1.0, 0.0, -0.5])
    kw = {"no_reference": dict(ref=None, lo=0.2, hi=0.3, c=0.5),
          "no_kl_weight": dict(ref=reference, lo=0.2, hi=0.3, c=0.0),
          "open_clip": dict(ref=reference, lo=1.0, hi=math.inf, c=0.1),
          "closed_clip": dict(ref=reference, lo=0.0, hi=0.0, c=0.1)}[kind]
    want = ref.policy_loss(x, lens, y, old, adv, **kw)
    out = semicrf.policy_loss(d, lengths.cuda(), y.cuda(), old.cuda(), adv.cuda(),
                              ref_logp=None if kw["ref"] is None else kw["ref"].cuda(),
                              clip_low=kw["lo"], clip_high=kw["hi"], kl_coef=kw["c"])
    _policy_tolerances(out, want, lens, V, 1.0, kw["c"])
    scale = (want["logp"] - old.double()).exp() + 0.5
    _check_grad(out["grad_logits"], want["grad_logits"], scale, torch.float32, V, 1.0, 2.0)


@pytest.mark.parametrize("dtype,pad", LAYOUTS, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("B,T,V", [s for s in SIZES if s[0] % 2 == 0])
def test_preference_loss(B, T, V, dtype, pad):
    from semi_markov_crf_b200 import semicrf
    lens, lengths = _case(B, T)
    tau = 0.8 if V % 2 else 1.0
    x, d = _logits(B, T, V, dtype, V + 2, pad)
    y = _labels(B, T, V, lens, V + 7)
    _, reference = _policy_inputs(x, lens, y, tau, V + 1)
    w = torch.rand(B // 2, generator=_gen(11), dtype=torch.float64) + 0.5
    kw = dict(beta=0.3, margin=0.1, smoothing=0.1 if V % 3 else 0.0, average=V % 5 == 0)
    want = ref.preference_loss(x, lens, y, reference, tau=tau, w=w, **kw)
    ws = semicrf.LossWorkspace(B, T)
    out = semicrf.preference_loss(d, lengths.cuda(), y.cuda(), ref_logp=reference.cuda(),
                                  temperature=tau, grad_loss=w.cuda(), ws=ws, **kw)
    assert semicrf.get_status(ws) == 0
    _check("logp", out["logp"], want["logp"], lse_tol(V) + U * want["logp"].abs())
    # |logp - ref| < 2 here: its float32 rounding adds 2 u to every position
    e = 0.3 * T * (lse_tol(V) + 2 * U)
    _check("reward", out["reward"], want["reward"], e + U * want["reward"].abs())
    _check("loss", out["loss"], want["loss"], 2 * e + U * want["loss"].abs())
    _check_grad(out["grad_logits"], want["grad_logits"],
                want["slope"].abs() * (1 + T), dtype, V, tau)


def _teacher(x, k, seed, ragged=True):
    B, T, V = x.shape
    t = 0.8 * x.float() + torch.randn(B, T, V, generator=_gen(seed))
    top = t.topk(k, -1)
    ids = top.indices.int()
    if ragged:
        n = torch.randint(0, k + 1, (B, T, 1), generator=_gen(seed + 1))
        ids = torch.where(torch.arange(k) < n, ids, torch.full_like(ids, -1))
    return ids.contiguous(), top.values.contiguous(), t


def _check_distill(out, want, lens, dtype, V, tau):
    # terms p (log p - log q): sum p <= 1, |log p - log q| errors of both sums and
    # of the float32 exponential of log p (|log p| <= 40)
    e = tau * tau * (2 * lse_tol(V) + 60 * U)
    _check("token_loss", out["token_loss"], want["token_loss"],
           e * (1 + want["token_loss"].abs() / tau ** 2) + U * want["token_loss"].abs())
    n = torch.tensor([max(1, v) for v in lens], dtype=torch.float64)
    _check("loss", out["loss"], want["loss"],
           e * (n + want["token_loss"].abs().sum(1) / tau ** 2) + 2 * U * want["token_loss"].abs().sum(1))
    _check_grad(out["grad_logits"], want["grad_logits"], want["slope"], dtype, V, tau, 2.0)


@pytest.mark.parametrize("dtype,pad", LAYOUTS, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("B,T,V", SIZES)
def test_distill_loss(B, T, V, dtype, pad):
    from semi_markov_crf_b200 import semicrf
    lens, lengths = _case(B, T)
    tau = 2.0 if V % 2 else 1.0
    k = min(V, [1, 8, 33, 128, 1000][V % 5])
    x, d = _logits(B, T, V, dtype, V + 3, pad)
    ids, teacher, whole = _teacher(x, k, V)
    lse = (whole.double() / tau).logsumexp(-1).float() if V % 3 else None
    w = torch.rand(B, generator=_gen(12), dtype=torch.float64) + 0.5
    want = ref.distill_loss(x, lens, ids, teacher, lse, tau, w)
    ws = semicrf.LossWorkspace(B, T)
    out = semicrf.distill_loss(d, lengths.cuda(), ids.cuda(), teacher.cuda(),
                               None if lse is None else lse.cuda(), tau, w.cuda(), ws=ws)
    assert semicrf.get_status(ws) == 0
    _check_distill(out, want, lens, dtype, V, tau)


@pytest.mark.parametrize("V,k", [(6, 6), (40, 12), (700, 64), (5000, 1024), (40000, 200)])
def test_distill_equal_labels_and_empty_entries(V, k):
    """The same label in several entries adds up; entries of logit -inf and
    unused entries do nothing; a position with neither has no loss."""
    from semi_markov_crf_b200 import semicrf
    B, T = 3, 4
    lens = [4, 4, 3]
    x, d = _logits(B, T, V, torch.float32, V)
    ids = torch.randint(0, min(V, max(2, k // 3)), (B, T, k), generator=_gen(1), dtype=torch.int32)
    teacher = 2 * torch.randn(B, T, k, generator=_gen(2))
    ids[0, 0] = 1                       # one label in every entry
    ids[0, 1] = -1                      # no entry
    teacher[0, 2] = -math.inf           # no probability
    teacher[1, :, ::2] = -math.inf
    ids[2, :, 1::2] = -1
    teacher[2, :, 1::2] = math.nan      # behind an unused entry: never looked at
    want = ref.distill_loss(x, lens, ids, teacher)
    out = semicrf.distill_loss(d, torch.tensor(lens, dtype=torch.int32).cuda(), ids.cuda(),
                               teacher.cuda())
    _check_distill(out, want, lens, torch.float32, V, 1.0)
    assert float(out["grad_logits"][0, 1:3].abs().max()) == 0.0


LOW = {t: torch.finfo(t).min for t in DTYPES}


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("V", [5, 130, 1500, 9000, 70001])
def test_masked_scores(V, dtype):
    """-inf and the type's lowest value beside finite scores are labels of
    probability zero; a row of nothing but the lowest value is uniform; a
    label of probability zero has logp -inf; a row of -inf, or one that holds
    NaN or +inf, gives NaN and leaves the other rows alone."""
    from semi_markov_crf_b200 import semicrf
    B, T = 2, 6
    x, _ = _logits(B, T, V, dtype, V)
    y = torch.randint(0, V, (B, T), generator=_gen(4), dtype=torch.int32)
    low = LOW[dtype]
    for t, value in ((0, -math.inf), (1, low)):
        keep = torch.rand(V, generator=_gen(t)) < 0.1
        keep[y[0, t].item()] = True
        x[0, t] = torch.where(keep, x[0, t], torch.full_like(x[0, t], value))
    x[0, 2] = low
    x[0, 3, y[0, 3].item()] = -math.inf
    x[0, 4] = -math.inf
    x[0, 5, V // 2] = math.nan
    x[1, 0, 0] = math.inf
    lens = [T, T - 1]
    x[1, T - 1] = math.nan  # behind the sequence
    want = ref.label_logprob(x, lens, y)
    out = semicrf.label_logprob(x.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), y.cuda(),
                                grad=True)
    bad = [(0, 4), (0, 5), (1, 0)]
    for b, t in bad:
        assert math.isnan(out["logp"][b, t])
        assert torch.isnan(out["grad_logits"][b, t]).any()
        want["logp"][b, t] = math.nan
    _check("logp", out["logp"], want["logp"], lse_tol(V) + U * want["logp"].abs())
    fine = torch.ones(B, T, dtype=torch.bool)
    for b, t in bad:
        fine[b, t] = False
    _check_grad(out["grad_logits"].cpu()[fine], want["grad_logits"][fine], want["slope"][fine],
                dtype, V, 1.0)
    assert out["logp"][0, 3].item() == -math.inf
    assert abs(out["logp"][0, 2].item() + math.log(V)) <= lse_tol(V) + U * math.log(V)


@pytest.mark.parametrize("V", [6, 300, 6000])
def test_malformed_labels_and_lengths(V):
    from semi_markov_crf_b200 import semicrf
    B, T = 4, 5
    x, d = _logits(B, T, V, torch.float32, V)
    y = torch.randint(0, V, (B, T), generator=_gen(4), dtype=torch.int32)
    y[0, 2] = V
    lengths = torch.tensor([T, T, T + 1, -1], dtype=torch.int32).cuda()
    old = torch.full((B, T), -3.0).cuda()
    ws = semicrf.LossWorkspace(B, T)
    out = semicrf.policy_loss(d, lengths, y.cuda(), old, torch.ones(B).cuda(), ref_logp=old, ws=ws)
    assert semicrf.get_status(ws) == 6
    assert torch.isnan(out["loss"].cpu()).tolist() == [True, False, True, True]
    assert math.isnan(out["logp"][0, 2]) and not torch.isnan(out["logp"][1]).any()
    g = out["grad_logits"]
    assert float(g[0, 2].abs().max()) == 0 and float(g[2:].abs().max()) == 0
    assert not torch.isnan(g).any()
    want = ref.policy_loss(x, [0, T, 0, 0], y, old.cpu(), torch.ones(B))  # positions the clip holds are 0
    _check_grad(g[1], want["grad_logits"][1], (want["logp"][1] + 3.0).exp(), torch.float32, V, 1.0, 2.0)
    # one malformed sequence takes the gradient of its pair with it
    pairs = semicrf.preference_loss(d, torch.full((B,), T, dtype=torch.int32).cuda(), y.cuda(), ws=ws)
    assert semicrf.get_status(ws) == 0
    assert torch.isnan(pairs["loss"].cpu()).tolist() == [True, False]
    g = pairs["grad_logits"]
    assert float(g[0].abs().max()) == 0 and float(g[2].abs().max()) == 0
    assert float(g[1].abs().max()) > 0 and float(g[3].abs().max()) > 0
    pairs = semicrf.preference_loss(d, lengths, y.cuda(), ws=ws)
    assert semicrf.get_status(ws) == 6
    assert torch.isnan(pairs["loss"]).all() and float(pairs["grad_logits"].abs().max()) == 0
    ids = torch.zeros(B, T, 3, dtype=torch.int32)
    ids[1, 1, 2] = V
    dist = semicrf.distill_loss(d, lengths, ids.cuda(), torch.zeros(B, T, 3).cuda(), ws=ws)
    assert semicrf.get_status(ws) == 6
    assert torch.isnan(dist["token_loss"].cpu()).sum() == 1 and math.isnan(dist["token_loss"][1, 1])
    assert float(dist["grad_logits"][1, 1].abs().max()) == 0


@pytest.mark.parametrize("B,T", [(0, 4), (2, 0), (0, 0)])
def test_empty_batches(B, T):
    from semi_markov_crf_b200 import semicrf
    V = 7
    d = torch.empty(B, T, V, device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    y = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    z = torch.zeros(B, T, device="cuda")
    ws = semicrf.LossWorkspace(B, T)
    for out in (semicrf.label_logprob(d, lengths, y, grad=True, ws=ws),
                semicrf.policy_loss(d, lengths, y, z, z, ws=ws),
                semicrf.distill_loss(d, lengths, torch.zeros(B, T, 2, dtype=torch.int32).cuda(),
                                     torch.zeros(B, T, 2).cuda(), ws=ws)):
        assert semicrf.get_status(ws) == 0
        assert float(out.get("loss", out.get("score")).abs().sum()) == 0.0
    pairs = semicrf.preference_loss(d, lengths, y, margin=0.5, ws=ws)
    assert semicrf.get_status(ws) == 0
    want = ref.preference_term(-0.5, 0.0)[0]
    assert torch.allclose(pairs["loss"].cpu(), torch.full((B // 2,), want), atol=1e-6)


@pytest.mark.parametrize("V", [6, 128, 1000, 40000])
def test_accumulate_adds_to_the_gradient(V):
    from semi_markov_crf_b200 import semicrf
    B, T = 4, 6
    lens, lengths = _case(B, T)
    x, d = _logits(B, T, V, torch.float32, V)
    y = _labels(B, T, V, lens, V).cuda()
    lengths = lengths.cuda()
    ids, teacher, _ = _teacher(x, min(V, 16), V)
    old = torch.randn(B, T, generator=_gen(1)).cuda() - 3
    calls = [lambda **k: semicrf.label_logprob(d, lengths, y, grad=True, **k),
             lambda **k: semicrf.policy_loss(d, lengths, y, old, old[:, 0].contiguous(), **k),
             lambda **k: semicrf.preference_loss(d, lengths, y, old, **k),
             lambda **k: semicrf.distill_loss(d, lengths, ids.cuda(), teacher.cuda(), **k)]
    start = torch.randn(B, T, V, generator=_gen(2)).cuda()
    for call in calls:
        plain = call()["grad_logits"]
        added = call(out={"grad_logits": start.clone()}, accumulate=True)["grad_logits"]
        # one rounding of the sum, and of the parts the kernel adds up
        tol = 2 * U * (start.abs() + plain.abs()) + 4 * U * plain.abs().amax(-1, keepdim=True)
        assert bool(((added - (start + plain)).abs() <= tol).all())
        assert torch.equal(added[1], start[1])  # an empty sequence is left as it was


@pytest.mark.parametrize("V", [39, 2000, 50001])
def test_gradients_against_differences(V):
    """Directional central differences of the kernels' own losses.  In a
    direction e with |e_v| <= 1 the third derivative of a log-sum-exp is at
    most 2 and its first two at most 1, so the loss of one position moves by
    its slope plus h^2 D / 6 with D <= 40 for the losses here (|A| r <= 3,
    temperature 1), and its rounding gives (4 LSE + 16 u) / h more."""
    from semi_markov_crf_b200 import semicrf
    B, T = 4, 1
    x, d = _logits(B, T, V, torch.float32, V)
    lengths = torch.ones(B, dtype=torch.int32).cuda()
    y = x.argmax(-1).int().cuda()
    e = (2 * torch.rand(B, T, V, generator=_gen(8)) - 1).cuda()
    now = semicrf.label_logprob(d, lengths, y)["logp"]
    old = now + 0.05 * torch.tensor([[1.0], [-1.0], [1.5], [-1.5]]).cuda()
    adv = torch.tensor([1.0, -1.0, 2.0, 0.5]).cuda()
    ids, teacher, _ = _teacher(x, 16, V, ragged=False)
    ids, teacher = ids.cuda(), teacher.cuda()
    calls = {"logprob": lambda z, **k: semicrf.label_logprob(z, lengths, y, grad=True),
             "policy": lambda z: semicrf.policy_loss(z, lengths, y, old, adv, ref_logp=old - 0.1,
                                                     kl_coef=0.2),
             "preference": lambda z: semicrf.preference_loss(z, lengths, y, old, beta=0.5),
             "distill": lambda z: semicrf.distill_loss(z, lengths, ids, teacher)}
    h = 2.0 ** -5
    for name, call in calls.items():
        out = call(d)
        key = "score" if name == "logprob" else "loss"
        up, down = call(d + h * e)[key].double(), call(d - h * e)[key].double()
        moved = ((up - down) / (2 * h)).sum().item()
        slope = (out["grad_logits"].double() * e).sum().item()
        size = 8.0  # |loss| here
        tol = B * (40 * h * h / 6 + (4 * lse_tol(V) + 16 * U * size) / h)
        assert abs(moved - slope) <= tol, (name, moved, slope, tol)


@pytest.mark.parametrize("n", [1, 31, 1000])
def test_path_forms(n):
    """float64 in and out: a few roundings of 2^-53 on exponentials of ratios
    up to e^2 and scores near 300; 1e-12 is a thousand times that."""
    from semi_markov_crf_b200 import semicrf
    g = _gen(n)
    rnd = lambda: torch.randn(n, generator=g, dtype=torch.float64)
    logp = -20 + 5 * rnd()
    old, reference, adv = logp - 0.3 * rnd(), logp + 0.3 * rnd(), rnd()
    w = torch.rand(n, generator=g, dtype=torch.float64)
    got = semicrf.policy_scores(logp.cuda(), old.cuda(), adv.cuda(), reference.cuda(), 0.2, 0.3, 0.1,
                                w.cuda())
    want = [ref.policy_term(*(float(v[i]) for v in (logp, old, adv, reference)), 0.2, 0.3, 0.1)
            for i in range(n)]
    for i in range(n):
        assert abs(got["loss"][i].item() - want[i][0]) <= 1e-12
        assert abs(got["kl"][i].item() - want[i][1]) <= 1e-12
        assert abs(got["grad_logp"][i].item() - float(w[i]) * want[i][2]) <= 1e-12
    c = 300 + 20 * rnd()
    r, rc, rr = c - 4 + 30 * rnd(), c + 3 * rnd(), c + 3 * rnd()
    got = semicrf.preference_scores(c.cuda(), r.cuda(), rc.cuda(), rr.cuda(), 0.2, 0.1, 0.05,
                                    w.cuda())
    for i in range(n):
        u = 0.2 * float((c[i] - r[i]) - (rc[i] - rr[i])) - 0.1
        loss, slope = ref.preference_term(u, 0.05)
        assert abs(got["loss"][i].item() - loss) <= 1e-11
        assert abs(got["grad_chosen"][i].item() - 0.2 * slope * float(w[i])) <= 1e-12
        assert got["grad_rejected"][i].item() == -got["grad_chosen"][i].item()
    bare = semicrf.preference_scores(c.cuda(), r.cuda(), beta=0.2)
    assert abs(bare["loss"][0].item() - ref.preference_term(0.2 * float(c[0] - r[0]), 0)[0]) <= 1e-11
    assert semicrf.policy_scores(*(torch.empty(0, dtype=torch.float64).cuda(),) * 3)["loss"].numel() == 0


def _calls(V, dtype, seed=0, B=4, T=6):
    """One call of each logits form, with its inputs held."""
    from semi_markov_crf_b200 import semicrf
    lens, lengths = _case(B, T)
    x, d = _logits(B, T, V, dtype, seed)
    y = _labels(B, T, V, lens, seed).cuda()
    old, reference = (v.cuda() for v in _policy_inputs(x, lens, y.cpu(), 1.0, seed))
    ids, teacher, _ = _teacher(x, min(V, 20), seed)
    ids, teacher, lengths = ids.cuda(), teacher.cuda(), lengths.cuda()
    adv = torch.randn(B, generator=_gen(seed)).cuda()
    return d, {
        "logprob": lambda **k: semicrf.label_logprob(d, lengths, y, grad=True, **k),
        "policy": lambda **k: semicrf.policy_loss(d, lengths, y, old, adv, ref_logp=reference,
                                                  kl_coef=0.1, **k),
        "preference": lambda **k: semicrf.preference_loss(d, lengths, y, reference, **k),
        "distill": lambda **k: semicrf.distill_loss(d, lengths, ids, teacher, **k)}


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("V", [39, 1000, 33000])
def test_runs_are_identical_and_captured_graphs_replay(V, dtype):
    """Two eager runs agree bit for bit; graphs captured one after the other
    on one workspace replay on new inputs, in either order; a call on a side
    stream agrees too."""
    from semi_markov_crf_b200 import semicrf
    d, calls = _calls(V, dtype)
    ws = semicrf.LossWorkspace(4, 6)
    outs = {n: call(ws=ws, out={}) for n, call in calls.items()}
    first = {n: {k: v.clone() for k, v in o.items()} for n, o in outs.items()}

    def same(name, got, want):
        for k, v in want.items():
            assert torch.equal(torch.nan_to_num(got[k].float()), torch.nan_to_num(v.float())), (name, k)

    for n, call in calls.items():
        same(n, call(ws=ws), first[n])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        others = {n: call() for n, call in calls.items()}
    torch.cuda.current_stream().wait_stream(side)
    for n in calls:
        same(n, others[n], first[n])
    graphs = {}
    for n, call in calls.items():
        graphs[n] = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[n]):
            call(ws=ws, out=outs[n])
    d.mul_(0.5)
    want = {n: {k: v.clone() for k, v in call().items()} for n, call in calls.items()}
    for order in (list(calls), list(calls)[::-1]):
        for n in order:
            for v in outs[n].values():
                v.zero_()
        for n in order:
            graphs[n].replay()
        torch.cuda.synchronize()
        for n in order:
            same(n, outs[n], want[n])


WIDTHS = list(range(1, 140)) + [160, 200, 255, 256, 257, 260, 264, 300, 333, 511, 512, 513, 520, 700, 767,
                                 1000, 1023, 1024, 1025, 1032, 1400, 2000, 2047, 2048, 2049, 2056, 2500,
                                 4095, 4096, 4097, 5000, 8191, 8192, 8193, 9000]


@pytest.mark.parametrize("dtype,pad", LAYOUTS + [(torch.float16, 8), (torch.float32, 4)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_every_width(dtype, pad):
    """Each width takes its kernel, lanes and layout: log-probabilities with and
    without a gradient, pairs and distillation with three list lengths, against
    vectorised float64 forms."""
    from semi_markov_crf_b200 import semicrf
    B, T = 2, 3
    lengths = torch.tensor([3, 2], dtype=torch.int32).cuda()
    live = (torch.arange(T, device="cuda")[None] < lengths[:, None])[..., None]
    for V in WIDTHS:
        x, d = _logits(B, T, V, dtype, V, pad)
        q = torch.softmax(d.double(), -1)
        y = torch.randint(0, V, (B, T), generator=_gen(V), dtype=torch.int32).cuda()
        hot = torch.zeros_like(q).scatter_(2, y.long()[..., None], 1.0)
        base = torch.where(live, hot - q, torch.zeros_like(q)).cpu()
        logp = torch.where(live[..., 0], q.gather(2, y.long()[..., None])[..., 0].log(),
                           torch.zeros_like(q[..., 0])).cpu()
        ones = torch.ones(B, T, dtype=torch.float64)
        out = semicrf.label_logprob(d, lengths, y, grad=True)
        bare = semicrf.label_logprob(d, lengths, y)
        tol = lse_tol(V) + U * logp.abs()
        _check(f"logp {V}", out["logp"], logp, tol)
        _check(f"bare {V}", bare["logp"], logp, tol)
        _check_grad(out["grad_logits"], base, ones, dtype, V, 1.0)
        pairs = semicrf.preference_loss(d, lengths, y, beta=0.5)
        w = 0.5 * ref.preference_term(float(pairs["reward"][0] - pairs["reward"][1]), 0.0)[1]
        slope = torch.tensor([w, -w], dtype=torch.float64)[:, None] * ones
        _check_grad(pairs["grad_logits"], slope[..., None] * base, slope.abs() * (1 + T), dtype, V, 1.0)
        for k in (1, 20, 100):
            if k > 2 * V + 4:
                continue
            ids = torch.randint(0, V, (B, T, k), generator=_gen(V + k), dtype=torch.int32).cuda()
            t = torch.randn(B, T, k, generator=_gen(k)).cuda()
            p = torch.softmax(t.double(), -1)
            want = torch.where(live, q.scatter_add(2, ids.long(), -p), torch.zeros_like(q)).cpu()
            dist = semicrf.distill_loss(d, lengths, ids, t)
            _check_grad(dist["grad_logits"], want, ones, dtype, V, 1.0, 2.0)
            loss = (p * (p.log() - q.gather(2, ids.long()).log())).sum(-1)
            loss = torch.where(live[..., 0], loss, torch.zeros_like(loss)).cpu()
            _check(f"token {V} {k}", dist["token_loss"], loss,
                   (2 * lse_tol(V) + 60 * U) * (1 + loss.abs()) + U * loss.abs())


@pytest.mark.parametrize("V,k", [(4096 * 40, 1024), (2048, 128), (2048, 700)])
def test_teacher_labels_that_share_their_low_bits(V, k):
    """Labels a power of two apart: the search for repeated ones stays short
    (the time is not tested, the values are)."""
    from semi_markov_crf_b200 import semicrf
    B, T = 1, 2
    x, d = _logits(B, T, V, torch.float32, V)
    step = V // k
    ids = (torch.arange(k) * step).int().expand(B, T, k).contiguous()
    teacher = torch.randn(B, T, k, generator=_gen(1))
    want = ref.distill_loss(x, [2], ids, teacher)
    out = semicrf.distill_loss(d, torch.tensor([2], dtype=torch.int32).cuda(), ids.cuda(), teacher.cuda())
    _check_distill(out, want, [2], torch.float32, V, 1.0)


@pytest.mark.parametrize("V", [9, 300, 1300, 5000, 70000])
def test_single_positions(V):
    """T = 1, the step that emits a label: the row pass writes the sequences'
    sums itself, bad lengths and malformed labels included."""
    from semi_markov_crf_b200 import semicrf
    B, T = 7, 1
    x, d = _logits(B, T, V, torch.bfloat16, V)
    lens = [1, 1, 0, 1, 2, -1, 1]
    lengths = torch.tensor(lens, dtype=torch.int32)
    good = [v if v in (0, 1) else 0 for v in lens]
    y = torch.randint(0, V, (B, T), generator=_gen(V), dtype=torch.int32)
    y[3], y[6] = -1, V
    ry = y.clone()
    ry[6] = -1
    old, reference = _policy_inputs(x, good, ry, 1.0, V)
    adv = torch.randn(B, generator=_gen(1)).clamp(-2, 2)
    want = ref.policy_loss(x, good, ry, old, adv, reference, 0.2, 0.3, 0.1)
    for key in ("loss", "kl"):
        want[key][[4, 5, 6]] = math.nan
    want["logp"][6] = math.nan
    ws = semicrf.LossWorkspace(B, T)
    out = semicrf.policy_loss(d, lengths.cuda(), y.cuda(), old.cuda(), adv.cuda(),
                              ref_logp=reference.cuda(), clip_high=0.3, kl_coef=0.1, ws=ws)
    assert semicrf.get_status(ws) == 6
    _policy_tolerances(out, want, good, V, 2.0, 0.1)
    scale = (2 * (torch.nan_to_num(want["logp"]) - old.double()).exp() + 0.1) * (want["slope"] != 0)
    _check_grad(out["grad_logits"], want["grad_logits"], scale, torch.bfloat16, V, 1.0, 2.0)
    ids, teacher, _ = _teacher(x, 5, V)
    out = semicrf.distill_loss(d, torch.ones(B, dtype=torch.int32).cuda(), ids.cuda(), teacher.cuda(),
                               ws=ws)
    assert semicrf.get_status(ws) == 0
    want = ref.distill_loss(x, [1] * B, ids, teacher)
    _check_distill(out, want, [1] * B, torch.bfloat16, V, 1.0)
    out = semicrf.label_logprob(d, torch.ones(B, dtype=torch.int32).cuda(), ry.cuda(), ws=ws)
    want = ref.label_logprob(x, [1] * B, ry)
    _check("score", out["score"], want["score"], lse_tol(V) + 2 * U * want["score"].abs())


@pytest.mark.parametrize("T", [2049, 9000, 70001])
def test_long_sequences(T):
    """Sums over sequences that one CTA does not cover: the kernels' own
    per-position values added in float64 here (n u^2 of that sum is nothing:
    one rounding of the float32 result, u, and one of each float32 term)."""
    from semi_markov_crf_b200 import semicrf
    B, V = 2, 5
    x, d = _logits(B, T, V, torch.float32, T)
    lens = [T, T - 700]
    lengths = torch.tensor(lens, dtype=torch.int32).cuda()
    y = torch.randint(0, V, (B, T), generator=_gen(T), dtype=torch.int32)
    y[:, ::7] = -1
    at = torch.arange(T)[None] < torch.tensor(lens)[:, None]
    counts = (y >= 0) & at
    logq = torch.log_softmax(x.double(), -1).gather(-1, y.clamp_min(0).long()[..., None])[..., 0]
    logp = torch.where(counts, logq, torch.zeros_like(logq))
    out = semicrf.label_logprob(d, lengths, y.cuda())
    tol = (2 * U * logp.abs() + counts * lse_tol(V)).sum(1)
    _check("score", out["score"], logp.sum(1), tol + U * logp.sum(1).abs())
    reference = (logq + 0.1 * torch.randn(B, T, generator=_gen(2), dtype=torch.float64)).float()
    for average in (False, True):
        pairs = semicrf.preference_loss(d, lengths, y.cuda(), reference.cuda(), beta=0.01,
                                        average=average)
        n = counts.sum(1).double() if average else torch.ones(B, dtype=torch.float64)
        ratio = torch.where(counts, logq - reference.double(), torch.zeros_like(logq))
        want = 0.01 * ratio.sum(1) / n
        e = 0.01 * counts.sum(1) * (lse_tol(V) + U) / n
        _check("reward", pairs["reward"], want, e + U * want.abs())
        slope = 0.01 * ref.preference_term(float(want[0] - want[1]), 0.0)[1]
        q = torch.softmax(x.double(), -1)
        base = torch.nn.functional.one_hot(y.clamp_min(0).long(), V).double() - q
        sign = torch.tensor([slope, -slope], dtype=torch.float64) / n
        grad = torch.where(counts[..., None], base * sign[:, None, None], torch.zeros_like(base))
        # the weight's own error: 0.01 (d reward) on top of an entry's
        _check("grad", pairs["grad_logits"], grad,
               (sign.abs() * (3 * lse_tol(V) + 12 * U + 2 * float(e.max())))[:, None, None] + U * grad.abs())
    old = (logq + 0.05).float()
    pol = semicrf.policy_loss(d, lengths, y.cuda(), old.cuda(), torch.tensor([1.0, -1.0]).cuda(),
                              ref_logp=reference.cuda(), kl_coef=0.1)
    assert pol["clipped"].tolist() == [0, 0]  # exp(-0.05) is inside the clip
    gap = torch.where(counts, reference.double() - logq, torch.zeros_like(logq))
    kl = (torch.expm1(gap) - gap).sum(1)
    _check("kl", pol["kl"], kl, counts.sum(1) * 2 * (lse_tol(V) + 4 * U) + U * kl)


@pytest.mark.parametrize("V,dtype,k", [(8, torch.float32, 20), (300, torch.bfloat16, 100),
                                       (1500, torch.float32, 129), (2048, torch.float16, 1024),
                                       (3001, torch.float32, 1024), (262145, torch.float32, 30),
                                       (600001, torch.float32, 40), (900001, torch.bfloat16, 3)])
def test_distill_list_lengths(V, dtype, k):
    """Lists of every length class at short, long and very wide rows (the last
    two are wider than the rings of a cluster hold with a gradient), labels
    repeated where the list is longer than a third of the vocabulary."""
    from semi_markov_crf_b200 import semicrf
    B, T = 2, 2
    x, d = _logits(B, T, V, dtype, V)
    ids = torch.randint(0, V, (B, T, k), generator=_gen(k), dtype=torch.int32)
    ids[1, :, k // 2:] = -1
    teacher = 2 * torch.randn(B, T, k, generator=_gen(k + 1))
    want = ref.distill_loss(x, [2, 2], ids, teacher, None, 1.5)
    out = semicrf.distill_loss(d, torch.tensor([2, 2], dtype=torch.int32).cuda(), ids.cuda(),
                               teacher.cuda(), temperature=1.5)
    _check_distill(out, want, [2, 2], dtype, V, 1.5)


@pytest.mark.parametrize("dtype,pad", [(torch.float32, 0), (torch.float32, 1), (torch.bfloat16, 3)], ids=str)
@pytest.mark.parametrize("V,k", [(17, 5), (38, 8), (38, 16), (38, 17), (38, 32), (64, 33), (64, 64),
                                 (128, 16), (128, 40), (160, 65), (296, 128), (296, 129), (777, 20),
                                 (2048, 5), (2049, 5), (2049, 17), (8200, 20), (8200, 200)])
def test_one_repeated_teacher_label(V, k, dtype, pad):
    """Positions without a repeated label and positions with one pair of them,
    the lowest and the highest label, and neighbours across 32, among them."""
    from semi_markov_crf_b200 import semicrf
    B, T = 7, 9
    lens = [T] * B
    x, d = _logits(B, T, V, dtype, V + k, pad)
    ids = torch.rand(B, T, V, generator=_gen(V * k)).argsort(-1)[..., :k].int()
    pairs = [(0, 1), (0, k - 1), (k - 2, k - 1), (1, k // 2)]
    for n in range(B * T):
        row = ids[n // T, n % T]
        if n % 3 == 0:
            a, b = pairs[n % 4]
            label = [0, V - 1, 31 % V, 32 % V, int(row[a])][n % 5]
            row[row == label] = row[a].clone()      # its old place takes another
            row[a] = row[b] = label
    teacher = torch.randn(B, T, k, generator=_gen(k))
    want = ref.distill_loss(x, lens, ids, teacher)
    out = semicrf.distill_loss(d, torch.tensor(lens, dtype=torch.int32).cuda(), ids.cuda(), teacher.cuda())
    _check_distill(out, want, lens, dtype, V, 1.0)


@pytest.mark.parametrize("V,dtype", [(600001, torch.float32), (900001, torch.bfloat16)])
def test_very_wide_rows(V, dtype):
    from semi_markov_crf_b200 import semicrf
    B, T = 2, 2
    x, d = _logits(B, T, V, dtype, V)
    y = torch.randint(0, V, (B, T), generator=_gen(V), dtype=torch.int32)
    lens = [2, 1]
    lengths = torch.tensor(lens, dtype=torch.int32).cuda()
    want = ref.label_logprob(x, lens, y, 0.9)
    out = semicrf.label_logprob(d, lengths, y.cuda(), 0.9, grad=True)
    _check("logp", out["logp"], want["logp"], lse_tol(V) + U * want["logp"].abs())
    _check_grad(out["grad_logits"], want["grad_logits"], want["slope"], dtype, V, 0.9)
    pairs = semicrf.preference_loss(d, lengths, y.cuda(), beta=0.1)
    pref = ref.preference_loss(x, lens, y, beta=0.1)
    _check_grad(pairs["grad_logits"], pref["grad_logits"], pref["slope"].abs() * (1 + T) + 1e-9, dtype, V,
                1.0)


@pytest.mark.parametrize("V", [6, 300, 1001, 5000, 140000])
@pytest.mark.parametrize("pads", [(0, 5), (5, 0), (8, 8), (3, 7)])
def test_gradient_rows_of_their_own_stride(V, pads):
    """Scores and gradient with rows apart by different strides: what lies
    between the gradient's rows stays as it was."""
    from semi_markov_crf_b200 import semicrf
    B, T = 3, 3
    lens, lengths = [3, 0, 2], torch.tensor([3, 0, 2], dtype=torch.int32).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        x, d = _logits(B, T, V, dtype, V, pads[0])
        y = torch.randint(0, V, (B, T), generator=_gen(V), dtype=torch.int32)
        ids, teacher, _ = _teacher(x, 6, V)
        wide = torch.full((B, T, V + pads[1]), 7.0, dtype=dtype, device="cuda")
        for name in ("label", "distill"):
            wide.fill_(7.0)
            out = {"grad_logits": wide[..., :V]}
            if name == "label":
                want = ref.label_logprob(x, lens, y)
                semicrf.label_logprob(d, lengths, y.cuda(), grad=True, out=out)
            else:
                want = ref.distill_loss(x, lens, ids, teacher)
                semicrf.distill_loss(d, lengths, ids.cuda(), teacher.cuda(), out=out)
            _check_grad(out["grad_logits"], want["grad_logits"], want["slope"], dtype, V, 1.0, 2.0)
            assert bool((wide[..., V:] == 7.0).all())


def test_accumulate_over_a_cluster():
    """A float32 row shared by a cluster, its gradient added to."""
    from semi_markov_crf_b200 import semicrf
    B, T, V = 2, 2, 131075
    x, d = _logits(B, T, V, torch.float32, 3)
    lengths = torch.tensor([2, 1], dtype=torch.int32).cuda()
    ids, teacher, _ = _teacher(x, 50, 4, ragged=False)
    plain = semicrf.distill_loss(d, lengths, ids.cuda(), teacher.cuda())["grad_logits"]
    start = torch.randn(B, T, V, generator=_gen(2)).cuda()
    added = semicrf.distill_loss(d, lengths, ids.cuda(), teacher.cuda(), accumulate=True,
                                 out={"grad_logits": start.clone()})["grad_logits"]
    tol = 2 * U * (start.abs() + plain.abs()) + 4 * U * plain.abs().amax(-1, keepdim=True)
    assert bool(((added - (start + plain)).abs() <= tol).all())
    assert torch.equal(added[1, 1], start[1, 1])


def test_two_streams_at_once():
    """Calls of two streams, each with its workspace, while the other runs."""
    from semi_markov_crf_b200 import semicrf
    sizes = [(33000, torch.bfloat16), (70000, torch.float32), (300, torch.float32)]
    made = [_calls(V, dtype, seed=i, B=6, T=30) for i, (V, dtype) in enumerate(sizes)]
    want = [{n: call() for n, call in calls.items()} for _, calls in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [[] for _ in made]
    for _ in range(3):
        for i, (_, calls) in enumerate(made):
            with torch.cuda.stream(streams[i]):
                got[i].append({n: call() for n, call in calls.items()})
    torch.cuda.synchronize()
    for i, runs in enumerate(got):
        for run in runs:
            for n, o in run.items():
                for k, v in o.items():
                    assert torch.equal(torch.nan_to_num(v.float()),
                                       torch.nan_to_num(want[i][n][k].float())), (sizes[i], n, k)


def test_refused_calls_leave_the_outputs_alone():
    from semi_markov_crf_b200 import semicrf
    B, T, V = 2, 3, 40
    d = torch.zeros(B, T, V, device="cuda")
    lengths = torch.full((B,), T, dtype=torch.int32, device="cuda")
    y = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    g = torch.full((B, T, V), 5.0, device="cuda")
    cases = [
        (semicrf.SemiCRFError, dict(temperature=0.0)),
        (TypeError, dict(labels=y.long())),
        (TypeError, dict(labels=y[:, :2].contiguous())),
        (TypeError, dict(logits=d.transpose(1, 2))),
        (TypeError, dict(out={"grad_logits": g.bfloat16()})),
        (TypeError, dict(out={"grad_logits": g, "logp": torch.zeros(B, T + 1, device="cuda")})),
        (semicrf.SemiCRFError, dict(out={"grad_logits": d})),       # in place
        (ValueError, dict(ws=semicrf.LossWorkspace(B, T + 1))),
        (ValueError, dict(accumulate=True, out={})),
        (semicrf.SemiCRFError, dict(logits=d.bfloat16(), accumulate=True,
                                    out={"grad_logits": g.bfloat16()})),
    ]
    for error, change in cases:
        kw = dict(logits=d, lengths=lengths, labels=y, grad=True, out={"grad_logits": g})
        kw.update(change)
        with pytest.raises(error):
            semicrf.label_logprob(**kw)
    with pytest.raises(semicrf.SemiCRFError):
        semicrf.preference_loss(d[:1], lengths[:1], y[:1])
    assert bool((g == 5.0).all()) and bool((d == 0.0).all())


def test_first_call_inside_a_capture():
    """A process whose first call of each kind is captured (nothing may be
    allocated or synchronised in there)."""
    code = """
import sys; sys.path[:0] = [%r, %r]
import torch
from semi_markov_crf_b200 import semicrf
for V in (50, 1500, 20000, 140000):
    B, T = 4, 3
    d = torch.randn(B, T, V, device="cuda")
    lengths = torch.full((B,), T, dtype=torch.int32, device="cuda")
    y = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    ws = semicrf.LossWorkspace(B, T)
    out = {k: torch.zeros(s, device="cuda") for k, s in
           (("loss", (B // 2,)), ("reward", (B,)), ("logp", (B, T)), ("grad_logits", (B, T, V)))}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        semicrf.preference_loss(d, lengths, y, ws=ws, out=out)
    g.replay()
    torch.cuda.synchronize()
    want = semicrf.preference_loss(d, lengths, y)
    assert torch.equal(want["grad_logits"], out["grad_logits"]), V
    assert semicrf.get_status(ws) == 0
print("captured")
"""
    here = os.path.dirname(os.path.abspath(__file__))
    res = subprocess.run([sys.executable, "-c", code % (os.path.dirname(here), here)],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "captured" in res.stdout, res.stderr[-2000:]


@pytest.mark.parametrize("op,rows,V,dtype", [
    ("distill", 1500, 100003, torch.float32), ("policy", 1500, 100003, torch.float32),
    ("logprob", 3000, 65537, torch.bfloat16), ("preference", 3000, 40001, torch.float32),
    ("policy", 4000, 30000, torch.float16), ("distill", 6000, 6000, torch.bfloat16),
    ("logprob", 40000, 1001, torch.float32)])
def test_streamed_rows_are_whole_and_the_same_every_time(op, rows, V, dtype):
    """Many rows through every ring: a chunk given back before its last reader
    has it mixes rows.  Each gradient row against an elementary float32 form of
    it (errors of that form: as the kernel's), and 12 runs bit for bit.  The
    form takes its factor a from float32 outputs: a ratio from logp, u |logp|
    relative and 12 u for the sum and the exponential; the pair's slope from
    two rewards, each rounded by u |reward|, and the logistic's slope changes by
    at most its own value per unit."""
    from semi_markov_crf_b200 import semicrf
    B, T = 2, rows // 2
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    d = torch.empty(B, T, V, dtype=dtype, device="cuda")
    d.normal_(generator=g).mul_(2)
    lengths = torch.tensor([T, T - 5], dtype=torch.int32).cuda()
    y = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32)
    old = torch.full((B, T), -8.0, device="cuda")
    adv = torch.tensor([0.5, -0.5]).cuda()
    ids = torch.argsort(torch.rand(B, T, 90, generator=g, device="cuda"), -1).int() * (V // 100)
    teacher = torch.randn(B, T, 90, generator=g, device="cuda")
    w = torch.ones(B, dtype=torch.float64, device="cuda")
    call = {"logprob": lambda: semicrf.label_logprob(d, lengths, y, grad=True),
            "policy": lambda: semicrf.policy_loss(d, lengths, y, old, adv),
            "preference": lambda: semicrf.preference_loss(d, lengths, y, beta=0.001),
            "distill": lambda: semicrf.distill_loss(d, lengths, ids, teacher, grad_loss=w)}[op]
    first = {k: v.clone() for k, v in call().items()}
    for _ in range(12):
        for k, v in call().items():
            assert torch.equal(v, first[k]), k
    logp = semicrf.label_logprob(d, lengths, y)["logp"]
    if op == "preference":
        slope = 0.001 * ref.preference_term(float(first["reward"][0] - first["reward"][1]), 0.0)[1]
    for b in range(B):
        for t0 in range(0, T, 250):
            at = slice(t0, min(t0 + 250, T))
            q = torch.softmax(d[b, at].float(), -1)
            n = q.shape[0]
            live = (torch.arange(t0, t0 + n, device="cuda") < lengths[b])[:, None]
            if op == "distill":
                p = torch.softmax(teacher[b, at], -1)
                want = q.scatter_add(1, ids[b, at].long(), -p)
                a = torch.ones(n, 1, device="cuda")
            else:
                hot = torch.zeros_like(q).scatter_(1, y[b, at].long()[:, None], 1.0)
                a = torch.ones(n, 1, device="cuda")
                if op == "preference":
                    a = a * (slope if b == 0 else -slope)
                if op == "policy":
                    r = (logp[b, at] + 8.0).exp()[:, None]
                    held = (r > 1.2) if b == 0 else (r < 0.8)
                    a = torch.where(held, torch.zeros_like(r), -adv[b] * r)
                want = a * (hot - q)
            want = torch.where(live, want, torch.zeros_like(want))
            own = (U * (logp[b, at].abs()[:, None] + 12) if op == "policy" else
                   U * (2 * float(first["reward"].abs().max()) + 12) if op == "preference" else 0.0)
            tol = a.abs() * (q * (8 * lse_tol(V) + 40 * U) + 2e-7 + own) + HALF[dtype] * want.abs() \
                + TINY[dtype]
            err = (first["grad_logits"][b, at].float() - want).abs()
            assert bool((err <= tol + 1e-30).all()), (b, t0, float((err - tol).max()))


@pytest.mark.parametrize("B,T,V,dtype,k", [
    (2000, 5, 16500, torch.bfloat16, 64), (500, 8, 40000, torch.bfloat16, 100),
    (200, 9, 30000, torch.float32, 20), (200, 6, 70001, torch.float32, 130),
    (120, 9, 100003, torch.float32, 40)])
@pytest.mark.parametrize("grad", [True, False])
def test_many_short_teacher_sequences(B, T, V, dtype, k, grad):
    """Dozens of rows through each ring, rows that do not count (any number of
    them in turn) and rows with a label outside the range among them."""
    from semi_markov_crf_b200 import semicrf
    g = torch.Generator(device="cuda")
    g.manual_seed(V + k)
    tau = 1.5
    d = torch.empty(B, T, V, dtype=dtype, device="cuda")
    d.normal_(generator=g).mul_(2)
    lens = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[B // 3:B // 3 + 40] = 0
    live = torch.arange(T, device="cuda") < lens[:, None]
    ids = torch.randint(0, V // k, (B, T, k), generator=g, device="cuda", dtype=torch.int32) \
        + torch.arange(k, device="cuda", dtype=torch.int32) * (V // k)
    ids[..., 1] = torch.where(torch.rand(B, T, generator=g, device="cuda") < 0.3, ids[..., 0], ids[..., 1])
    bad = torch.rand(B, T, generator=g, device="cuda") < 0.1
    ids[..., k // 2] = torch.where(bad, V + 3, ids[..., k // 2])
    teacher = torch.randn(B, T, k, generator=g, device="cuda")
    w = torch.rand(B, generator=g, dtype=torch.float64, device="cuda") + 0.5
    ws = semicrf.LossWorkspace(B, T)
    out = semicrf.distill_loss(d, lens, ids, teacher, temperature=tau, grad_loss=w if grad else None,
                               grad=grad, ws=ws)
    assert semicrf.get_status(ws) == 0
    token = out["token_loss"].double()
    assert torch.equal(torch.isnan(token), bad & live)
    assert bool((token[~live] == 0).all())
    good = (live & ~bad).nonzero()
    p = torch.softmax(teacher.double() / tau, -1)
    for at in good.split(200):
        b, t = at[:, 0], at[:, 1]
        logq = torch.log_softmax(d[b, t].double() / tau, -1)
        i = ids[b, t].long()
        want = tau ** 2 * (p[b, t] * (p[b, t].log() - logq.gather(1, i))).sum(1)
        tol = tau * tau * (2 * lse_tol(V) + 60 * U) * (1 + want.abs() / tau ** 2) + U * want.abs()
        assert bool(((token[b, t] - want).abs() <= tol).all())
        if grad:
            a = tau * w[b][:, None]
            want = a * logq.exp().scatter_add(1, i, -p[b, t])
            tol = a * 2 * (3 * lse_tol(V) + 12 * U) + HALF[dtype] * want.abs()
            assert bool(((out["grad_logits"][b, t].double() - want).abs() <= tol).all())
    if grad:
        for at in (~live | bad).nonzero().split(400):
            assert not bool(out["grad_logits"][at[:, 0], at[:, 1]].any())


def test_rows_beyond_32_bit_offsets():
    """More than 2^31 scores: the last rows against the same rows alone."""
    from semi_markov_crf_b200 import semicrf
    B, T, V = 2, 17000, 65536
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    d = torch.empty(B, T, V, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    d.normal_(generator=g)
    lengths = torch.tensor([T, T], dtype=torch.int32).cuda()
    y = torch.full((B, T), -1, dtype=torch.int32)
    y[1, -3:] = torch.tensor([5, V - 1, 0])
    y[0, :2] = 7
    out = semicrf.label_logprob(d, lengths, y.cuda(), grad=True)
    few = torch.stack([d[1, -3:], torch.cat([d[0, :2], d[0, :1]])])
    fy = torch.stack([y[1, -3:], torch.tensor([7, 7, -1], dtype=torch.int32)])
    alone = semicrf.label_logprob(few, torch.tensor([3, 3], dtype=torch.int32).cuda(), fy.cuda(),
                                  grad=True)
    assert torch.equal(out["logp"][1, -3:], alone["logp"][0])
    assert torch.equal(out["grad_logits"][1, -3:], alone["grad_logits"][0])
    assert torch.equal(out["grad_logits"][0, :2], alone["grad_logits"][1, :2])
    assert float(out["grad_logits"][1, 100:200].abs().max()) == 0.0


# ------------------------------------------------------------ with the CRF itself
def _crf(B=3, T=60):
    case = synth.make("speech", B=B, T=T)
    dev = {k: torch.from_numpy(case[k]).cuda() for k in ("em", "lengths", "trans", "dur")}
    return case, dev


def test_training_step_with_distilled_emissions():
    """One step's emission gradient: the CRF's NLL (forward, backward, gold
    path) and a distillation term added to the same buffer, against the float64
    oracle's NLL gradient plus the float64 distillation gradient."""
    from semi_markov_crf_b200 import semicrf
    case, dev = _crf()
    em, lengths, trans, dur = (dev[k] for k in ("em", "lengths", "trans", "dur"))
    B, T, C = em.shape
    K = dur.shape[0]
    logZ, ws = semicrf.forward(em, lengths, trans, dur)
    grads = semicrf.backward(ws, lengths, trans, dur)
    gold = torch.from_numpy(case["gold"]).cuda()
    starts = torch.from_numpy(case["gold_start"]).cuda()
    semicrf.path_score(em, lengths, trans, dur, gold, starts, ws=ws, negate=True, grads=grads)
    ids, teacher, _ = _teacher(torch.from_numpy(case["em"]), 5, 3)
    w = torch.full((B,), 0.3, dtype=torch.float64)
    semicrf.distill_loss(em, lengths, ids.cuda(), teacher.cuda(), temperature=2.0,
                         grad_loss=w.cuda(), accumulate=True,
                         out={"grad_logits": grads["grad_em"]})
    fb = oracle.forward_backward(case["em"], case["lengths"], case["trans"], case["dur"], K)
    cnt = oracle.path_counts(case["lengths"], case["gold"], case["gold_start"], C, K)
    want = torch.from_numpy(fb["grad_e"] - cnt["grad_em"])
    want = want + ref.distill_loss(torch.from_numpy(case["em"]), case["lengths"], ids, teacher,
                                   None, 2.0, w)["grad_logits"]
    # 1e-4 for the recursions' posteriors (as the backward's own parity tests) + the term's own
    _check("grad_em", grads["grad_em"], want, 1e-4 + 2 * (3 * lse_tol(C) + 12 * U))


def test_preference_step_on_segmentations():
    """Decoded against gold segmentations: path scores -> preference loss ->
    path-score gradients, against differences of the loss in the emissions.
    The scores are linear in the emissions and float64, so a step h truncates
    h^2 / 6 * 0.1 |du|^3 (the logistic's third derivative is below 0.1, |du| < 4
    per pair here: below 1e-5 over the batch); the gradient's float32 entries,
    at most 0.05 and with two roundings, give 2 u * 0.05 * |step| summed, below
    2e-4 for 7020 entries of |step| <= 4."""
    from semi_markov_crf_b200 import semicrf
    case, dev = _crf()
    em, lengths, trans, dur = (dev[k] for k in ("em", "lengths", "trans", "dur"))
    gold = (torch.from_numpy(case["gold"]).cuda(), torch.from_numpy(case["gold_start"]).cuda())
    _, lab, seg = semicrf.viterbi(em * 0.3, lengths, trans, dur)

    def loss_of(e):
        c = semicrf.path_score(e, lengths, trans, dur, *gold)
        r = semicrf.path_score(e, lengths, trans, dur, lab, seg)
        return semicrf.preference_scores(c, r, beta=0.05)

    out = loss_of(em)
    grads = {"grad_em": torch.zeros_like(em)}
    semicrf.path_score(em, lengths, trans, dur, *gold, grad_score=out["grad_chosen"], grads=grads)
    semicrf.path_score(em, lengths, trans, dur, lab, seg, grad_score=out["grad_rejected"],
                       grads=grads)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    step = torch.zeros_like(em).normal_(generator=g).clamp_(-4, 4)
    h = 2.0 ** -7
    up, down = em + h * step, em - h * step
    moved = (loss_of(up)["loss"] - loss_of(down)["loss"]).sum().item() / (2 * h)
    slope = (grads["grad_em"].double() * (up.double() - down.double())).sum().item() / (2 * h)
    assert abs(slope) > 1e-2
    assert abs(moved - slope) <= 2.1e-4, (moved, slope)


def test_policy_step_on_segmentations():
    """log-probability = path score - log Z: the loss at the library's own
    log-probabilities (float64: 1e-12), and the gradient through both scores
    against the float64 oracle's expected and gold counts, at the backward
    pass's own tolerance for counts."""
    from semi_markov_crf_b200 import semicrf
    case, dev = _crf()
    em, lengths, trans, dur = (dev[k] for k in ("em", "lengths", "trans", "dur"))
    C, K = trans.shape[0], dur.shape[0]
    gold = (torch.from_numpy(case["gold"]).cuda(), torch.from_numpy(case["gold_start"]).cuda())
    adv = torch.tensor([1.0, -0.5, 2.0], dtype=torch.float64).cuda()
    logZ, ws = semicrf.forward(em, lengths, trans, dur)
    logp = semicrf.path_score(em, lengths, trans, dur, *gold, ws=ws) - logZ
    old = logp + torch.tensor([0.05, -0.1, -0.5], dtype=torch.float64).cuda()
    out = semicrf.policy_scores(logp, old, adv, ref_logp=old - 0.1, kl_coef=0.1)
    for i in range(3):
        loss, kl, slope, _ = ref.policy_term(float(logp[i]), float(old[i]), float(adv[i]),
                                             float(old[i]) - 0.1, 0.2, 0.2, 0.1)
        assert abs(out["loss"][i].item() - loss) <= 1e-12
        assert abs(out["grad_logp"][i].item() - slope) <= 1e-12
    grads = semicrf.backward(ws, lengths, trans, dur, grad_logZ=-out["grad_logp"])
    semicrf.path_score(em, lengths, trans, dur, *gold, ws=ws, grad_score=out["grad_logp"],
                       grads=grads)
    g = out["grad_logp"].cpu().numpy()
    fb = oracle.forward_backward(case["em"], case["lengths"], case["trans"], case["dur"], K,
                                 grad_logZ=-g)
    cnt = oracle.path_counts(case["lengths"], case["gold"], case["gold_start"], C, K)
    gold_trans = torch.from_numpy((g[:, None, None] * cnt["trans_count"]).sum(0))
    want = torch.from_numpy(fb["grad_trans"]) + gold_trans
    tol = 1e-4 * torch.maximum(torch.ones(()), gold_trans.abs()) * 4  # |g| < 4
    _check("grad_trans", grads["grad_trans"], want, tol)
