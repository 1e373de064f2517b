"""CPU checks of the training losses over label scores: the host side refuses
bad arguments before anything is launched, the binding refuses tensors it
cannot take, and the float64 reference statements agree with differences of
themselves (no GPU needed for any of this)."""

import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import loss_reference as ref

VP, U, D, LL, SZ = ctypes.c_void_p, ctypes.c_uint, ctypes.c_double, ctypes.c_int64, ctypes.c_size_t
FAKE, OTHER, WS = 1 << 30, 1 << 40, 1 << 20  # never dereferenced: every call fails its checks first


@pytest.fixture(scope="module")
def lib():
    from semi_markov_crf_b200 import build
    build.build()
    from semi_markov_crf_b200 import semicrf
    return semicrf.lib


def _logprob(lib, **kw):
    a = dict(logits=FAKE, dtype=0, ld=9, lengths=FAKE, labels=FAKE, B=2, T=3, V=9, tau=1.0, flags=0,
             ws=WS, nbytes=1 << 30, grad_logp=None, logp=FAKE, score=FAKE, g=OTHER, ldg=9)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.semicrf_label_logprob(*a.values(), None)


BAD_ROWS = [
    (dict(logits=None), 1), (dict(lengths=None), 1), (dict(labels=None), 1), (dict(ws=None), 1),
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(ld=8), 1), (dict(ldg=8), 1), (dict(B=-1), 1),
    (dict(T=-1), 1), (dict(V=0), 1), (dict(tau=0.0), 1), (dict(tau=-1.0), 1),
    (dict(tau=math.nan), 1), (dict(tau=math.inf), 1), (dict(tau=1e-4), 1), (dict(tau=2e3), 1),
    (dict(flags=0x1), 1), (dict(flags=0x20), 1), (dict(flags=0x40), 1), (dict(ws=WS + 8), 1),
    (dict(dtype=1, flags=0x10), 1), (dict(logits=FAKE + 2), 1), (dict(g=OTHER + 1), 1),
    (dict(dtype=1, logits=FAKE + 1), 1), (dict(g=FAKE), 1), (dict(g=FAKE + 4 * 50), 1),
    (dict(ld=1 << 61), 1), (dict(nbytes=300), 3),
    (dict(V=(1 << 24) + 1, ld=1 << 25, ldg=1 << 25), 2), (dict(B=1 << 21), 2),
    (dict(B=1 << 14, T=1 << 14), 2),
]


@pytest.mark.parametrize("change,code", BAD_ROWS, ids=lambda v: str(v))
def test_row_arguments_are_refused(lib, change, code):
    assert _logprob(lib, **change) == code


def _policy(lib, lo=0.2, hi=0.2, c=0.0, old=FAKE, adv=FAKE, flags=0):
    return lib.semicrf_policy_loss(FAKE, 0, 9, FAKE, FAKE, 2, 3, 9, 1.0, old, None, adv, 0, lo, hi, c,
                                   flags, WS, 1 << 30, None, None, None, None, None, OTHER, 9, None)


def test_policy_arguments_are_refused(lib):
    for kw in (dict(lo=-0.1), dict(lo=1.1), dict(hi=-0.1), dict(lo=math.nan), dict(hi=math.nan),
               dict(c=math.nan), dict(c=math.inf), dict(old=None), dict(adv=None), dict(flags=0x20)):
        assert _policy(lib, **kw) == 1, kw


def _preference(lib, B=2, beta=0.1, margin=0.0, smoothing=0.0, flags=0):
    return lib.semicrf_preference_loss(FAKE, 0, 9, FAKE, FAKE, B, 3, 9, 1.0, None, beta, margin,
                                       smoothing, flags, WS, 1 << 30, None, None, None, None, OTHER, 9,
                                       None)


def test_preference_arguments_are_refused(lib):
    for kw in (dict(B=3), dict(beta=math.nan), dict(beta=math.inf), dict(margin=math.nan),
               dict(smoothing=-0.1), dict(smoothing=1.1), dict(smoothing=math.nan), dict(flags=0x8)):
        assert _preference(lib, **kw) == 1, kw


def _distill(lib, k=2, ids=FAKE, teacher=FAKE):
    return lib.semicrf_distill_loss(FAKE, 0, 9, FAKE, ids, teacher, None, k, 2, 3, 9, 1.0, 0, WS,
                                    1 << 30, None, None, None, OTHER, 9, None)


def test_distill_arguments_are_refused(lib):
    assert _distill(lib, k=0) == 1 and _distill(lib, k=-1) == 1
    assert _distill(lib, k=1025) == 2
    assert _distill(lib, ids=None) == 1 and _distill(lib, teacher=None) == 1


def test_path_form_arguments_are_refused(lib):
    def policy(n=4, logp=FAKE, old=FAKE, adv=FAKE, lo=0.2, hi=0.2, c=0.0):
        return lib.semicrf_policy_scores(logp, old, None, adv, n, lo, hi, c, None, FAKE, None, None,
                                         None)

    def pairs(n=4, chosen=FAKE, rejected=FAKE, rc=None, rr=None, beta=0.1, margin=0.0, smooth=0.0):
        return lib.semicrf_preference_scores(chosen, rejected, rc, rr, n, beta, margin, smooth, None,
                                             FAKE, None, None, None)

    for kw in (dict(n=-1), dict(logp=None), dict(old=None), dict(adv=None), dict(lo=2.0),
               dict(hi=-1.0), dict(c=math.nan)):
        assert policy(**kw) == 1, kw
    for kw in (dict(n=-1), dict(chosen=None), dict(rejected=None), dict(rc=FAKE), dict(rr=FAKE),
               dict(beta=math.nan), dict(margin=math.inf), dict(smooth=1.5)):
        assert pairs(**kw) == 1, kw
    assert policy(n=0, logp=None) == 0 and pairs(n=0) == 0  # nothing to do, nothing launched


def test_workspace_bytes(lib):
    from semi_markov_crf_b200 import semicrf
    assert semicrf.loss_workspace_bytes(0, 0) >= 256
    assert semicrf.loss_workspace_bytes(4, 100) < semicrf.loss_workspace_bytes(4, 1000)
    for args in ((-1, 4), (4, -1)):
        with pytest.raises(semicrf.SemiCRFError) as info:
            semicrf.loss_workspace_bytes(*args)
        assert info.value.code == 1
    with pytest.raises(semicrf.SemiCRFError) as info:
        semicrf.loss_workspace_bytes(1 << 14, 1 << 14)
    assert info.value.code == 2


def test_the_binding_refuses_what_it_cannot_take(lib):
    from semi_markov_crf_b200 import semicrf
    x = torch.zeros(2, 3, 5)
    n = torch.zeros(2, dtype=torch.int32)
    y = torch.zeros(2, 3, dtype=torch.int32)
    f = torch.zeros(2, 3)
    with pytest.raises(TypeError):
        semicrf.label_logprob(x, n, y)      # not on a GPU
    with pytest.raises(TypeError):
        semicrf.policy_loss(x, n, y, f, f)
    with pytest.raises(TypeError):
        semicrf.preference_loss(x, n, y)
    with pytest.raises(TypeError):
        semicrf.distill_loss(x, n, torch.zeros(2, 3, 2, dtype=torch.int32), torch.zeros(2, 3, 2))
    with pytest.raises(TypeError):
        semicrf.policy_scores(torch.zeros(2).double(), torch.zeros(2).double(), torch.zeros(2).double())
    with pytest.raises(TypeError):
        semicrf.preference_scores(torch.zeros(2).double(), torch.zeros(2).double())


def test_row_strides():
    """Which layouts the binding takes, and the row stride it passes on."""
    from semi_markov_crf_b200.semicrf import _row_stride
    assert _row_stride(torch.empty(2, 3, 5), "x") == 5
    assert _row_stride(torch.empty(2, 3, 8)[..., :5], "x") == 8
    assert _row_stride(torch.empty(2, 9, 5)[:1, :3], "x") == 5
    assert _row_stride(torch.empty(4, 1, 5)[::2], "x") == 10
    assert _row_stride(torch.empty(1, 1, 5), "x") == 5
    assert _row_stride(torch.empty(0, 3, 5), "x") == 5
    for bad in (torch.empty(2, 9, 5)[:, :3], torch.empty(2, 3, 5).transpose(1, 2),
                torch.empty(1, 1, 5).expand(2, 3, 5), torch.empty(2, 3, 10)[..., ::2],
                torch.empty(5, 3, 2).permute(2, 1, 0)):
        with pytest.raises(TypeError):
            _row_stride(bad, "x")


def test_reference_gradients_agree_with_differences():
    """The float64 statements the GPU tests compare with: h = 1e-5 truncates
    below 1e-9 and rounds below 1e-10 at losses of a few units."""
    g = torch.Generator()
    g.manual_seed(0)
    B, T, V = 2, 3, 6
    x = torch.randn(B, T, V, generator=g, dtype=torch.float64)
    lens = [3, 2]
    y = torch.tensor([[1, -1, 4], [0, 5, 3]])
    old = torch.randn(B, T, generator=g, dtype=torch.float64) * 0.1 - 1.8
    adv = torch.tensor([1.0, -1.0])
    ids = torch.tensor([[[0, 1, -1], [2, 2, 3], [5, 0, 1]], [[1, 2, 3], [-1, -1, -1], [0, 0, 0]]])
    teacher = torch.randn(B, T, 3, generator=g, dtype=torch.float64)
    lse = teacher.logsumexp(-1) + 0.3
    w = torch.tensor([0.7, 1.3], dtype=torch.float64)
    losses = {
        "logprob": lambda z: ref.label_logprob(z, lens, y, 1.3),
        "policy": lambda z: ref.policy_loss(z, lens, y, old, adv, old - 0.1, 0.2, 0.3, 0.1, 1.3),
        "preference": lambda z: ref.preference_loss(z, lens, y, old, 0.5, 0.1, 0.1, True, 1.3),
        "distill": lambda z: ref.distill_loss(z, lens, ids, teacher, None, 1.3),
        "distill_mass": lambda z: ref.distill_loss(z, lens, ids, teacher, lse, 1.3),
    }
    h = 1e-5
    for name, f in losses.items():
        key = "score" if name == "logprob" else "loss"
        grad = f(x)["grad_logits"]
        for _ in range(4):
            e = torch.randn(B, T, V, generator=g, dtype=torch.float64)
            moved = (f(x + h * e)[key] - f(x - h * e)[key]).sum() / (2 * h)
            assert abs(moved - (grad * e).sum()) <= 1e-8, name
