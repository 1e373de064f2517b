"""CPU checks of the training losses over label scores: outputs that overlap an
input are refused before anything is launched (a row's inputs are read by several
warps and CTAs, one of which writes its outputs)."""

import pytest

pytest.importorskip("torch")

MB = 1 << 20
WS = 64 * MB  # addresses that are never dereferenced


@pytest.fixture(scope="module")
def lib():
    from semi_markov_crf_b200 import build
    build.build()
    from semi_markov_crf_b200 import semicrf
    return semicrf.lib


B, T, V, K = 4, 3, 9, 2
N, NB, ROWS = 4 * B * T, 4 * B, 4 * B * T * V


def _places(names, start=100 * MB):
    return {n: start + i * MB for i, n in enumerate(names)}


def logprob(lib, p):
    return lib.semicrf_label_logprob(p["logits"], 0, V, p["lengths"], p["labels"], B, T, V, 1.0, 0, WS,
                                     16 * MB, p["grad_logp"], p["logp"], p["score"], p["grad"], V, None)


def policy(lib, p):
    return lib.semicrf_policy_loss(p["logits"], 0, V, p["lengths"], p["labels"], B, T, V, 1.0, p["old"],
                                   p["ref"], p["adv"], 1, 0.2, 0.2, 0.0, 0, WS, 16 * MB, p["w"],
                                   p["loss"], p["kl"], p["clipped"], p["logp"], p["grad"], V, None)


def preference(lib, p):
    return lib.semicrf_preference_loss(p["logits"], 0, V, p["lengths"], p["labels"], B, T, V, 1.0,
                                       p["ref"], 0.1, 0.0, 0.0, 0, WS, 16 * MB, p["w"], p["loss"],
                                       p["reward"], p["logp"], p["grad"], V, None)


def distill(lib, p):
    return lib.semicrf_distill_loss(p["logits"], 0, V, p["lengths"], p["ids"], p["teacher"], p["lse"],
                                    K, B, T, V, 1.0, 0, WS, 16 * MB, p["w"], p["loss"], p["token"],
                                    p["grad"], V, None)


def policy_paths(lib, p):
    return lib.semicrf_policy_scores(p["logp"], p["old"], p["ref"], p["adv"], B, 0.2, 0.2, 0.0, p["w"],
                                     p["loss"], p["kl"], p["grad"], None)


def preference_paths(lib, p):
    return lib.semicrf_preference_scores(p["chosen"], p["rejected"], p["rc"], p["rr"], B, 0.1, 0.0, 0.0,
                                         p["w"], p["loss"], p["gc"], p["gr"], None)


# inputs and outputs of each call, with their bytes
CALLS = {
    logprob: (dict(logits=ROWS, lengths=NB, labels=N, grad_logp=N), dict(logp=N, score=NB, grad=ROWS)),
    policy: (dict(logits=ROWS, lengths=NB, labels=N, old=N, ref=N, adv=N, w=2 * NB),
             dict(loss=NB, kl=NB, clipped=NB, logp=N, grad=ROWS)),
    preference: (dict(logits=ROWS, lengths=NB, labels=N, ref=N, w=NB),
                 dict(loss=NB // 2, reward=NB, logp=N, grad=ROWS)),
    distill: (dict(logits=ROWS, lengths=NB, ids=N * K, teacher=N * K, lse=N, w=2 * NB),
              dict(loss=NB, token=N, grad=ROWS)),
    policy_paths: (dict(logp=8 * B, old=8 * B, ref=8 * B, adv=8 * B, w=8 * B),
                   dict(loss=8 * B, kl=8 * B, grad=8 * B)),
    preference_paths: (dict(chosen=8 * B, rejected=8 * B, rc=8 * B, rr=8 * B, w=8 * B),
                       dict(loss=8 * B, gc=8 * B, gr=8 * B)),
}


@pytest.mark.parametrize("call", list(CALLS), ids=lambda f: f.__name__)
def test_outputs_in_an_inputs_place_are_refused(lib, call):
    inputs, outputs = CALLS[call]
    step = 8 if call in (policy_paths, preference_paths) else 4
    for o, ob in outputs.items():
        for i, ib in inputs.items():
            for at in (0, ib - step, step - ob):  # the same place, its last element, its first
                p = _places(list(inputs) + list(outputs))
                p[o] = p[i] + at
                assert call(lib, p) == 1, (o, i, at)
