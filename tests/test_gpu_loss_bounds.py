"""The label-score losses in the bounds-checking build: its index checks (scores
at labels and entries, vectors and single elements of rows, chunks and their
copies, slots of rings and peers, positions of sequences) find nothing on sizes
that reach every row kernel, and the outputs stay right."""

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_checked_losses_run_clean():
    env = dict(os.environ, SEMICRF_LIBRARY="check")
    res = subprocess.run([sys.executable, os.path.join(HERE, "loss_bounds_child.py")], env=env,
                         capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    out = json.loads(res.stdout.strip().splitlines()[-1])
    from semi_markov_crf_b200.build import source_digest
    assert out["calls"] == 768 and out["digest"] == source_digest()
