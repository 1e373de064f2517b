"""Rings of the label-score losses whose waits give up: the kernel ends with an
error status, the context stays usable and the next call is right.  (A warp that
gave up passes nothing on any more, and a CTA of a cluster that may still be sent
to ends last; the bounds-checking build can be told to stall.)"""

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_stalled_rings_end_with_a_status():
    env = dict(os.environ, SEMICRF_LIBRARY="check")
    res = subprocess.run([sys.executable, os.path.join(HERE, "ring_stall_child.py")], env=env,
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    cases = json.loads(res.stdout.strip().splitlines()[-1])
    assert len(cases) == 20
    for name, status, same in cases:
        assert status == [0, 5, 0] and same, (name, status, same)
