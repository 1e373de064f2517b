"""Runs the label-score losses through the bounds-checking build, on widths,
layouts and forms that reach every row kernel, and checks status words and
outputs.  Prints one JSON line.  Started by tests/test_gpu_loss_bounds.py in a
process of its own."""

import json
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import torch

from semi_markov_crf_b200 import semicrf
from test_gpu_loss_edges import OPS, Problem, _scores

SIZES = [(4, 5, 1), (4, 5, 6), (4, 5, 39), (2, 300, 128), (4, 3, 257), (4, 3, 1000), (4, 3, 2047),
         (4, 3, 2048), (4, 3, 5000), (2, 40, 8192), (2, 60, 9001), (4, 1, 32768), (2, 70, 40000),
         (2, 2, 131072), (2, 30, 140001), (2, 2, 600001)]


def main():
    assert semicrf.library_path.endswith("libsemicrf_b200_check.so"), semicrf.library_path
    calls = 0
    for B, T, V in SIZES:
        for dtype, pad, other in ((torch.float32, 0, 0), (torch.float32, 1, 2), (torch.bfloat16, 0, 0),
                                  (torch.bfloat16, 3, 3), (torch.float16, 5, 0)):
            p = Problem(_scores(B, T, V, dtype, V, pad), [T, 0, max(1, T - 1), T][:B], tau=1.5, seed=V,
                        k=min(V, [1, 7, 40, 140, 600][(V + pad) % 5]), lse=V % 2 == 1)
            for op in OPS:
                for kw in (dict(pad=other), dict(grad=False)) + \
                        ((dict(accumulate=True),) if dtype is torch.float32 else ()):
                    ws = semicrf.LossWorkspace(B, T)
                    out = p.call(op, ws=ws, **kw)
                    status = semicrf.get_status(ws)
                    assert status == 0, (B, T, V, dtype, pad, op, kw, status & 0xff, status >> 8)
                    if T < 10:
                        p.check(op, out, accumulated="accumulate" in kw)
                    calls += 1
    torch.cuda.synchronize()
    print(json.dumps({"calls": calls, "digest": semicrf.source_digest()}), flush=True)


if __name__ == "__main__":
    main()
