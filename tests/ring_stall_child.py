"""Runs the label-score losses through the bounds-checking build with rings that
stall on request (selftest_ring_stall): each call must end with the status of a
wait that gave up, and the next one must be right again.  Prints one JSON line.
Started by tests/test_gpu_ring_stall.py in a process of its own."""

import json
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))

import torch

from semi_markov_crf_b200 import semicrf

# a ring a group of warps, a ring a CTA, rows shared by clusters (a few rows, spread
# wide, and many)
CASES = [(4, 50, 12000, torch.bfloat16), (2, 100, 40000, torch.float32),
         (2, 1, 32768, torch.bfloat16), (2, 3, 140001, torch.float32),
         (3, 60, 140001, torch.float32)]


def main():
    assert semicrf.library_path.endswith("libsemicrf_b200_check.so"), semicrf.library_path
    out = []
    for B, T, V, dtype in CASES:
        g = torch.Generator(device="cuda")
        g.manual_seed(V)
        x = torch.randn(B, T, V, generator=g, device="cuda").to(dtype)
        n = torch.full((B,), T, dtype=torch.int32, device="cuda")
        y = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32)
        ids = torch.randint(0, V, (B, T, 30), generator=g, device="cuda", dtype=torch.int32)
        t = torch.randn(B, T, 30, generator=g, device="cuda")
        old, adv = torch.full((B, T), -9.0, device="cuda"), torch.ones(B, device="cuda")
        ws = semicrf.LossWorkspace(B, T)
        calls = {
            "logprob": lambda: semicrf.label_logprob(x, n, y, ws=ws),
            "policy": lambda: semicrf.policy_loss(x, n, y, old, adv, ws=ws),
            "distill": lambda: semicrf.distill_loss(x, n, ids, t, ws=ws),
            "distill bare": lambda: semicrf.distill_loss(x, n, ids, t, grad=False, ws=ws),
        }
        for name, call in calls.items():
            want = call()
            status = [semicrf.get_status(ws)]
            semicrf.selftest_ring_stall(2000)
            call()
            status.append(semicrf.get_status(ws))
            semicrf.selftest_ring_stall(0)
            got = call()
            status.append(semicrf.get_status(ws))
            same = all(torch.equal(got[k], v) for k, v in want.items())
            out.append([f"{name} {B}x{T}x{V}", status, same])
    print(json.dumps(out), flush=True)


if __name__ == "__main__":
    main()
