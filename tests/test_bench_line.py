"""bench.py's one line stays short: readers that keep only the last kilobytes of
the output must still find its beginning."""

import importlib.util
import json
import os

import pytest

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bench():
    spec = importlib.util.spec_from_file_location("bench_line_under_test", os.path.join(ROOT, "bench.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_workload_entries_are_brief(bench):
    number = 0.12345678901234567
    roof = {"kernel": "finalize_positions_kernel", "bound": "mufu", "achieved": number, "peak": number,
            "unit": "Gop/s", "frac": number, "note": "x" * 200}
    entry = dict(workload="genomic", B=8, T=100000, K=1000, C=128, sum_lengths=10 ** 6,
                 edges_per_step=10 ** 12, padded_edges_per_step=10 ** 12, ms_per_step=number,
                 ms_per_step_eager=number, launch="one CUDA graph replay per step", value=number,
                 positions_per_s=number, padded_edge_evals_per_s=number, fwd_bwd_kernel_ms_per_step=number,
                 kernels={f"kernel_number_{i}": {"ms_total": number, "launches": 5, "ms_per_launch": number}
                          for i in range(14)},
                 gpu_launches_per_step=14.0, step_mufu_frac=number, roofline=roof,
                 roofline_all={f"kernel_number_{i}": roof for i in range(7)},
                 memory={"peak_bytes": 123456789, "itemised_sum": 1, "items": {"inputs": 1}, "note": "x" * 300},
                 clocks={"sm_mhz": 1965.0, "sm_max_mhz": 1965.0, "reasons": [], "samples": 2},
                 cpu_baseline={"value": number, "unit": "edge evals/s", "cores": 16, "kind": "oracle",
                               "sample": "x" * 200, "positions_per_s": number})
    out = bench.brief(entry)
    assert len(json.dumps(out)) <= 520   # four of them beside the headline's 5.5 KB: below 8 KB
    assert out["peak_hbm_bytes"] == 123456789 and out["roofline"]["frac"] == number
    assert out["cpu_baseline_value"] == number and out["clocks"]["reasons"] == []
    for k in ("value", "ms_per_step", "positions_per_s"):
        assert out[k] == entry[k]
    assert "kernels" not in out and "roofline_all" not in out
    assert len(bench.EXTRAS) * 520 + 5600 <= 8 * 1024
