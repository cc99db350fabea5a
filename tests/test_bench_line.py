"""The line that bench.py prints (no GPU): short enough for the tail of a log, with every key of a
benchmark line, and enough of each workload for --summarize."""

import copy
import json

import bench

ROOF = {"bound": "hbm", "achieved": 4141.3, "peak": 8000.0, "unit": "GB/s", "frac": 0.5177,
        "measured_read_GB_s_at": {"bytes": 41943040, "GB_s": 4976.6}, "frac_of_measured": 0.8321}
ENTRY = {"us_per_launch": 59.999, "GB_s": 3264.9, "hbm_frac": 0.4081, "TFLOP_s": 339.03, "mfma_frac": 0.1356,
         "bytes": 175027104, "flops": 18175229952, "copies": 7, "reps_us": [56.613, 53.609, 53.294],
         "spread_pct": 6.19, "kernels": ["gather_qmm_kernel<4, MmTile4<4, 2, 4, 4, 2, 1, 48, false, true>> "
                                         "grid=768x1 block=256 lds=49152"] * 2,
         "roofline": ROOF, "reconciliation": {"traced_kernel_sum_us": 63.423, "kernel_share_pct": 118.3},
         "counters": {"traffic_bytes_per_launch": 176268727.0, "MfmaUtil_pct": 24.3, "VALUBusy_pct": 44.1}}
KEYS = {"metric": "qmv HBM GB/s (% of peak); qmm & MoE gather_qmm TFLOPS (% of MFMA peak)", "value": 3850.0,
        "unit": "GB/s", "n_gpus": 1, "steps": 200, "warmup": 20, "ms_per_step": 0.014186,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
        "data": "synthetic", "config": {"workload": "w" * 160, "step": "s" * 80}}


def record():
    """A whole record of the default run's shape."""
    names = bench.suite_names()
    sizes = {str(1 << i): 4976.6 for i in range(23, 28)}
    return {**KEYS, "roofline": ROOF,
            "per_kernel": [{"workload": w, **ENTRY} for w in ("qmv_M1_K5120_N5120_b4", "qmv_M1_K5120_N13824_b4")],
            "measured_ceilings": {"read_GB_s": sizes, "read_unroll": sizes, "mfma_bf16_TFLOP_s": 2128.6,
                                  "mfma_probe": "m" * 80, "read_probe": "r" * 240},
            "suite": [{"workload": w, **ENTRY} for w in names],
            "bits_8_vs_4": [{"pair": "p" * 60, "bytes_ratio": 1.888, "time_ratio": 1.347}] * 4,
            "cpu_baseline": {"value": 1.58, "unit": "GB/s", "cores": 16, "kind": "oracle", "sample": "s" * 120,
                             "per_config": [{"workload": w, "threads": 16, "sample": "s" * 20, "seconds": 0.4,
                                             "gpu_speedup": 1834.1} for w in names]}}


def test_the_line_is_short():
    whole = record()
    assert len(json.dumps(whole)) > 16000  # the record itself outgrows a tail
    assert len(json.dumps(bench.printed(whole))) < 8000


def test_the_line_keeps_the_headline_and_each_workload(tmp_path):
    whole = record()
    before = copy.deepcopy(whole)
    line = bench.printed(whole)
    assert whole == before  # the record is not changed
    assert {k: line[k] for k in KEYS} == KEYS
    assert line["roofline"] == ROOF and line["measured_ceilings"] == whole["measured_ceilings"]
    assert line["cpu_baseline"]["value"] == 1.58 and "per_config" not in line["cpu_baseline"]
    assert [e["workload"] for e in line["suite"]] == bench.suite_names()
    log = tmp_path / "bench.log"
    log.write_text("noise\n" + json.dumps(line) + "\n")
    for name in bench.suite_names():
        assert bench.workload_bytes(str(log), name) == ENTRY["bytes"]


def test_parts_that_did_not_run():
    assert bench.printed({"suite": []}) == {"suite": []}
    assert bench.printed({**KEYS, "cpu_baseline": None}) == {**KEYS, "cpu_baseline": None}
