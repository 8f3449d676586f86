"""The benchmark's JSON line, on the CPU: short, whatever the tables hold, with
the keys that its readers need.
"""
import json

import pytest

import bench


def result():
    """A result as large as a real one or larger."""
    row = {"us": 123.456, "GB/s": 1234.5, "frac": 0.8765, "note": "x" * 200}
    return {
        "metric": bench.METRIC, "value": 6412.34, "unit": "GB/s", "n_gpus": 8, "steps": 400, "warmup": 5, "ms_per_step": 3.2671,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f32", "data": "synthetic (seeded payloads, recipe in synth/)",
        "config": {"workload": bench.WORKLOAD_NAME, "tensors": 225, "elements": 7504658432, "bytes_in": 5938274304, "bytes_out": 15009316864,
                   "out_dtype": "bf16", "elements/s": 1.8376e13, "frac_of_8TBs": 0.8015, "l2": "inputs larger than L2 (20.9 GB moved per step)",
                   "parallelism": "replicas x8"},
        "roofline": {"bound": "hbm", "achieved": 6412.3, "peak": 6774.6, "unit": "GB/s", "frac": 0.9465,
                     "traffic": {"bytes": 20910000000, "ratio": 0.998, "source": "k_decode_whole_model.json"},
                     "peak_source": "measured copy bandwidth of this GPU model", "kernel": "k" * 300},
        "parity": {"bit_exact": True, "elements": 7504658432, "mismatches": 0, "tensors": 225, "what": "w" * 400, "first": [1] * 50},
        "payload_sha256": {"whole_model": "0" * 64, "tensors": 225, "what": "w" * 200, "first": "1" * 64, "embedding": "2" * 64},
        "cpu_baseline": {"value": 15.9012, "unit": "GB/s", "cores": 16, "kind": "oracle", "elements/s": 5.7e9, "seconds": 1.32,
                         "sample": "first 1/1 of every tensor's blocks of the same whole-model payloads (7504658432 elements, 20.948 GB in+out), "
                                   "decoded to bf16, 16 threads over 329 disjoint block ranges of about equal size", "1_core": row},
        "e2e": {"value": 123.45, "unit": "GB/s", "ms_per_step": 99.123, "steps": 5, "h2d_bytes_per_step": 5938274304,
                "d2h_bytes_per_step": 15009316864, "link_alone_GB/s": {"h2d": 89.9, "d2h": 193.1}, "gpu_launches_per_step": 96, "path": "p" * 300},
        "gpu_launches": 1200, "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": ["sw_power_cap"], "samples": 52, "power_w_max": 816.43},
        "per_workload": {f"w{i}": row for i in range(40)}, "per_workload_next_formats": {f"n{i}": row for i in range(40)},
        "fused_matmul": {"tables": {f"f{i}": row for i in range(90)}},
    }


def test_the_line_is_short_and_holds_the_contract():
    res = result()
    line = bench.result_line(res)
    assert len(line) < bench.LINE_MAX <= 2500 and "\n" not in line
    d = json.loads(line)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline", "dtype",
                "data", "gpu_launches"):
        assert d[key] == res[key], key
    assert d["config"] == res["config"] and d["clocks"] == res["clocks"]
    for key in ("value", "unit", "h2d_bytes_per_step", "d2h_bytes_per_step"):
        assert d["e2e"][key] == res["e2e"][key]
    assert d["parity"]["mismatches"] == 0 and d["roofline"]["frac"] == 0.9465 and d["cpu_baseline"]["kind"] == "oracle"
    assert "per_workload" not in d and "fused_matmul" not in d


def test_parts_that_were_not_measured_are_null():
    res = result()
    for key in ("parity", "payload_sha256", "cpu_baseline", "e2e", "per_workload", "fused_matmul"):
        res[key] = None
    d = json.loads(bench.result_line(res))
    assert d["e2e"] is None and d["parity"] is None and d["value"] == 6412.34


def test_a_line_that_grew_too_long_is_an_error():
    res = result()
    res["config"]["workload"] = "w" * bench.LINE_MAX
    with pytest.raises(RuntimeError):
        bench.result_line(res)
