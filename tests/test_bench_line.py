"""The benchmark's line stays short: its tables go to stderr."""
import importlib.util
import json
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bench():
    spec = importlib.util.spec_from_file_location("bench_line", os.path.join(ROOT, "bench.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_tables_leave_the_line():
    table = {f"kernel_{i}": {"launches": 20, "avg_us": 62.33120169490576, "bound": "tensor",
                             "note": "a re-read or layout pass"} for i in range(12)}
    e2e = {"value": 7380.0, "unit": "us/layer", "h2d_bytes_per_step": 1, "d2h_bytes_per_step": 2,
           "median_us": 7380.0, "steps_us": [7380.0] * 500}
    layer = {"us_per_layer": 180.0, "kernels": table, "rows": table, "clocks": {}, "e2e": e2e}
    full = {"metric": "m", "value": 1720.0, "unit": "us/layer", "n_gpus": 1, "steps": 20,
            "warmup": 5, "ms_per_step": 1.72, "config": {"workload": "w"}, "roofline": {"frac": 0.9},
            "rows": table, "kernels": table, "variants": table, "gpu_launches": 200,
            "clocks": {"sm_mhz": 2070.0}, "e2e": e2e, "cpu_baseline": {"value": 1.0},
            "per_workload": {f"layer-{i}": layer for i in range(4)}}
    line, details = _bench().split_line(full)
    assert len(json.dumps(line)) < 2500
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "config",
                "roofline", "gpu_launches", "clocks", "cpu_baseline"):
        assert line[key] == full[key], key
    assert {k: line["e2e"][k] for k in ("value", "unit", "h2d_bytes_per_step",
                                        "d2h_bytes_per_step")} == {
        k: e2e[k] for k in ("value", "unit", "h2d_bytes_per_step", "d2h_bytes_per_step")}
    assert line["per_workload"]["layer-2"] == {"us_per_layer": 180.0, "e2e_us": 7380.0}
    assert details["per_workload"] == full["per_workload"] and details["kernels"] == table
    assert details["rows"] == details["variants"] == table
    assert details["e2e_steps_us"] == e2e["steps_us"]
