"""The bench's printed line: every contract key, short enough to be read whole from a log's tail."""
import json

import bench


def full_line():
    f = 1234.5678901234567
    call = {k: f for k in ("us_per_call", "us_per_call_median", "us_per_row", "GBps", "frac_of_measured_hbm",
                           "per_row_launch_us_per_row", "us_per_call_warm_l2", "router_fused_us_per_window")}
    tile = {"us": f, "us_median": f, "TFLOPs": f, "tile": "256x128"}
    both = {k: f for k in ("gemv_us_per_row", "gemm_us_per_row", "gemv_us", "gemm_us", "gemv_us_median", "gemm_us_median",
                           "gemm_TFLOPs")}
    head = {"metric": "us_per_row", "value": f, "unit": "us/row", "n_gpus": 1, "steps": 20, "warmup": 5, "ms_per_step": f,
            "higher_is_better": False, "scaling": "weak", "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
            "config": {"workload": "w" * 200}, "gpu_launches": 100, "clocks": {"sm_mhz": f, "reasons": []},
            "roofline": {"frac": f}, "e2e": {"value": f, "h2d_bytes_per_step": 1, "d2h_bytes_per_step": 2}}
    return dict(head, curve={s: dict({str(m): call for m in (1, 2, 4, 8, 16)}, batching_speedup_m1_over_m8=f) for s in "abc"} | {"note": "n"},
                gemm={"chunk": {f"{m}x{n}": tile for m in range(8) for n in range(7)}, "narrow": {"512": dict(call)},
                      "raster_study": {"2048x6144": {str(i): tile for i in range(6)}}, "summary": {"frac_of_peak_mean": f}},
                path_sweep={s: {"curve": {str(m): both for m in range(12)}, "crossover_m": 16, "note": "n" * 80} for s in "ab"})


def test_the_line_is_short_and_keeps_the_contract():
    line = full_line()
    short = json.loads(json.dumps(bench.short_line(line)))
    assert len(json.dumps(line)) > 16000 and len(json.dumps(short)) < 8000
    for key, value in line.items():
        if key not in ("curve", "gemm", "path_sweep", "roofline", "clocks", "e2e", "value", "ms_per_step"):
            assert short[key] == value, key
    assert abs(short["value"] / line["value"] - 1) < 1e-6 and abs(short["ms_per_step"] / line["ms_per_step"] - 1) < 1e-6
    assert short["curve"]["a"]["8"] == short["value"] and short["path_sweep"] == {"a": 16, "b": 16}
    assert short["gemm"]["chunk"]["7x6"] == short["value"] and "frac_of_peak_mean" in short["gemm"]["summary"]
    assert bench.short_line(dict(line, gemm=None, path_sweep=None))["gemm"] is None
