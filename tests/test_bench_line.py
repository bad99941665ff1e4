"""What bench.py prints and what its traffic figures are keyed by (CPU)."""
import json
import os

import bench


def roofline(kind):
    return {"bound": "hbm", "achieved": 6282.213850870123, "peak": 6661.3, "unit": "GB/s", "frac": 0.9430912660997287,
            "traffic": 4_682_118_912, "kernel": f"{kind}_kernel", "peak_source": "measured hbm_gbs (of measured)",
            "bytes_used_for_frac": "unique: each physical block once (+ q/out)", "unique_bytes_per_launch": 665985024,
            "algorithmic_bytes_per_launch": 665985024, "launch_ms": 0.10601119920611382, "sms": 105}


def record():
    """A record of full length: every configuration, every key."""
    cpu = {"value": 790.8459469800449, "unit": "tokens/s", "cores": 16, "kind": "oracle", "sample": "6 full passes", "seconds": 2.0}
    mode = {"ms_per_step": 0.7252345678901234, "value": 6000345.678901234}
    return {
        "metric": bench.METRIC, "value": 6000345.678901234, "unit": "tokens/s", "n_gpus": 1, "steps": 200, "warmup": 10,
        "ms_per_step": 0.7252345678901234, "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
        "dtype": "bf16 q/out, e4m3 kv",
        "data": "synthetic (seeded N(0,1) bf16 q/k/v and cache pool, seeded lengths and block permutation)",
        "config": {"workload": max((d for d, _ in bench.WORKLOADS.values()), key=len), "name": "mixed", "tokens_per_step": 4352,
                   "seed": 0, "kv_cache_dtype": "bf16",
                   "l2": "flushed between timed steps (256 MiB write + read-back, outside the step events)",
                   "step": bench.step_desc(True, True), "write": "separate", "launch": "graph", "host_plan": "x" * 150,
                   "modes": {"eager": mode, "graph": mode}, "kernel_times": "x" * 90, "side_by_side": True,
                   "parallelism": "single GPU"},
        "roofline": roofline("decode"), "roofline_extend": roofline("extend"), "cpu_baseline": cpu,
        "e2e": {"value": 4712345.678901234, "unit": "tokens/s", "h2d_bytes_per_step": 53_477_376,
                "d2h_bytes_per_step": 35_651_584, "ms_per_step": 0.9234567890123456, "path": "x" * 600},
        "gpu_launches": 1200, "kernels_ms": {}, "device_error_bits": 0, "wall_s_main_workload": 3.0, "plan": {},
        "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": ["hw_slowdown", "sw_power_cap"], "samples": 1234,
                   "source": "nvml, every ~2 ms during the timed steps"},
        "per_config": {name: {"ms_per_step": 0.10441919937729835, "roofline": roofline("decode")} for name, _, _ in bench.PER_CONFIG},
    }


def test_the_printed_line_is_short_and_whole():
    full = record()
    line = bench.short_line(full)
    text = json.dumps(line)
    assert len(text) < 2600 and "\n" not in text          # logs have kept the last 3 KB of a run
    assert json.loads(text) == line
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "gpu_launches"):
        assert line[key] == full[key], key
    for key in ("value", "unit", "h2d_bytes_per_step", "d2h_bytes_per_step"):
        assert line["e2e"][key] == full["e2e"][key], key
    assert {"workload", "l2", "parallelism"} <= line["config"].keys()
    assert {"sm_mhz", "sm_max_mhz", "reasons"} <= line["clocks"].keys()
    assert line["per_config"].keys() == full["per_config"].keys()
    assert line["per_config"]["decode"] == [0.1044, 0.943]


def test_the_printed_line_without_the_optional_parts():
    full = {**record(), "roofline_extend": None, "cpu_baseline": None, "per_config": None}
    line = bench.short_line(full)
    assert line["roofline_extend"] is None and line["cpu_baseline"] is None and "per_config" not in line


def test_traffic_figures_are_keyed_by_the_kernels_headers_too():
    names = {kind: {os.path.basename(f) for f in bench.kernel_files(kind)} for kind in bench.KERNEL_SOURCES}
    assert {"k_decode.cu", "dev.cuh", "pa_internal.h"} <= names["decode"]
    assert {"k_extend.cu", "tiles.cuh", "dev.cuh", "pa_internal.h"} <= names["extend"]
    keys = {(k[0], k[3]) for k in bench.TRAFFIC}
    assert {kind for kind, _ in keys} == set(bench.KERNEL_SOURCES) and len(keys) == 2   # one source each


def test_a_changed_header_changes_the_key(tmp_path, monkeypatch):
    (tmp_path / "k.cu").write_text('#include "a.cuh"\n#include <cstdio>\n')
    (tmp_path / "a.cuh").write_text('#include "sub/b.h"\n')
    (tmp_path / "sub").mkdir()
    (tmp_path / "sub" / "b.h").write_text('#include "../a.cuh"\n// 1\n')
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    monkeypatch.setitem(bench.KERNEL_SOURCES, "k", "k.cu")
    before = bench.source_sha("k")
    assert [os.path.basename(f) for f in bench.kernel_files("k")] == ["a.cuh", "k.cu", "b.h"]
    (tmp_path / "sub" / "b.h").write_text('#include "../a.cuh"\n// 2\n')
    assert bench.source_sha("k") != before
