"""Host checks of bench.py's contract (no GPU): the single-GPU refusal, the
workload table and the HBM traffic record's guard."""

import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402
import pytest  # noqa: E402


def test_more_than_one_gpu_exits_with_a_message():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--gpus", "2"], capture_output=True,
                       text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 2
    assert "one GPU only" in r.stderr and r.stdout == ""


def test_headline_workload_and_units():
    assert "fp32_transpose" in bench.WORKLOADS
    for name in ("bf16_gemm", "bf16_gemm_fused", "bf16_gemm_fused_bf16c", "map_batch", "u8_narrow16", "fp32_rows3",
                 "u8_rows48"):
        assert name in bench.WORKLOADS, name


def test_traffic_bytes_only_while_the_kernel_sources_match(tmp_path, monkeypatch):
    """bench.py reports counter bytes only from a record taken on the kernel
    sources as they are now (same digest); a stale record gives null."""
    rec = {"workloads": {"fp32_transpose": {"bytes_per_launch": 123}}}
    f = tmp_path / "traffic.json"
    monkeypatch.setattr(bench, "TRAFFIC_FILE", str(f))
    f.write_text(json.dumps(dict(rec, kernel_sources_sha256=bench.kernel_sources_digest())))
    assert bench.measured_traffic("fp32_transpose") == 123
    assert bench.measured_traffic("no_such_workload") is None
    f.write_text(json.dumps(dict(rec, kernel_sources_sha256="0" * 64)))
    assert bench.measured_traffic("fp32_transpose") is None
    f.write_text("not json")
    assert bench.measured_traffic("fp32_transpose") is None


def test_conflict_counters_equal_the_models_prediction_for_every_layout():
    """The recorded SQ_LDS_BANK_CONFLICT readings (rocprofv3, one record per
    workload and layout) equal, per tile, what swz_predict_conflicts predicts
    under the built-in gfx950 bank model -- zero for every swizzled and
    direct-fill kernel ("CuTe Swizzle 学习手册", ⑥: verify with a measured
    count that the swizzle removes the conflicts)."""
    import tiled_movement_amd as T

    with open(bench.CONFLICT_FILE) as f:
        rec = json.load(f)
    rows = {"fp32_rows3", "u8_rows48"}
    assert len(rec["workloads"]) == 11 and rows <= set(rec["workloads"])
    for wname, layouts in rec["workloads"].items():
        if wname in rows:  # the flat-row kind: its reads depend on the width, so no per-kind prediction
            assert set(layouts) == {"swizzle", "plain"}, wname
            sw, pl = layouts["swizzle"], layouts["plain"]
            assert sw["conflict_cycles_per_lds_instr"] < 1e-3, wname
            assert sw["SQ_LDS_BANK_CONFLICT"] <= pl["SQ_LDS_BANK_CONFLICT"], wname
            continue
        assert set(layouts) == {"swizzle", "pad", "plain", "direct"}, wname
        for layout, r in layouts.items():
            w, rd = T.swz_predict_conflicts(r["read_kind"], layout)
            assert r["conflict_cycles_per_tile"] == pytest.approx(w + rd, abs=0.5), (wname, layout)
            if layout in ("swizzle", "direct"):
                assert r["SQ_LDS_BANK_CONFLICT"] == 0, (wname, layout)


def test_conflicts_reported_only_while_the_kernel_sources_match(tmp_path, monkeypatch):
    rec = {"workloads": {"fp32_transpose": {"swizzle": {"conflict_cycles_per_tile": 0.0, "conflict_cycles_per_lds_instr": 0.0,
                                                        "SQ_LDS_BANK_CONFLICT": 0, "SQ_LDS_IDX_ACTIVE": 1,
                                                        "SQ_INSTS_LDS": 1}}}}
    f = tmp_path / "lds.json"
    monkeypatch.setattr(bench, "CONFLICT_FILE", str(f))
    f.write_text(json.dumps(dict(rec, kernel_sources_sha256=bench.kernel_sources_digest())))
    assert bench.measured_conflicts("fp32_transpose")["swizzle"]["conflict_cycles_per_tile"] == 0.0
    assert bench.measured_conflicts("bf16_stage") is None
    f.write_text(json.dumps(dict(rec, kernel_sources_sha256="0" * 64)))
    assert bench.measured_conflicts("fp32_transpose") is None


def test_source_digest_follows_code_not_comments():
    """The counter records stay valid across comment edits of the kernel
    sources and go stale on any change of the code."""
    src = "int f(int x) {  // one\n  /* two\n three */ return x ^ 3;\n}\n"
    assert bench.code_text(src) == bench.code_text(src.replace("// one", "// changed").replace("two", "other"))
    assert bench.code_text(src) == "int f(int x) {\n   return x ^ 3;\n}"
    assert bench.code_text(src) != bench.code_text(src.replace("x ^ 3", "x ^ 5"))


def test_the_line_stays_short_whatever_is_measured():
    """One rate a workload and layout on stdout; shapes, parameters and counters only in --record's file."""
    rec = {"layout": "swizzle", "shape": [1, 8192, 8192], "elem_bytes": 4, "params": [5, 0, 5], "pad_elems": 0, "lds_bytes": 4096,
           "threads": 256, "buffer_pairs": 4, "predicted_conflict_cycles_per_tile": {"write": 96, "read": 992}, "GBps": 3977.1,
           "frac": 0.4971, "us_per_step": 33.75, "frac_of_copy": 0.6548, "measured_conflict_cycles_per_tile": 1088.0}
    cpu = {"value": 13.8, "unit": "GB/s", "cores": 16, "sample": "x" * 120, "matches_gpu": True}
    extra = {f"{w}/{lay}": dict(rec) for w in bench.WORKLOADS for lay in ("swizzle", "pad", "plain", "direct")}
    extra.update({"map/swizzle": {"us_per_call": 1.9, "batch_us_per_125_triples": 6.5}, "torch_mm_bf16": {"TFLOPs": 1311.7, "m": 8192},
                  "fp32_transpose_long/swizzle": {"shape": [1, 8192, 2048], "GBps_default_order": 4700.0, "GBps_tuned_order": 5790.0},
                  "cpu_baseline": {w: dict(cpu) for w in bench.ORACLE_TIMED}})
    line = {"metric": bench.METRIC, "value": 5669.2, "config": {"workload": bench.WORKLOADS["fp32_transpose"]}, "cpu_baseline": cpu,
            "extra": extra}
    out = bench.short(line)
    assert len(json.dumps(line)) > 16000 > 4 * len(json.dumps(out))
    assert {k: v for k, v in out.items() if k != "extra"} == {k: v for k, v in line.items() if k != "extra"}
    assert out["extra"]["fp32_transpose/plain"] == 3977.1 and out["extra"]["torch_mm_bf16"] == 1311.7
    assert out["extra"]["map/swizzle"] == 1.9 and out["extra"]["fp32_transpose_long/swizzle"] == 5790.0
    assert set(out["extra"]["cpu_baseline"].values()) == {13.8} and line["extra"]["fp32_transpose/plain"] == rec
    assert bench.short({"extra": {}}) == {"extra": {}}
