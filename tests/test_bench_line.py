"""bench.py's JSON line: short enough that the end of a run's output holds all of it, with every key that is read."""
import json

import bench

CONFIG = {"workload": "b256: long-context batch 256: every sequence 2048 tokens (128 pages), 16 layers, 32 Q / 8 KV heads, "
                      "head_dim 64, pool of 524288 pages (32 KiB BF16 or 17 KiB FP8 each), random page permutation",
          "batch": 256, "layers": 16, "seq_len_max": 2048, "seq_len_mean": 2048.0, "pages_per_chunk": 128,
          "kernel_variant": "default", "cuda_graph": True, "path": "fused", "pdl": True, "ring": 3, "sorted_units": False,
          "split_merge": False, "chains": 2, "pipelined": False, "steps_per_graph": 25, "kv_pages": "bf16",
          "kv_bytes_per_step": 17179869184, "l2": "inputs larger than L2 (17.18 GB of KV per step vs 129 MB L2), no flush",
          "seed": 12}
LONG = "how it was measured, at length; " * 12


def fields():
    return {"value": 7260.426582453431, "unit": "GB/s", "ms_per_step": 2.366234130859375, "steps": 400,
            "hbm_frac_of_peak": 1.0881608138924838, "hbm_frac_of_nominal": 0.9190413395510673,
            "hbm_frac_of_read_ceiling": 0.9774316441968942, "steps_per_s": 422.6124475612345,
            "tokens_per_s": 108188.78657564, "attended_kv_tokens_per_s": 3545090122.5106,
            "dtype": "fp8e4m3 KV, f16 MMA, f32 softmax", "config": CONFIG,
            "roofline": {"bound": "hbm", "achieved": 7260.426582453432, "peak": 6672.2, "unit": "GB/s", "frac": 1.088160813892484,
                         "traffic": 539714048, "kernel": LONG, "timing": LONG, "algorithmic_bytes_per_launch": 536870912,
                         "launch_alone": {"achieved": 6130.866621226505, "frac": 0.918867333297339}},
            "e2e": {"value": 7203.802274790778, "unit": "GB/s", "h2d_bytes_per_step": 25167872, "d2h_bytes_per_step": 16777216,
                    "steps": 400, "ms_per_step": 2.3848335266113283,
                    "path": "DecodeEngine.run_host_steps (per step: one H2D copy; " + LONG + ")", "steps_per_graph": 8},
            "cpu_baseline": {"value": 2.7231611526494452, "unit": "GB/s", "cores": 16, "kind": "oracle", "sample": LONG,
                             "single_thread": {"value": 0.204316690408056, "unit": "GB/s", "cores": 1, "sample": LONG}},
            "gpu_launches": 25600,
            "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": ["sw_power_cap"], "samples": 2, "power_w_max": 1028.56}}


def whole():
    line = {"metric": bench.METRIC, "n_gpus": 1, "warmup": 5, "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
            "data": "synthetic", **fields(), "read_ceiling": {"gbs": 7428.0658146882015, "best_probe": "bulk_1",
                                                             "probes": {"ldg_1": 6424.975213437647}, "how": LONG},
            "nominal_hbm_gbs": 7900.0, "configs": {spec: fields() for spec in bench.EXTRA_DEFAULT}}
    return line


def test_the_line_is_short_and_has_what_is_read(capsys):
    line = whole()
    assert len(json.dumps(line)) > 4 * bench.LINE_LIMIT
    bench.print_line(line)
    out, err = capsys.readouterr()
    assert out.count("\n") == 1 and len(out) < bench.LINE_LIMIT
    got = json.loads(out)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "config", "gpu_launches", "clocks"):
        assert got[key] == line[key], key
    assert {k: got["e2e"][k] for k in ("unit", "h2d_bytes_per_step", "d2h_bytes_per_step")} == \
        {k: line["e2e"][k] for k in ("unit", "h2d_bytes_per_step", "d2h_bytes_per_step")}
    assert abs(got["e2e"]["value"] / line["e2e"]["value"] - 1) < 1e-5
    for spec in bench.EXTRA_DEFAULT:
        assert abs(got["configs"][spec]["value"] / line["configs"][spec]["value"] - 1) < 1e-5
    # everything, on standard error
    assert err.startswith("detail: ") and json.loads(err[len("detail: "):]) == line


def test_what_was_not_measured_is_left_out():
    line = whole()
    line.update(e2e=None, cpu_baseline=None, roofline=None, read_ceiling=None, configs={})
    got = bench.brief(line)
    assert got["e2e"] is got["cpu_baseline"] is got["roofline"] is got["read_ceiling"] is None and got["configs"] == {}
    del line["configs"], line["read_ceiling"]
    assert "configs" not in bench.brief(line)
