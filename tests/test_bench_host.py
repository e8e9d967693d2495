"""Host-side logic of bench.py that needs no GPU: the tensor peak chosen from the sampled clocks,
and the kernel each problem takes under the library's documented dispatch rule."""
import bench

PEAKS = {"hbm_gbs": 6541.8, "bf16_tflops": 1624.0, "bf16_tflops_sustained": 1366.7}


def test_full_clock_takes_the_burst_peak():
    peak, kind = bench.fp8_tensor_peak(PEAKS, {"sm_mhz": 1965, "sm_max_mhz": 1965, "reasons": []})
    assert peak == 2 * 1624.0 and kind.startswith("bf16_tflops (burst")


def test_power_cap_takes_the_sustained_peak():
    peak, kind = bench.fp8_tensor_peak(PEAKS, {"sm_mhz": 1717, "sm_max_mhz": 1965, "reasons": ["sw_power_cap"]})
    assert peak == 2 * 1366.7 and kind.startswith("bf16_tflops_sustained")
    # a power-cap reason alone is enough, even at a clock near the maximum
    assert bench.fp8_tensor_peak(PEAKS, {"sm_mhz": 1950, "sm_max_mhz": 1965,
                                         "reasons": ["sw_power_cap"]})[0] == 2 * 1366.7


def test_low_clock_without_a_reason_takes_the_sustained_peak():
    assert bench.fp8_tensor_peak(PEAKS, {"sm_mhz": 1500, "sm_max_mhz": 1965, "reasons": []})[0] == 2 * 1366.7


def test_no_clock_samples_take_the_burst_peak():
    assert bench.fp8_tensor_peak(PEAKS, {"sm_mhz": None, "sm_max_mhz": None, "reasons": []})[0] == 2 * 1624.0


def test_missing_sustained_figure_falls_back_to_burst():
    peaks = {"hbm_gbs": 1.0, "bf16_tflops": 100.0}
    assert bench.fp8_tensor_peak(peaks, {"sm_mhz": 1000, "sm_max_mhz": 1965, "reasons": []})[0] == 200.0


def test_every_page_configuration_is_measured():
    """The headline (prefill) plus the workloads object cover every configuration of the pages:
    the 64x2112x7168 C = 0 decode shape, decode M = 64 and 128 cold and warm, contiguous, masked."""
    keys = {k for k, _, _ in bench.SUB_WORKLOADS}
    assert {"config1", "decode64_cold", "decode64_warm", "decode128_cold", "decode128_warm",
            "contiguous", "masked"} <= keys
    # and the rows beyond the page configurations: the other layouts and the K-grouped GEMM
    assert {"layouts", "k_grouped"} <= keys
    c1 = bench.WORKLOADS["config1"]
    assert c1["M"] == 64 and c1["shapes"] == [(2112, 7168)] and not c1["with_c"]
    for name in ("decode64", "decode128"):
        assert bench.WORKLOADS[name]["shapes"] == bench.PREFILL_SHAPES
    assert bench.WORKLOADS["contiguous"]["G"] == 8 and bench.WORKLOADS["masked"]["G"] == 16


def test_algorithmic_bytes_of_the_decode_headline_shape():
    """64x2112x7168 with C = 0: A and B e4m3, their fp32 scales, D bf16 (15.9 MB)."""
    p = {"kind": "dense", "rows": 64, "N": 2112, "K": 7168, "G": 1, "with_c": False}
    kb, nb = 56, 17
    assert bench.algorithmic_bytes(p) == 64 * 7168 + 4 * 64 * kb + 2112 * 7168 + 4 * nb * kb + 2 * 64 * 2112


def test_stored_traffic_is_dropped_when_the_kernels_change(tmp_path, monkeypatch):
    import json
    prof = tmp_path / "profiles"
    prof.mkdir()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    monkeypatch.setattr(bench, "source_digest", lambda: "f" * 40)     # the current kernels' digest
    (prof / "traffic.json").write_text(json.dumps({
        "prefill": {"bytes_per_launch": 123.0, "source_sha1": "f" * 40},
        "decode64": {"bytes_per_launch": 7.0, "source_sha1": "0" * 40}}))
    assert bench.stored_traffic("prefill") == 123.0
    assert bench.stored_traffic("decode64") is None
    assert bench.stored_traffic("masked") is None


def test_k_grouped_problem_sizes_and_bytes():
    """The K-grouped workload: G = 8 groups of U{2048..6144} tokens padded to 128, gradient
    shapes (M,N) from the expert weights; bytes = both e4m3 operands, their per-channel scales
    and the fp32 D."""
    probs = bench.make_problems(dict(bench.WORKLOADS["k_grouped"], shapes=[(256, 128)]))
    (p,) = probs
    assert len(p["ks"]) == 8 and all(k % 128 == 0 and 2048 <= k <= 6144 + 127 for k in p["ks"])
    T = sum(p["ks"])
    assert p["K"] == T and p["x"].shape == (T, 256) and p["w"].shape == (T, 128)
    assert p["flops"] == 2.0 * 256 * 128 * T
    assert bench.algorithmic_bytes(p) == T * 256 + T * 128 + 4 * (T // 128) * (256 + 128) + 4 * 8 * 256 * 128


def test_source_digest_follows_the_gemm_sources(tmp_path, monkeypatch):
    """The digest changes with every file that a GEMM is built from, and with no other."""
    import os
    import shutil
    real = os.path.join(bench.ROOT, "moe_grouped_gemm_sm_b200", "csrc")
    csrc = tmp_path / "moe_grouped_gemm_sm_b200" / "csrc"
    shutil.copytree(real, csrc)
    before = bench.source_digest()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.source_digest() == before
    for name in sorted(os.listdir(csrc)):
        text = (csrc / name).read_bytes()
        (csrc / name).write_bytes(text + b"// another line\n")
        gemm = name in ("dg_api.cu", "dg_ptx.cuh") or name.startswith("dg_gemm")
        assert (bench.source_digest() != before) == gemm, name
        (csrc / name).write_bytes(text)
    # a GEMM file includes none but the ones counted
    for name in os.listdir(csrc):
        if name.startswith("dg_gemm") or name == "dg_ptx.cuh":
            for line in (csrc / name).read_text().splitlines():
                if line.startswith('#include "'):
                    assert line.split('"')[1].startswith(("dg_gemm", "dg_ptx")), (name, line)


def test_result_line_is_short_and_whole():
    """The line on standard output fits the 2.8 KB that a caller keeps of it, with every key of the contract and every
    other workload's value."""
    import json
    problem = {"N": 24576, "K": 16384, "rows": 4096, "G": 1, "layout": "nt", "flops": 309237645312.0, "gemm_us": 1351.18,
               "kernel": "gemm_kernel (CTA pairs, last-wave split 7)", "tflops": 1765.5, "roof_frac": 0.541}
    roof = {"bound": "tensor", "achieved": 1820.8, "peak": 3262.0, "unit": "TFLOP/s", "frac": 0.5582,
            "peak_source": "measured: 2 x bf16_tflops_sustained (the power cap was active or the clock below max); "
                           "fp8 = 2x bf16 nominal ratio", "frac_of_burst_peak": 0.5582, "frac_of_sustained_peak": 0.6543,
            "roofline_time_frac": 0.5994, "timing": "t" * 250, "traffic": 311666176.0,
            "kernel": "gemm_kernel (CTA pairs) + gemm_kernel (CTA pairs, last-wave split 7) (6 problems, aggregate over "
                      "launches)"}
    wl = bench.WORKLOADS["prefill"]
    result = {"metric": bench.METRIC, "value": 1635.82, "unit": "TFLOP/s", "n_gpus": 1, "steps": 200, "warmup": 10,
              "ms_per_step": 1.1576, "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "e4m3",
              "data": "synthetic",
              "config": {"workload": wl["desc"], "shapes_NK": [list(s) for s in wl["shapes"]], "parallelism": "single GPU",
                         "step": "per-token cast of A + GEMM per problem; weights cast offline",
                         "l2": max(bench.L2_TEXT.values(), key=len)},
              "roofline": roof, "per_problem": [problem] * 6, "weight_cast": {"gbs": 1650.7, "ms_total": 0.42},
              "e2e": {"value": 65.06, "unit": "TFLOP/s", "h2d_bytes_per_step": 923271168, "d2h_bytes_per_step": 638058496,
                      "steps": 5, "path": "p" * 90},
              "gpu_launches": 2600, "launch": "each step replays a CUDA graph of its launches",
              "clocks": {"sm_mhz": 1965, "sm_max_mhz": 1965, "reasons": ["sw_power_cap"], "samples": 5},
              "cpu_baseline": {"value": 0.056148, "unit": "TFLOP/s", "cores": 16, "kind": "oracle", "sample": "s" * 140},
              "workloads": {key: {"workload": "w" * 120, "value": 1234.56, "unit": "TFLOP/s", "ms_per_step": 0.0187,
                                  "steps": 30, "l2": "l" * 300, "roofline": roof, "per_problem": [problem] * 6, "clocks": {}}
                            for key, _, _ in bench.SUB_WORKLOADS}}
    line = bench.result_line(result)
    assert len(json.dumps(line)) < 2800 < len(json.dumps(result))
    assert set(result) - set(line) == {"per_problem"}
    for key in ("metric", "value", "config", "e2e", "gpu_launches", "clocks", "cpu_baseline", "vs_baseline"):
        assert line[key] == result[key]
    assert line["roofline"]["frac"] == 0.5582 and line["roofline"]["traffic"] == 311666176.0
    assert {k: w["value"] for k, w in line["workloads"].items()} == {k: 1234.56 for k in result["workloads"]}
