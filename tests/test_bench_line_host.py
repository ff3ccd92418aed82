"""The line that bench.py prints stays short (no GPU)."""

import json

import bench


def test_a_row_of_the_line_is_short():
    row = {"shape": "28672x8192", "M": 128, "us": 71.23, "tflops": 843.21, "gbs": 1824.5, "hbm_frac": 0.2281, "mfma_frac": 0.3373,
           "roofline_frac": 0.3373, "kernel": "wide_gemm<PolicyW4A16M32,16>", "plan": {"mb": 64, "nb": 128, "wpt": 16},
           "mfma_frac_of_achievable": 0.5123, "hbm_frac_of_achievable": 0.3011}
    short = bench.short_row(row)
    assert {"shape", "M", "us", "tflops", "hbm_frac"} <= set(short) and all(short[k] == row[k] for k in short)
    # sixteen of them, and 2 KB for everything else
    assert 16 * (len(json.dumps(short)) + 2) < 2048
