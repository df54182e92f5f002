"""The benchmark's line on stdout: short, whole, and with every key that names the run."""
from __future__ import annotations

import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_the_line_is_short_and_keeps_its_keys():
    import bench

    cfg, rows = bench.describe("sweep")
    text = "path=tc M=1024 N=34816 K=5120 group=128 m_tile=256 k_chunk=128 stages=3 tmem_stages=4 issuers=1 dequant_warps=16 " \
           "split_k=1 grid=(152,1,1) persistent tail_items=24 tail_split=5 tail_grid=(120,1,1) tmem_cols=512 smem=223140"
    third = 1234.5 / 3
    table = [dict(matrix="gate_up", M=m, us=third, plan=text) for m in range(44)]
    record = {"metric": bench.METRIC, "value": third, "unit": "GB/s", "n_gpus": 1, "steps": 50, "warmup": 5, "ms_per_step": third,
              "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f16", "data": "synthetic",
              "config": dict(cfg, l2="x" * 110, timing="y" * 80, parallelism="single GPU"), "value_is": "z" * 80, "tflops": third,
              "step_roofline_frac": third, "layer_step": {str(m): third for m in range(11)}, "rows": table, "cold_launch_us": table,
              "decode_step_chain": table, "nvfp4": table, "w4a8": table,
              "roofline": dict(bound="tensor", achieved=third, peak=third, unit="TFLOP/s", frac=third, traffic=128174848,
                               traffic_source="profiles/tc_gemm_mt256_m1024_5120x34816_traffic.md", kernel=text, us_per_launch=third,
                               share_of_step=third, algorithmic_bytes=173703168, algorithmic_flops=365072220160, peak_source="w" * 64),
              "cpu_baseline": dict(value=third, unit="GB/s", cores=16, kind="oracle", cpu="0xd4f", sample="s" * 112, single_thread=table),
              "e2e": dict(value=third, unit="GB/s", h2d_bytes_per_step=134152192, d2h_bytes_per_step=213805056, ms_per_step=third, steps=10,
                          streams=8), "gpu_launches": 960,
              "clocks": dict(sm_mhz=2070.0, sm_max_mhz=2070.0, reasons=[], samples=46),
              "peaks": dict(hbm_gbs=6779.0, bf16_tflops=1912.7, bf16_tflops_sustained=1706.2, source="measured")}
    line = bench.short_line(record)
    assert len(line) < 1950 and "\n" not in line
    got = json.loads(line)
    for key in set(record) - set(bench.TABLES):
        assert key in got
    assert not set(bench.TABLES) & set(got) and "single_thread" not in got["cpu_baseline"]
    assert got["steps"] == 50 and abs(got["value"] - third) < 1e-5 * third and got["e2e"]["d2h_bytes_per_step"] == 213805056
    assert record["rows"] is table and "single_thread" in record["cpu_baseline"]
