"""What the expert layer's products read of a plan (csrc/moe_plan.h), built with the host compiler: whatever a workspace holds,
experts, rows and slots stay in range, and a plan that is one stays as it is."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_bounds(tmp_path):
    exe = str(tmp_path / "moe_plan")
    src = os.path.join(ROOT, "tests", "native", "moe_plan_main.cpp")
    inc = os.path.join(ROOT, "weight_only_quantized_matmul_amd", "csrc")
    b = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-I", inc, src, "-o", exe], capture_output=True, text=True, timeout=120)
    assert b.returncode == 0, b.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout[-2000:]


def test_description_is_refused_without_a_layer():
    import ctypes

    import weight_only_quantized_matmul_amd as wq

    buf = ctypes.create_string_buffer(64)
    assert wq.lib.wq_describe_moe(None, wq.WQ_DT_F32, 1, 1, 64, buf, len(buf)) == wq.WQ_E_INVAL
