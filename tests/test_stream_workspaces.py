"""The rules of the streams' workspaces (csrc/stream_workspaces.h), built with the host compiler against a memory that
records every block: a block that a captured call holds is neither freed nor given to another stream."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rules(tmp_path):
    exe = str(tmp_path / "stream_workspaces")
    src = os.path.join(ROOT, "tests", "native", "stream_workspaces_main.cpp")
    inc = os.path.join(ROOT, "weight_only_quantized_matmul_amd", "csrc")
    b = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-I", inc, src, "-o", exe], capture_output=True, text=True,
                       timeout=120)
    assert b.returncode == 0, b.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout[-2000:]
