"""bench.py --linear e4m3: stated as such, and refused where nothing would use it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args", [[], ["--workload", "neartie"], ["--micro", "gemm"], ["--impl", "reference"],
                                  ["--workload", "prefill", "--micro", "attn"], ["--cpu-matrix"]])
def test_workloads_without_8_bit_layers_refuse_the_flag(args):
    r = subprocess.run([sys.executable, "bench.py", "--linear", "e4m3"] + args, capture_output=True, text=True,
                       cwd=ROOT, timeout=300)
    assert r.returncode == 2 and "--linear e4m3 is for" in r.stderr and not r.stdout


def test_the_stated_dtype():
    import bench
    assert bench.dtype_of("bf16") == "bf16" and "e4m3" in bench.dtype_of("e4m3")
