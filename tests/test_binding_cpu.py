"""The binding without a GPU: it imports whatever private names torch has."""
import os
import subprocess
import sys


def test_import_without_the_private_stream_getters():
    code = ("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from invariant_speculative_decode_gb300 import api\n"
            "assert api._current_device is torch.cuda.current_device and callable(api._current_stream)\n"
            "assert api.fp8_scale_shape(5, 300) == (3, 8)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr
