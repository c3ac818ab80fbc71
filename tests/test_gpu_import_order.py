"""The library loaded before the program imports torch (needs an MI355X)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sizes_asked_before_torch_is_imported():
    code = ("import post_weight_quantization_accum_amd as P; assert P.mx_codes_per_row(128) == 64 and P.version();"
            "import torch; c, s = P.mx_quantize(torch.ones(2, 128, device='cuda'));"
            "assert s.tolist() == [[125] * 4] * 2 and (c == 0x66).all()")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
