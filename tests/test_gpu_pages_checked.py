"""The checked build (-DDSA_CHECKS=1) reports out-of-range device-side inputs of the paged
operators (GPU).  The library is chosen at its first load, so the cases run in a process of
their own (tests/pages_checked_case.py) with DSA_CHECKED=1."""
import os
import subprocess
import sys

import pytest
import torch

from dynamic_sparse_attention_gb300 import _build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_checked_build_reports_bad_pages_and_lengths():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    _build.build(checked=True)
    r = subprocess.run([sys.executable, os.path.join(HERE, "pages_checked_case.py")],
                       env=dict(os.environ, DSA_CHECKED="1"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "pages checked-build ok" in r.stdout
