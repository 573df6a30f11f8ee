"""The operators around the feed-forward block under the checks library (device-side index checks, DG_CHECKS=1):
their tests again, in a child process; no check may fire (dg_device_error() is 0 where they look)."""
import os
import subprocess
import sys

import pytest

from discrete_diffusion_lm_b200 import build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_block_operators_under_the_checks_library():
    build.build(checks=True)
    env = dict(os.environ, DG_LIB="checks")
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_block_ops.py", "-x", "-q", "-m", "gpu", "-k",
                        "norm_forward or norm_row or norm_backward or quantize or product or test_block or path"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]
