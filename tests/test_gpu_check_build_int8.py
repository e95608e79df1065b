"""The int8 and group norm suites under the debug build: every copy of their kernels is checked before it is
issued, and none is refused."""
import os
import subprocess
import sys

import pytest

from helpers import require_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_int8_suites_pass_under_the_check_build():
    require_gpu()
    from w4a4_rank_absorbed_b200 import build
    build.build(check=True)
    env = dict(os.environ, SVDQ_LIBRARY="check")
    res = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "tests/test_gpu_int8.py",
                          "tests/test_gpu_group_norm.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-2000:]
