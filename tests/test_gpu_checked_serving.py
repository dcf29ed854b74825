"""The checked build on the serving operators' edge shapes, in a fresh process (see checked_build_serving.py)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_checked_build_serving_operators(cuda_device):
    env = dict(os.environ, DIFFQKV_BOUNDS_CHECK="1")
    r = subprocess.run([sys.executable, os.path.join(HERE, "checked_build_serving.py")], env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "all cases ok" in r.stdout
