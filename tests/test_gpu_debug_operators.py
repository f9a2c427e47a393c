"""The fused-epilogue, grouped and row operators in the debug build (liblq_debug.so, LQ_DEBUG=1): their GPU tests
run in a child process, whose last check is that lq_get_device_status reports no access outside a buffer."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_operators_in_the_debug_build():
    env = dict(os.environ, LQ_DEBUG="1")
    env.pop("LQ_FAULT", None)
    which = "layer_epilogue or cut_along_k or grouped or group_rows or combine_rows or few_steps"
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_operators.py", "-m", "gpu", "-x", "-q", "-k", which],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert " passed" in r.stdout
