"""Calls on a machine without a GPU return an error; they do not end the process."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CALL = """
import sys
sys.path[:0] = [%r, %r]
import moe_expert_ffn_sqrt_gb300 as M
import test_ws_alignment as T
assert T.calls(M)[%d]() == M.ERR_CUDA
"""


@pytest.mark.parametrize("i", range(13))
def test_a_call_without_a_device_returns(i):
    r = subprocess.run([sys.executable, "-c", CALL % (os.path.dirname(HERE), HERE, i)], capture_output=True, text=True, timeout=300,
                       env={**os.environ, "CUDA_VISIBLE_DEVICES": ""})
    assert r.returncode == 0, (r.returncode, r.stderr[-1000:])
