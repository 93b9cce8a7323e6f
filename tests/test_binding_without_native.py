"""The binding where _native.so does not load: one warning, and the calls' own checks and ctypes calls."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import sys
import warnings
import torch
sys.modules["moe_expert_ffn_sqrt_gb300._native"] = None          # an import of it fails
import moe_expert_ffn_sqrt_gb300 as M
x, w, ws = torch.ones(4, 256, dtype=torch.bfloat16), torch.ones(256), torch.zeros(4096, dtype=torch.uint8)
ids, tw, w2, q = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.ones(256, 256, dtype=torch.bfloat16), M.new_rows8(4, 256, "cpu")
calls = (lambda: M.rms_norm(x, w, 1e-6, y=x), lambda: M.rms_norm_backward(x, x, w, 1e-6, x, ws),
         lambda: M.select(x, ids, tw, "sigmoid"), lambda: M.select_backward(x, ids, tw, tw, x, ws, "sigmoid"),
         lambda: M.pack_rows8(x, q), lambda: M.unpack_rows8(q, x), lambda: M.linear_backward8(x, w2, ws, x8=q, dw=w2))
M._at_home = lambda *t: None              # (a machine without a GPU has no current device)
with warnings.catch_warnings(record=True) as told:
    warnings.simplefilter("always")
    for f in calls:
        try:
            f()
        except ValueError as e:
            assert "CUDA tensor" in str(e), e
            continue
        raise SystemExit("not refused")
assert len(told) == 1 and "_native.so" in str(told[0].message), told
print("warned once")
"""


def test_the_calls_do_without_it():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "CUDA_VISIBLE_DEVICES": ""})
    assert r.returncode == 0 and r.stdout.strip() == "warned once", r.stderr[-2000:]
