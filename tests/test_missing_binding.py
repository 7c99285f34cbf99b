"""Without the compiled binding the package loads and its other calls work; the
8-bit and AdamW calls say what is missing."""

import os
import subprocess
import sys

import pytest

pytest.importorskip("scan_linear_rnn_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.modules["scan_linear_rnn_amd._binding"] = None      # importing it raises ImportError
import torch
import scan_linear_rnn_amd as sr
x = torch.zeros(2, 3, 4)
try:
    sr.mingru_forward(k=x, p=x)
except ValueError as e:
    assert "GPU" in str(e)                               # the ctypes calls check as ever
assert sr.raw_library().scanrnn_version() and sr.quantized_row_bytes(5) == 128
calls = [lambda: sr.quantize_rows(x), lambda: sr.quantize_columns(x), lambda: sr.matmul_i8(x, x, x, x),
         lambda: sr.mingru_step_i8(x, x, x), lambda: sr.mingru_forward_i8(x, x, x),
         lambda: sr.adamw_step([x], [x], x, x, step=1), lambda: sr.AdamW([x]).step([x])]
for call in calls:
    try:
        call()
    except ImportError as e:
        assert "compiled binding" in str(e) and "build.py" in str(e)
    else:
        raise SystemExit("no error")
print("done")
"""


def test_the_other_calls_load_without_it():
    res = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.strip().endswith("done"), res.stderr[-3000:]
