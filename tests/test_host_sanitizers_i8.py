"""The refusals of the 8-bit and AdamW calls against the copy of the library
whose host code is built with AddressSanitizer and UndefinedBehaviorSanitizer
(test_host_sanitizers.py does the same for the other calls)."""

import os
import subprocess
import sys

import pytest

from tests.test_host_sanitizers import ROOT, _build_module

FILES = ["test_abi_i8.py", "test_abi_adamw_each.py", "test_abi_adamw_shared.py", "test_abi_step_overlap.py"]


def test_refusals_pass_under_host_sanitizers(tmp_path):
    build = _build_module()
    try:
        build.asan_runtime()
    except RuntimeError as e:
        pytest.skip(str(e))
    lib = build.build_host_sanitized(str(tmp_path / "hostsan"))
    logs = tmp_path / "reports"
    logs.mkdir()
    env = build.host_sanitizer_env(lib, str(logs / "san"))
    res = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
         *(os.path.join(ROOT, "tests", f) for f in FILES)],
        cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    reports = "".join(open(p).read() for p in sorted(logs.iterdir()))
    assert not reports, reports[-6000:]
    assert res.returncode == 0 and " passed" in out and "failed" not in out, out[-6000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-6000:]
