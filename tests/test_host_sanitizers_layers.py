"""The refusals of the selective scan's, the convolution's and the norm's calls
against the copy of the library whose host code is built with AddressSanitizer and
UndefinedBehaviorSanitizer (test_host_sanitizers.py does the same for the other
calls)."""

import os
import subprocess
import sys

import pytest

from tests.test_host_sanitizers import ROOT, _build_module


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
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                          os.path.join(ROOT, "tests", "test_abi_layers.py")],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    reports = "".join(open(p).read() for p in sorted(logs.iterdir()))
    assert not reports, reports[-6000:]
    assert res.returncode == 0 and " passed" in out and "failed" not in out, out[-6000:]
