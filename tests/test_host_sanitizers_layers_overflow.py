"""The refusals of sizes near 2^63 in the selective scan's, the convolution's and the
norm's calls under AddressSanitizer and UndefinedBehaviorSanitizer.  Only the checks
(api_layers.cpp) are built again, with the objects of the normal build beside them."""

import os
import subprocess
import sys

import pytest

from tests.test_host_sanitizers import ROOT, _build_module


def test_large_sizes_pass_under_host_sanitizers(tmp_path):
    build = _build_module()
    try:
        build.asan_runtime()
    except RuntimeError as e:
        pytest.skip(str(e))
    objs = [os.path.join(build.OBJ, os.path.splitext(s)[0] + ".o") for s in build.SOURCES if s != "api_layers.cpp"]
    if not all(map(os.path.exists, objs)):
        build.build()
    objs.append(build._compile("api_layers.cpp", str(tmp_path), build.SANITIZE_HOST))
    lib = str(tmp_path / "libscanrnn_checks.so")
    subprocess.run([build._hipcc(), f"--offload-arch={build.ARCH}", "-shared", "-fPIC", "-shared-libasan",
                    "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", *objs, "-o", lib],
                   check=True, capture_output=True)
    logs = tmp_path / "reports"
    logs.mkdir()
    env = build.host_sanitizer_env(lib, str(logs / "san"))
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                          os.path.join(ROOT, "tests", "test_abi_layers_overflow.py")],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    reports = "".join(open(p).read() for p in sorted(logs.iterdir()))
    assert not reports, reports[-6000:]
    assert res.returncode == 0 and " passed" in out and "failed" not in out, out[-6000:]
