"""The launches of the adapters of many requests at sizes up to the largest
that the entry points take: salr_adapters_api.cpp built with the launchers of
tests/host_adapters_launches_driver.cpp, which check that a launch has fewer
than 2^32 threads and that what the kernels write lies in the workspace."""

import os
import subprocess

import pytest

from tests.test_host_sanitizers import PKG, ROOT, _tool


def test_launches_fit(tmp_path):
    hipcc = _tool("hipcc", os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc")
    if not hipcc:
        pytest.skip("hipcc is needed")
    exe = str(tmp_path / "launches")
    r = subprocess.run([hipcc, "-O1", "-std=c++17", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.join(PKG, "csrc"), os.path.join(PKG, "csrc", "salr_adapters_api.cpp"),
                        os.path.join(ROOT, "tests", "host_adapters_launches_driver.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout, r.stderr[:3000])
