"""The host code of the adapters of many requests and of the orthogonalised
step (validation, size arithmetic, the plans' layout) under AddressSanitizer
and UndefinedBehaviorSanitizer, as tests/test_train_sanitizers.py does for the
routing and AdamW: their two files built with both for the host, linked with
the library's other objects into tests/host_sanitize_adapters_driver.c."""

import os
import subprocess

import pytest

from tests.test_host_sanitizers import BUILD, PKG, ROOT, SAN, _tool

FILES = ("salr_adapters_api.cpp", "salr_muon_api.cpp")


def test_adapters_host_code_under_asan_ubsan(tmp_path):
    hipcc = _tool("hipcc", os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc")
    cc = _tool("gcc", "/usr/bin/gcc")
    if not hipcc or not cc:
        pytest.skip("hipcc and gcc are needed")
    objs = sorted(os.path.join(BUILD, f) for f in os.listdir(BUILD)) if os.path.isdir(BUILD) else []
    objs = [o for o in objs if o.endswith(".o") and not o.endswith(tuple(f + ".o" for f in FILES))]
    if not objs:
        pytest.skip("library objects not built (python -m sparse_rank_linear_amd.build)")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc")]
    drv_o, exe = tmp_path / "drv.o", tmp_path / "drv"
    run = lambda cmd: subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    api = []
    for f in FILES:
        api.append(str(tmp_path / (f + ".o")))
        r = run([hipcc, "-O1", "-g", "-std=c++17", "-fPIC", *inc, *SAN, "-c", os.path.join(PKG, "csrc", f), "-o",
                 api[-1]])
        assert r.returncode == 0, r.stderr[-3000:]
    r = run([cc, "-O1", "-g", *inc, "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-c",
             os.path.join(ROOT, "tests", "host_sanitize_adapters_driver.c"), "-o", str(drv_o)])
    assert r.returncode == 0, r.stderr[-3000:]
    r = run([hipcc, "--offload-arch=gfx950", *SAN[:4], "-o", str(exe), str(drv_o), *api, *objs])
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1",
               HIP_VISIBLE_DEVICES="")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert "AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-3000:]
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout, r.stderr[-3000:])
