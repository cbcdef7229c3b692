"""The layer operators' host code (argument checks, overlap tests, work
plans) under AddressSanitizer and UndefinedBehaviorSanitizer: layers.cpp, grads.cpp,
plan.cpp and step.cpp compiled by g++ with both, linked with the device objects
as built, and tests/test_layers_cpu.py run on that library in a child process.
No GPU is touched."""

import glob
import os
import shutil
import subprocess
import sys

import pytest

from tests.test_sanitized_host import CSRC, HERE, PKG, ROOT, _gcc_runtime

HOST_SOURCES = ("plan.cpp", "step.cpp", "grads.cpp", "layers.cpp")


def test_layers_host_code_under_asan_and_ubsan(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    asan, ubsan = _gcc_runtime("libasan.so"), _gcc_runtime("libubsan.so")
    if not asan or not ubsan:
        pytest.skip("sanitizer runtimes not available")
    build_dir = os.path.join(PKG, "_build")
    if not glob.glob(os.path.join(build_dir, "*.o")):
        from muon_newton_schulz_02_amd import build as B
        B.build()
    flags = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fPIC",
             "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
             "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", CSRC,
             "-I", os.path.join(ROOT, "include")]
    objs = []
    for src in HOST_SOURCES:
        obj = str(tmp_path / (src + ".o"))
        subprocess.run(["g++", *flags, "-c", os.path.join(CSRC, src), "-o", obj], check=True)
        objs.append(obj)
    for k, obj in enumerate(sorted(glob.glob(os.path.join(build_dir, "*.o")))):
        if os.path.basename(obj).split(".")[0] + ".cpp" in HOST_SOURCES:
            continue
        dst = str(tmp_path / ("device_%d.o" % k))
        shutil.copy(obj, dst)
        objs.append(dst)
    lib = str(tmp_path / "libmuon_adamw_sanitized.so")
    subprocess.run(["g++", "-shared", "-fsanitize=address,undefined", "-o", lib, *objs,
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True)
    env = dict(os.environ)
    env["LD_PRELOAD"] = "%s %s" % (asan, ubsan)
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1:abort_on_error=0"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    driver = ("import sys; sys.path.insert(0, %r)\n"
              "import muon_newton_schulz_02_amd._abi as A\n"
              "A.load(%r)\n"
              "import pytest\n"
              "sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', %r]))\n"
              % (ROOT, lib, os.path.join(HERE, "test_layers_cpu.py")))
    res = subprocess.run([sys.executable, "-c", driver], cwd=ROOT, env=env, capture_output=True,
                         text=True, timeout=600)
    report = res.stdout[-3000:] + res.stderr[-3000:]
    assert res.returncode == 0, report
    assert "ERROR: AddressSanitizer" not in res.stderr and "runtime error" not in res.stderr, report
    assert " passed" in res.stdout, report
