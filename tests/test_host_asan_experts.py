"""The host code of the expert, grouped and 8-bit calls under AddressSanitizer
and the undefined-behaviour checks, on the CPU (no GPU).

All of the library's sources are rebuilt with both on their host side only (the
device code is compiled as usual but never runs here), and a C driver
(tests/cabi/host_asan_experts.c), itself instrumented, exercises what returns
before the first HIP call: the choices of kernel and the sort's plan over
200000 seeded sizes each, argument validation of every call, quick returns. A
memory error or undefined operation ends the driver with a report.
"""
import os
import subprocess

from conftest import ROOT
from precision_gemm_amd import _build
from test_host_asan import INCLUDE, ROCM, _tools

DRIVER = os.path.join(ROOT, "tests", "cabi", "host_asan_experts.c")
CHECKS = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
          "-fno-omit-frame-pointer"]


def test_host_paths_under_sanitizers(tmp_path):
    hip, cc = _tools()
    # The sanitizers apply to the host side of the build only.
    host = [f for c in CHECKS for f in ("-Xarch_host", c)]
    device = ["--offload-arch=gfx950", "-fPIC"]
    objects = [str(tmp_path / (os.path.basename(s) + ".o")) for s in _build.SOURCES]
    jobs = [subprocess.Popen([hip, *device, "-O1", "-g", "-std=c++17",
                              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                              *host, "-I", INCLUDE, "-c", s, "-o", o],
                             stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
            for s, o in zip(_build.SOURCES, objects)]
    assert [j.wait(timeout=900) for j in jobs] == [0] * len(jobs)
    lib = str(tmp_path / "libsgemm_asan.so")
    subprocess.run([hip, *device, "-shared", *host, *objects, "-o", lib], check=True,
                   capture_output=True, timeout=300)
    exe = str(tmp_path / "host_asan_experts")
    subprocess.run([cc, "-std=c11", "-O1", "-g", "-Wall", "-Wextra", "-Werror", *CHECKS,
                    "-I", INCLUDE, DRIVER, "-o", exe, "-L", str(tmp_path), "-lsgemm_asan",
                    "-Wl,-rpath," + str(tmp_path), "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
                    "-Wl,-rpath," + os.path.join(ROCM, "lib")],
                   check=True, capture_output=True, timeout=300)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    out = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    assert out.returncode == 0, out.stdout + out.stderr
    assert "host checks: 0 failures" in out.stdout
    assert "runtime error" not in out.stderr and "AddressSanitizer" not in out.stderr
