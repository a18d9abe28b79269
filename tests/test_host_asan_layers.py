"""The host code of the norms, the 4-bit calls and the experts' layer under
AddressSanitizer and the undefined-behaviour checks, on the CPU (no GPU), as
test_host_asan_experts.py does for the calls before them: the three sources are
rebuilt with both on their host side only, and an instrumented C driver
(tests/cabi/host_asan_layers.c) exercises what returns before the first HIP
call."""
import os
import subprocess

from conftest import ROOT
from precision_gemm_amd import _build
from test_host_asan import INCLUDE, ROCM, _tools

DRIVER = os.path.join(ROOT, "tests", "cabi", "host_asan_layers.c")
CHECKS = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
          "-fno-omit-frame-pointer"]


def test_host_paths_under_sanitizers(tmp_path):
    hip, cc = _tools()
    host = [f for c in CHECKS for f in ("-Xarch_host", c)]
    device = ["--offload-arch=gfx950", "-fPIC"]
    sources = [os.path.join(_build.CSRC, f)
               for f in ("norm.hip", "mx4gemm.hip", "expert_layer.hip")]
    objects = [str(tmp_path / (os.path.basename(s) + ".o")) for s in sources]
    jobs = [subprocess.Popen([hip, *device, "-O1", "-g", "-std=c++17",
                              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                              *host, "-I", INCLUDE, "-c", s, "-o", o],
                             stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
            for s, o in zip(sources, objects)]
    assert [j.wait(timeout=900) for j in jobs] == [0] * len(jobs)
    lib = str(tmp_path / "liblayers_asan.so")
    subprocess.run([hip, *device, "-shared", *host, *objects, "-o", lib], check=True,
                   capture_output=True, timeout=300)
    exe = str(tmp_path / "host_asan_layers")
    subprocess.run([cc, "-std=c11", "-O1", "-g", "-Wall", "-Wextra", "-Werror", *CHECKS,
                    "-I", INCLUDE, DRIVER, "-o", exe, "-L", str(tmp_path), "-llayers_asan",
                    "-Wl,-rpath," + str(tmp_path), "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
                    "-Wl,-rpath," + os.path.join(ROCM, "lib")],
                   check=True, capture_output=True, timeout=300)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    out = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    assert out.returncode == 0, out.stdout + out.stderr
    assert "host checks: 0 failures" in out.stdout
    assert "runtime error" not in out.stderr and "AddressSanitizer" not in out.stderr
