"""What expert_layer launches for its largest sizes, seen through stand-ins for the
runtime's calls (tests/cabi/hip_stub.c), without a GPU: every launch holds fewer
than 2^32 work-items, or the call is refused."""
import json
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT

STUB = os.path.join(ROOT, "tests", "cabi", "hip_stub.c")
RUN = r"""
import ctypes, json, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
i, p, ll, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_size_t
lib.expert_layer.argtypes = [i, i, i, i, i, p, i, i, p, i, p, p, i, i, ll, p, p, i, ll, p, p, i, p,
                             sz, p]
launches = ctypes.c_int.in_dll(stub, "stub_launches")
items = ctypes.c_uint64.in_dll(stub, "stub_most_items")
FAKE = 1 << 20  # never dereferenced
out = []
for tokens, topk, experts, H, F, type_, w_type, ldw1, ldw2 in json.loads(sys.argv[3]):
    launches.value = items.value = 0
    status = lib.expert_layer(tokens, topk, experts, H, F, FAKE, type_, H, FAKE, 4, None, FAKE,
                              w_type, ldw1, 0, FAKE, FAKE, ldw2, 0, FAKE, FAKE, H, FAKE,
                              1 << 62, None)
    out.append([status, launches.value, items.value])
print(json.dumps(out))
"""


def launches(cases, tmp_path):
    cc = shutil.which("cc") or shutil.which("gcc") or shutil.which("clang")
    if cc is None:
        pytest.skip("no C compiler")
    so = str(tmp_path / "hip_stub.so")
    subprocess.run([cc, "-std=c11", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", STUB,
                    "-o", so], check=True, timeout=120)
    import precision_gemm_amd as pg
    out = subprocess.run([sys.executable, "-c", RUN, so, pg.library_path(), json.dumps(cases)],
                         check=True, capture_output=True, text=True, timeout=300).stdout
    return json.loads(out)


# (tokens, topk, experts, H, F, type, w_type, ldw1, ldw2): F32 0, F16 1, BF16 2, I8 3, MX4 4
SMALL = (1, 2, 4, 64, 48, 2, 2, 64, 48)
EVEN = [(256, 8, 1024, H, 1 << 20, type_, w_type, ldw1, ldw2)
        for H, type_, w_type, ldw1, ldw2 in
        [(1024, 2, 2, 1024, 1 << 20), (1024, 2, 2, 2048, 1 << 20), (512, 0, 0, 512, 1 << 20),
         (2048, 1, 3, 2048, 1 << 20), (4096, 2, 4, 2048, 1 << 19), (64, 2, 2, 1 << 20, 1 << 20)]]
RAGGED = (256, 8, 1024, 1024, 1 << 20, 2, 2, 1025, 1 << 20)


def test_the_stand_ins_see_the_launches(tmp_path):
    (status, n, items), = launches([SMALL], tmp_path)
    assert (status, n) in ((0, 2), (0, 3)) and 0 < items < 1 << 20


def test_largest_layers_fit_a_launch(tmp_path):
    """2048 slots over 1024 experts of 2^20 inner values: even rows, whatever the
    distance between W1's, run in tiles of which a launch holds enough; others do
    not fit and are refused before the device is asked."""
    for case, (status, n, items) in zip(EVEN, launches(EVEN, tmp_path)):
        assert status == 0 and n == 3 and items < 1 << 32, (case, status, n, items)
    assert launches([RAGGED], tmp_path) == [[-22, 0, 0]]
