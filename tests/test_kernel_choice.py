"""Which kernel the grouped fp32 products and the 8-bit products take, without a
GPU: the calls that the GPU tests make reach every one, whatever the rules
become."""
import os
import re

import pytest

import kernel_cases as kc
from conftest import ROOT

CUS = 256


@pytest.fixture(scope="module")
def pg():
    import precision_gemm_amd as pg
    if not os.path.exists(pg.library_path()):
        from precision_gemm_amd import _build
        _build.build()
    pg._load()
    return pg


@pytest.mark.parametrize("case", kc.GROUPED + [kc.GROUPED_V1], ids=kc.name)
def test_grouped(pg, case):
    assert kc.grouped_choice(pg, case, CUS) == case.kernel


@pytest.mark.parametrize("case", kc.OUTER + [kc.OUTER_V1], ids=kc.name)
def test_outer(pg, case):
    assert kc.outer_choice(pg, case, CUS) == case.kernel


@pytest.mark.parametrize("case", kc.I8_CASES, ids=kc.name)
def test_i8(pg, case):
    assert kc.i8_choice(pg, case, CUS) == case.kernel


def test_every_kernel_is_reached(pg):
    """Each with both transposes and, of the streams, aligned and not."""
    reached = {(c.kernel, c.tB) for c in kc.GROUPED + [kc.GROUPED_V1]}
    assert reached == {(k, tB) for k in pg.GROUPED_KERNELS for tB in (0, 1)} - {("T64x64_V1", 1)}
    assert {c.kernel for c in kc.OUTER + [kc.OUTER_V1]} == set(pg.GROUPED_OUTER_KERNELS)
    reached = {(c.kernel, kc.i8_aligned(c)) for c in kc.I8_CASES}
    for k in pg.I8GEMM_KERNELS:
        assert (k, True) in reached, k
        assert k[0] == "L" or (k, False) in reached, k
    # groups and single products alike where both take a kernel
    for k in ("S16x32", "T64x64", "T128x128", "L256x256"):
        assert {c.counts is None for c in kc.I8_CASES if c.kernel == k} == {True, False}


def test_numbers(pg):
    text = open(os.path.join(ROOT, "include", "sgemm.h")).read()
    for prefix, names in (("SGEMM_GROUPED_", pg.GROUPED_KERNELS),
                          ("SGEMM_GROUPED_OUTER_", pg.GROUPED_OUTER_KERNELS)):
        numbers = dict(re.findall(r"%s((?!OUTER_)\w+) = (\d+)" % prefix, text))
        assert int(numbers.pop("COUNT")) == len(names)
        assert {n: int(v) for n, v in numbers.items()} == {n: i for i, n in enumerate(names)}


def test_invalid_sizes(pg):
    forward, outer = pg.sgemm_grouped_select_kernel, pg.sgemm_grouped_outer_select_kernel
    assert [forward(*a, 1, CUS) for a in ((2, 1, 1, 1), (0, -1, 1, 1), (0, 1, -1, 1),
                                          (0, 1, 1, -1), (0, 1, 1, 65537))] == \
        [-801, -802, -803, -805, -805]
    assert [outer(*a, 1, CUS) for a in ((-1, 1, 1), (1, -1, 1), (1, 1, -1))] == [-901, -902, -904]
    big = 2**31 - 1
    assert forward(0, big, 2**21 - 1, 1, 0, CUS) == -22 and outer(4096, 4096, big, 1, CUS) == -22
    assert forward(0, 0, 0, 0, 0, 0) >= 0 and outer(0, 0, 0, 0, 0) >= 0
