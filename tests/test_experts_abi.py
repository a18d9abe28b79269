"""The expert and 8-bit calls on the host: exported symbols, argument checks,
quick returns and messages, and what the binding refuses. Nothing here launches
a kernel, so it runs without a GPU."""
import os
import re
import subprocess
import sys

import pytest

from conftest import ROOT

FAKE = 1 << 20  # never dereferenced: every call below returns before any device work
CALLS = {
    "i8_quantize_rows": (100, dict(M=4, K=4, X=FAKE, x_type=0, ldx=4, Q=FAKE, ldq=4, scale=FAKE)),
    "i8gemm": (200, dict(M=4, N=4, K=4, A=FAKE, lda=4, scaleA=FAKE, B=FAKE, ldb=4, scaleB=FAKE,
                         bias=None, C=FAKE, c_type=0, ldc=4)),
    "i8gemm_grouped": (300, dict(M=4, N=4, K=4, groups=2, offsets=FAKE, A=FAKE, lda=4,
                                 scaleA=FAKE, B=FAKE, ldb=4, strideB=16, scaleB=FAKE, bias=None,
                                 C=FAKE, c_type=0, ldc=4)),
    "expert_sort": (400, dict(tokens=4, topk=2, experts=8, ids=FAKE, id_bytes=4, offsets=FAKE,
                              row_of_slot=FAKE, workspace=None, workspace_bytes=0)),
    "expert_gather": (500, dict(tokens=4, topk=2, cols=4, X=FAKE, type=0, ldx=4,
                                row_of_slot=FAKE, Y=FAKE, ldy=4)),
    "expert_combine": (600, dict(tokens=4, topk=2, cols=4, Y=FAKE, type=0, ldy=4,
                                 row_of_slot=FAKE, weights=None, out=FAKE, ldo=4)),
    "expert_combine_grad": (700, dict(tokens=4, topk=2, cols=4, dout=FAKE, type=0, ldo=4, Y=FAKE,
                                      ldy=4, row_of_slot=FAKE, weights=FAKE, dY=FAKE, lddy=4,
                                      dweights=FAKE)),
    "sgemm_grouped": (800, dict(transB=0, M=4, N=4, K=4, groups=2, offsets=FAKE, alpha=1.0,
                                A=FAKE, lda=4, B=FAKE, ldb=4, strideB=16, beta=0.0, C=FAKE,
                                ldc=4)),
    "sgemm_grouped_outer": (900, dict(M=4, N=4, K=4, groups=2, offsets=FAKE, alpha=1.0, A=FAKE,
                                      lda=4, B=FAKE, ldb=4, beta=0.0, C=FAKE, ldc=4,
                                      strideC=16)),
}


@pytest.fixture(scope="module")
def pg():
    import precision_gemm_amd as pg
    if not os.path.exists(pg.library_path()):
        from precision_gemm_amd import _build
        _build.build()
    pg._load()
    return pg


def call(pg, name, **over):
    args = dict(CALLS[name][1])
    assert set(over) <= set(args), over
    args.update(over)
    return getattr(pg._load(), name)(*args.values(), None)


def position(name, arg):
    return list(CALLS[name][1]).index(arg) + 1


@pytest.mark.parametrize("header,prefix", [("i8gemm.h", "i8"), ("experts.h", "expert")])
def test_headers(pg, header, prefix):
    """The headers compile as C, and the library exports what they declare."""
    path = os.path.join(ROOT, "include", header)
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(%s\w*)\s*\(" % prefix, text, re.M))
    assert names >= {n for n in CALLS if n.startswith(prefix)}
    for n in names:
        assert hasattr(pg._load(), n)
    subprocess.run(["gcc", "-x", "c", "-std=c99", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "include"), "-fsyntax-only", "-"],
                   input='#include "%s"\nint main(void){return 0;}\n' % header, text=True,
                   check=True)


REFUSED = [
    ("i8_quantize_rows", [("M", -1), ("K", -1), ("K", 2**31 - 1), ("X", None), ("x_type", 3),
                          ("x_type", -1), ("ldx", 3), ("Q", None), ("ldq", 3), ("scale", None)]),
    ("i8gemm", [("M", -1), ("N", -1), ("K", -1), ("K", 131072), ("A", None), ("lda", 3),
                ("scaleA", None), ("B", None), ("ldb", 3), ("scaleB", None), ("C", None),
                ("c_type", 3), ("ldc", 3)]),
    ("i8gemm_grouped", [("M", -1), ("N", -1), ("K", -1), ("K", 131072), ("groups", -1),
                        ("offsets", None), ("A", None), ("lda", 3), ("scaleA", None),
                        ("B", None), ("ldb", 3), ("strideB", -1), ("scaleB", None), ("C", None),
                        ("c_type", 4), ("ldc", 3)]),
    ("expert_sort", [("tokens", -1), ("tokens", 2**30), ("topk", 0), ("experts", 0),
                     ("experts", 1025), ("ids", None), ("id_bytes", 2), ("offsets", None),
                     ("row_of_slot", None)]),
    ("expert_gather", [("tokens", -1), ("tokens", 2**30), ("topk", 0), ("cols", -1), ("X", None),
                       ("type", 4), ("ldx", 3), ("row_of_slot", None), ("Y", None), ("ldy", 3)]),
    ("expert_combine", [("tokens", -1), ("tokens", 2**30), ("topk", 0), ("cols", -1), ("Y", None),
                        ("type", 3), ("ldy", 3), ("row_of_slot", None), ("out", None),
                        ("ldo", 3)]),
    ("expert_combine_grad", [("tokens", -1), ("tokens", 2**30), ("topk", 0), ("cols", -1),
                             ("dout", None), ("type", 3), ("ldo", 3), ("Y", None), ("ldy", 3),
                             ("row_of_slot", None), ("dY", None), ("lddy", 3)]),
    ("sgemm_grouped", [("transB", 2), ("M", -1), ("N", -1), ("K", -1), ("groups", -1),
                       ("offsets", None), ("A", None), ("lda", 3), ("lda", 1 << 21), ("B", None),
                       ("ldb", 3), ("ldb", 1 << 21), ("strideB", -1), ("C", None), ("ldc", 3),
                       ("ldc", 1 << 21)]),
    ("sgemm_grouped_outer", [("M", -1), ("N", -1), ("K", -1), ("groups", -1), ("offsets", None),
                             ("A", None), ("lda", 3), ("lda", 1 << 21), ("B", None), ("ldb", 3),
                             ("ldb", 1 << 21), ("C", None), ("ldc", 3), ("ldc", 1 << 21),
                             ("strideC", -1)]),
]


@pytest.mark.parametrize("name,arg,value", [(n, a, v) for n, av in REFUSED for a, v in av])
def test_argument_errors(pg, name, arg, value):
    """Each bad argument gives minus (the call's base + its position), with a
    message naming the call."""
    status = call(pg, name, **{arg: value})
    assert status == -(CALLS[name][0] + position(name, arg))
    text = pg.sgemm_status_string(status)
    assert text.startswith(name + ":") and str(position(name, arg)) in text


@pytest.mark.parametrize("name,over", [
    ("i8_quantize_rows", dict(M=0, X=None, Q=None, scale=None)),
    ("i8gemm", dict(M=0, A=None, C=None)), ("i8gemm", dict(N=0, B=None, C=None)),
    ("i8gemm_grouped", dict(groups=0, offsets=None)), ("i8gemm_grouped", dict(M=0, A=None)),
    ("expert_gather", dict(tokens=0, X=None, row_of_slot=None)),
    ("expert_gather", dict(cols=0, X=None, Y=None)),
    ("expert_combine", dict(tokens=0)), ("expert_combine", dict(cols=0, Y=None)),
    ("expert_combine_grad", dict(tokens=0)),
    ("expert_combine_grad", dict(cols=0, dweights=None, dY=None)),
    ("sgemm_grouped", dict(M=0)), ("sgemm_grouped", dict(groups=0, offsets=None)),
    ("sgemm_grouped", dict(K=0, beta=1.0, A=None, B=None)),
    ("sgemm_grouped", dict(alpha=0.0, beta=1.0)),
    ("sgemm_grouped_outer", dict(N=0)), ("sgemm_grouped_outer", dict(K=0, beta=1.0, A=None)),
])
def test_quick_returns_launch_nothing(pg, name, over):
    assert call(pg, name, **over) == 0


def test_sort_workspace(pg):
    size = pg.expert_sort_workspace_size
    assert size(4, 2, 8) == 0  # a single run needs none
    need = size(1 << 16, 8, 128)
    assert 0 < need <= 256 * 129 * 4
    big = size((1 << 28) - 1, 8, 1024)
    assert 0 < big <= 256 * 1025 * 4
    for bad in ((-1, 2, 8), (4, 0, 8), (4, 2, 0), (4, 2, 1025), (1 << 30, 2, 8)):
        assert size(*bad) == 0
    over = dict(tokens=1 << 16, topk=8, experts=128)
    assert call(pg, "expert_sort", **over, workspace=None, workspace_bytes=need) == -408
    assert call(pg, "expert_sort", **over, workspace=FAKE + 2, workspace_bytes=need) == -408
    assert call(pg, "expert_sort", **over, workspace=FAKE, workspace_bytes=need - 1) == -409


def test_oversize_grids_are_rejected(pg):
    """More output tiles than a launch holds: -22 before any device work."""
    n = 2**31 - 1
    assert call(pg, "i8gemm", M=n, N=n, ldc=n) == -22
    assert call(pg, "sgemm_grouped", M=n, N=(1 << 21) - 1, ldb=(1 << 21) - 1,
                ldc=(1 << 21) - 1) == -22
    assert call(pg, "sgemm_grouped_outer", groups=n, M=4096, N=4096, lda=4096, ldb=4096,
                ldc=4096) == -22


def test_too_many_groups_are_rejected(pg):
    for name, code in (("i8gemm_grouped", -304), ("sgemm_grouped", -805)):
        assert call(pg, name, groups=65537) == code
        assert call(pg, name, groups=2**31 - 1) == code
        assert "65536" in pg.sgemm_status_string(code)


def test_binding_refuses_host_tensors(pg):
    torch = pytest.importorskip("torch")
    x, q, s = torch.zeros(4, 4), torch.zeros(4, 4, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(TypeError, match="X must be a GPU tensor"):
        pg.i8_quantize_rows(4, 4, x, 4, q, 4, s)
    with pytest.raises(TypeError, match="A must be a GPU tensor"):
        pg.i8gemm(4, 4, 4, q, 4, s, q, 4, s, None, x, 4)
    with pytest.raises(TypeError, match="ids must be a GPU tensor"):
        pg.expert_sort(4, 1, 4, s, s, s, None)
    with pytest.raises(TypeError, match="offsets must be a GPU tensor"):
        pg.sgemm_grouped(0, 4, 4, 4, 1, s, 1.0, x, 4, x, 4, 16, 0.0, x, 4)


def test_binding_refuses_sizes_beyond_an_int(pg):
    """2^32 + 4 would reach the library as 4."""
    torch = pytest.importorskip("torch")
    from precision_gemm_amd import _experts
    for rows, cols, ld in ((2**32 + 4, 4, 4), (4, 2**31, 2**31), (4, 4, 2**31)):
        with pytest.raises(ValueError, match="below 2"):
            _experts._span(rows, cols, ld)
        with pytest.raises(ValueError, match="below 2"):
            _experts._spans(2, 16, rows, cols, ld)
    assert _experts._span(3, 4, 5) == 14 and _experts._span(0, 4, 5) == 0
    assert _experts._spans(2, 100, 3, 4, 5) == 114 and torch is not None


@pytest.fixture()
def on_host(pg, monkeypatch):
    """Host tensors that count as device 0's, for what the binding refuses, and
    calls that end before the library's."""
    torch = pytest.importorskip("torch")
    from precision_gemm_amd import _experts

    class OnDevice(torch.Tensor):
        is_cuda = property(lambda self: True)
        get_device = lambda self: 0  # noqa: E731

    monkeypatch.setattr(_experts, "_call", lambda fn, device, stream, check, *args: args)
    return torch, lambda *shape, dtype=torch.float32: \
        torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def test_binding_refuses_vectors_with_gaps(pg, on_host):
    """A part of a wider router's output, say: ids[:, :2] of [T, 4]. Taken as it
    lies, its elements would be those of other slots."""
    torch, make = on_host
    T, k, E, H, N = 6, 2, 4, 8, 4
    i32 = torch.int32
    x, y, q = make(T * k, H), make(T * k, H), make(T * k, H, dtype=torch.int8)
    vectors = dict(ids=make(T, 2 * k, dtype=i32), offsets=make(2 * E + 2, dtype=i32),
                   row_of_slot=make(T, 2 * k, dtype=i32), weights=make(T, 2 * k),
                   dweights=make(T, 2 * k), scale=make(2 * T), scaleA=make(2 * T),
                   scaleB=make(E, 2 * N), bias=make(E, 2 * N))
    gaps = {n: v[::2] if v.dim() == 1 else v[:, :v.shape[1] // 2] for n, v in vectors.items()}
    whole = {n: v.contiguous() for n, v in gaps.items()}
    calls = [
        (lambda v: pg.i8_quantize_rows(T, H, x, H, q, H, v["scale"]), ["scale"]),
        (lambda v: pg.i8gemm(T, N, H, q, H, v["scaleA"], q, H, v["scaleB"][:1], v["bias"][:1], x,
                             H),
         ["scaleA"]),
        (lambda v: pg.i8gemm_grouped(T, N, H, E, v["offsets"], q, H, v["scaleA"], q, H, 0,
                                     v["scaleB"], v["bias"], x, H),
         ["offsets", "scaleA", "scaleB", "bias"]),
        (lambda v: pg.expert_sort(T, k, E, v["ids"], v["offsets"], v["row_of_slot"], None),
         ["ids", "offsets", "row_of_slot"]),
        (lambda v: pg.expert_gather(T, k, H, x, H, v["row_of_slot"], y, H), ["row_of_slot"]),
        (lambda v: pg.expert_combine(T, k, H, y, H, v["row_of_slot"], v["weights"], x, H),
         ["row_of_slot", "weights"]),
        (lambda v: pg.expert_combine_grad(T, k, H, x, H, y, H, v["row_of_slot"], v["weights"], y, H,
                                          v["dweights"]), ["row_of_slot", "weights", "dweights"]),
        (lambda v: pg.sgemm_grouped(0, T, H, H, E, v["offsets"], 1.0, x, H, y, H, 0, 0.0, x, H),
         ["offsets"]),
        (lambda v: pg.sgemm_grouped_outer(H, 1, T, E, v["offsets"], 1.0, x, H, x, H, 0.0, y, 1, 8),
         ["offsets"]),
    ]
    for call_with, names in calls:
        call_with(whole)  # taken
        for name in names:
            with pytest.raises(ValueError, match="^%s must be contiguous" % name):
                call_with({**whole, name: gaps[name]})


def test_binding_refuses_sizes_below_an_int(pg, on_host):
    """-2^32 + 4 would reach the library as 4, past the check of the tensors'
    extents, which a negative size needs nothing of. (Negative ints are the
    library's to refuse.)"""
    torch, make = on_host
    n, big = 4 - 2**32, 4 - 2**64
    x, q, s = make(2), make(2, dtype=torch.int8), make(1)
    i = make(1, dtype=torch.int32)
    for bad in (
            lambda: pg.i8_quantize_rows(n, 4, x, 4, q, 4, s),
            lambda: pg.i8_quantize_rows(4, n, x, 4, q, 4, make(4)),
            lambda: pg.i8gemm(n, 1, 2, q, 2, s, q, 2, s, None, x, 1),
            lambda: pg.i8gemm(1, n, 2, q, 2, s, q, 2, s, None, x, 1),
            lambda: pg.i8gemm(2, 1, 1, q, n, make(2), q, 1, s, None, x, 1),
            lambda: pg.i8gemm_grouped(1, 1, 2, n, i, q, 2, s, q, 2, 2, s, None, x, 1),
            lambda: pg.i8gemm_grouped(1, 1, 2, 2, make(3, dtype=torch.int32), q, 2, s, q, 2, big,
                                      make(2), None, x, 1),
            lambda: pg.expert_sort(n, 1, 4, i, make(5, dtype=torch.int32), i, None),
            lambda: pg.expert_sort(1, n, 4, i, make(5, dtype=torch.int32), i, None),
            lambda: pg.expert_sort(1, 1, n, i, i, i, None),
            lambda: pg.expert_gather(1, n, 2, x, 2, i, x, 2),
            lambda: pg.expert_combine(1, n, 2, x, 2, i, None, x, 2),
            lambda: pg.expert_combine_grad(1, n, 2, x, 2, x, 2, i, None, x, 2, s),
            lambda: pg.sgemm_grouped(0, 1, 1, 1, n, i, 1.0, x, 1, x, 1, 1, 0.0, x, 1),
            lambda: pg.sgemm_grouped_outer(1, 1, 1, n, i, 1.0, x, 1, x, 1, 0.0, x, 1, 1),
            lambda: pg.sgemm_grouped_outer(1, 1, 1, 2, make(3, dtype=torch.int32), 1.0, x, 1, x, 1,
                                           0.0, x, 1, big)):
        with pytest.raises(ValueError, match="below 2"):
            bad()
    assert pg.i8gemm(-1, 1, 2, q, 2, s, q, 2, s, None, x, 1)[0] == -1


def test_without_torch(pg):
    """Every public name is there without torch, as those of the fp32 calls
    were before; the calls that take tensors say what they miss."""
    code = """
import sys
sys.modules["torch"] = None  # imports of it fail
from precision_gemm_amd import *
import precision_gemm_amd as pg
assert all(hasattr(pg, n) for n in pg.__all__)
assert I8GEMM_MAX_K == 131071 and expert_sort_workspace_size(65536, 8, 128) > 0
assert sgemm_select_variant(0, 0, 64, 64, 64, 1, 1, 256) >= 0
try:
    i8gemm(1, 1, 1, None, 1, None, None, 1, None, None, None, 1)
except ImportError as e:
    assert "torch" in str(e)
else:
    raise SystemExit("taken")
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr


def test_binding_refuses_other_workspaces(pg, on_host):
    torch, make = on_host
    i = make(8, dtype=torch.int32)
    for ws in (1 << 20, b"0" * 4096, torch.zeros(4096)):
        with pytest.raises(TypeError, match="workspace must be a GPU tensor"):
            pg.expert_sort(4, 2, 4, i, i, i, ws)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        pg.expert_sort(4, 2, 4, i, i, i, make(64, 2)[:, 0])
    assert pg.expert_sort(4, 2, 4, i, i, i, make(64))[-1] == 256


I8_THREADS = dict(S16x16=512, S16x16_W16=1024, S16x32=256, S32x16=512, S32x32=512, S32x64=256,
                  L32x64=128, L128x128=512, L128x256=512, L256x256=512)  # others 256


def i8_work_items(name, M, N, groups):
    """Work-items of a call's launch: every group may have a partly filled row tile."""
    bm, bn = map(int, re.match(r"[STL](\d+)x(\d+)", name).groups())
    rows = M // bm + min(groups, M) if groups else -(-M // bm)
    return rows * -(-N // bn) * I8_THREADS.get(name, 256)


def test_i8_kernel_numbers(pg):
    text = open(os.path.join(ROOT, "include", "i8gemm.h")).read()
    numbers = dict(re.findall(r"I8GEMM_KERNEL_(\w+) = (\d+)", text))
    assert int(numbers.pop("COUNT")) == len(pg.I8GEMM_KERNELS)
    assert {n: int(v) for n, v in numbers.items()} == \
        {n: i for i, n in enumerate(pg.I8GEMM_KERNELS)}


def test_i8_kernels_whose_tiles_fit_a_launch(pg):
    """A kernel whose tiles a launch does not hold is passed over for one whose
    tiles it does."""
    import random
    rng = random.Random(7)
    size = lambda most: int(2 ** rng.uniform(0, most))  # noqa: E731
    calls = [(524288, 8192, 4096, 65536, 1), (8192, 350000, 16, 1024, 1), (2**30, 1, 16, 0, 1),
             (1, 2**29, 64, 0, 1), (4, 2**30, 64, 0, 1), (16, 2**30, 64, 0, 0)]
    calls += [(size(31), size(31), rng.choice([1, 16, 100, 4096]), rng.choice([0, 0, size(16)]),
               rng.randrange(2)) for _ in range(20000)]
    refused = 0
    for M, N, K, groups, aligned in calls:
        kernel = pg.i8gemm_select_kernel(M, N, K, groups, aligned, 256)
        if kernel >= 0:
            name = pg.I8GEMM_KERNELS[kernel]
            assert i8_work_items(name, M, N, groups) < 2**32, (M, N, K, groups, aligned, name)
            assert name[0] != "L" or (aligned and K % 16 == 0)
            continue
        refused += 1
        assert kernel == -22
        largest = "L256x256" if aligned and K % 16 == 0 else "T128x128"
        assert i8_work_items(largest, M, N, groups) >= 2**32, (M, N, K, groups, aligned)
    assert 0 < refused < 20000
    assert pg.i8gemm_select_kernel(524288, 8192, 4096, 65536, 1, 256) >= 0
    for bad, status in (((-1, 1, 1, 0), -201), ((1, -1, 1, 0), -202), ((1, 1, 131072, 0), -203),
                        ((1, 1, 1, 65537), -304)):
        assert pg.i8gemm_select_kernel(*bad, 1, 256) == status
    assert pg.i8gemm_select_kernel(0, 0, 0, 0, 0, 0) >= 0
