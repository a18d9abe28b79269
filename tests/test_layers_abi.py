"""The norms, the 4-bit calls and the experts' layer on the host: exported
symbols, argument checks, quick returns, messages and what the binding refuses.
Nothing here launches a kernel, so it runs without a GPU."""
import os
import re
import subprocess
import sys

import pytest

from conftest import ROOT

FAKE = 1 << 20  # never dereferenced: every call below returns before any device work
NORM = dict(M=4, K=4, X=FAKE, type=0, ldx=4, R=FAKE, ldr=4, weight=FAKE, eps=1e-6, H=FAKE, ldh=4)
CALLS = {
    "rms_norm": (1000, dict(**NORM, Y=FAKE, ldy=4)),
    "rms_norm_i8": (1100, dict(**NORM, Q=FAKE, ldq=4, scale=FAKE)),
    "rms_norm_grad": (1200, dict(M=4, K=4, dY=FAKE, type=0, lddy=4, H=FAKE, ldh=4, weight=FAKE,
                                 eps=1e-6, dH=FAKE, lddh=4, dX=FAKE, lddx=4, dweight=FAKE,
                                 workspace=FAKE, workspace_bytes=1 << 20)),
    "mx4_quantize_rows": (1300, dict(M=4, K=8, X=FAKE, x_type=0, ldx=8, Q=FAKE, ldq=4, scale=FAKE,
                                     lds=4)),
    "mx4_dequantize_rows": (1400, dict(M=4, K=8, Q=FAKE, ldq=4, scale=FAKE, lds=4, Y=FAKE,
                                       y_type=0, ldy=8)),
    "mx4gemm": (1500, dict(M=4, N=6, K=8, A=FAKE, lda=4, scaleA=FAKE, ldsa=4, B=FAKE, ldb=4,
                           scaleB=FAKE, ldsb=6, bias=None, C=FAKE, c_type=0, ldc=6)),
    "mx4gemm_grouped": (1600, dict(M=4, N=6, K=8, groups=2, offsets=FAKE, A=FAKE, lda=4,
                                   scaleA=FAKE, ldsa=4, B=FAKE, ldb=4, strideB=24, scaleB=FAKE,
                                   ldsb=6, strideSB=24, bias=None, C=FAKE, c_type=0, ldc=6)),
    "expert_layer": (1700, dict(tokens=4, topk=2, experts=8, H=8, F=6, X=FAKE, type=2, ldx=8,
                                ids=FAKE, id_bytes=4, weights=None, W1=FAKE, w_type=3, ldw1=8,
                                strideW1=96, scale1=FAKE, W2=FAKE, ldw2=6, strideW2=48,
                                scale2=FAKE, out=FAKE, ldo=8, workspace=FAKE,
                                workspace_bytes=1 << 20)),
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


@pytest.mark.parametrize("header,prefix", [("norm.h", "rms"), ("mx4gemm.h", "mx4"),
                                           ("experts.h", "expert_layer")])
def test_headers(pg, header, prefix):
    """The headers compile as C, and the library exports what they declare."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(%s\w*)\s*\(" % prefix, text, re.M))
    assert names >= {n for n in CALLS if n.startswith(prefix)}
    for n in names:
        assert hasattr(pg._load(), n)
    subprocess.run(["gcc", "-x", "c", "-std=c99", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "include"), "-fsyntax-only", "-"],
                   input='#include "%s"\nint main(void){return 0;}\n' % header, text=True,
                   check=True)


def test_constants(pg):
    text = "".join(open(os.path.join(ROOT, "include", h)).read() for h in ("norm.h", "experts.h"))
    for name in ("RMS_NORM_GRAD_MAX_K", "EXPERT_LAYER_MAX_SLOTS", "EXPERT_LAYER_MAX_EXPERTS"):
        assert int(re.search(r"#define %s (\d+)" % name, text).group(1)) == getattr(pg, name)


NORM_BAD = [("M", -1), ("K", -1), ("K", 2**31 - 1), ("X", None), ("type", 3), ("type", -1),
            ("ldx", 3), ("ldr", 3), ("weight", None), ("eps", -1e-6), ("eps", float("nan")),
            ("ldh", 3)]
REFUSED = [
    ("rms_norm", NORM_BAD + [("Y", None), ("ldy", 3)]),
    ("rms_norm_i8", NORM_BAD + [("Q", None), ("ldq", 3), ("scale", None)]),
    ("rms_norm_grad", [("M", -1), ("K", -1), ("K", 16385), ("dY", None), ("type", 3), ("lddy", 3),
                       ("H", None), ("ldh", 3), ("weight", None), ("eps", -1.0),
                       ("eps", float("nan")), ("lddh", 3), ("dX", None), ("lddx", 3),
                       ("workspace", None), ("workspace", FAKE + 8), ("workspace_bytes", 15)]),
    ("mx4_quantize_rows", [("M", -1), ("K", -1), ("K", 2**31 - 1), ("X", None), ("x_type", 3),
                           ("ldx", 7), ("Q", None), ("ldq", 3), ("scale", None),
                           ("scale", FAKE + 2), ("lds", 3)]),
    ("mx4_dequantize_rows", [("M", -1), ("K", -1), ("Q", None), ("ldq", 3), ("scale", None),
                             ("scale", FAKE + 1), ("lds", 3), ("Y", None), ("y_type", 4),
                             ("ldy", 7)]),
    ("mx4gemm", [("M", -1), ("N", -1), ("K", -1), ("K", 2**31 - 1), ("A", None), ("lda", 3),
                 ("scaleA", None), ("scaleA", FAKE + 2), ("ldsa", 3), ("B", None), ("ldb", 3),
                 ("scaleB", None), ("scaleB", FAKE + 3), ("ldsb", 5), ("C", None), ("c_type", 3),
                 ("ldc", 5)]),
    ("mx4gemm_grouped", [("M", -1), ("N", -1), ("K", -1), ("groups", -1), ("groups", 65537),
                         ("offsets", None), ("A", None), ("lda", 3), ("scaleA", None),
                         ("scaleA", FAKE + 2), ("ldsa", 3), ("B", None), ("ldb", 3),
                         ("strideB", -1), ("scaleB", None), ("scaleB", FAKE + 3), ("ldsb", 5),
                         ("strideSB", -4), ("strideSB", 2), ("C", None), ("c_type", 3),
                         ("ldc", 5)]),
    ("expert_layer", [("tokens", -1), ("tokens", 1025), ("topk", 0), ("experts", 0),
                      ("experts", 1025), ("H", -1), ("H", 2**20 + 1), ("F", -1), ("F", 2**20 + 1),
                      ("X", None), ("type", 3), ("ldx", 7), ("ids", None), ("id_bytes", 2),
                      ("W1", None), ("w_type", 0), ("w_type", 5), ("w_type", -1), ("ldw1", 7),
                      ("strideW1", -1), ("scale1", None), ("scale1", FAKE + 2), ("W2", None),
                      ("ldw2", 5), ("strideW2", -1), ("scale2", None), ("scale2", FAKE + 1),
                      ("out", None), ("ldo", 7), ("workspace", None), ("workspace", FAKE + 8),
                      ("workspace_bytes", 100)]),
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
    ("rms_norm", dict(M=0, X=None, Y=None)), ("rms_norm", dict(K=0, X=None, weight=None, Y=None)),
    ("rms_norm_i8", dict(M=0, scale=None)),
    ("rms_norm_grad", dict(K=0, dY=None, H=None, dX=None)),
    ("rms_norm_grad", dict(M=0, dweight=None, workspace=None, workspace_bytes=0)),
    ("mx4_quantize_rows", dict(M=0, X=None, scale=None)),
    ("mx4_quantize_rows", dict(K=0, X=None, scale=None)),
    ("mx4_dequantize_rows", dict(M=0, Q=None)), ("mx4_dequantize_rows", dict(K=0, Y=None)),
    ("mx4gemm", dict(M=0, A=None, C=None)), ("mx4gemm", dict(N=0, B=None, C=None)),
    ("mx4gemm_grouped", dict(groups=0, offsets=None)), ("mx4gemm_grouped", dict(M=0, A=None)),
    ("expert_layer", dict(tokens=0, X=None, ids=None, workspace=None)),
    ("expert_layer", dict(H=0, X=None, out=None)),
])
def test_quick_returns_launch_nothing(pg, name, over):
    assert call(pg, name, **over) == 0


def test_parts_that_are_not_there(pg):
    """The leading dimension of an absent operand is not looked at; that of one
    that is there is."""
    for name in ("rms_norm", "rms_norm_i8"):
        assert call(pg, name, M=0, R=None, ldr=0, H=None, ldh=0) == 0
    assert call(pg, "rms_norm_grad", M=0, dH=None, lddh=0, dweight=None) == 0
    # weights of X's type have no scales
    assert call(pg, "expert_layer", w_type=2, scale1=None, scale2=None, workspace=None) == -1723


def test_oversize_grids_are_rejected(pg):
    """More output tiles than a launch holds: -22 before any device work."""
    n = 2**31 - 1
    assert call(pg, "mx4gemm", M=n, N=n, ldsa=n, ldsb=n, ldc=n) == -22
    assert call(pg, "mx4gemm_grouped", groups=65536, M=n, N=n, ldsa=n, ldsb=n, ldc=n) == -22
    size = pg._load().expert_layer_workspace_size(256, 8, 1 << 20, 1 << 20, 2)
    assert call(pg, "expert_layer", tokens=256, topk=8, experts=1024, H=1 << 20, F=1 << 20,
                ldx=1 << 20, ldw1=(1 << 20) + 1, ldw2=1 << 20, ldo=1 << 20,
                workspace_bytes=size) == -22


MX4_THREADS = dict(S16x16=512, S32x16=512, S32x32=512, L128x128=512, L128x128_R2=512,
                   L128x256=512, L256x256=512)  # others 256


def mx4_work_items(name, M, N, groups):
    """Work-items of a call's launch: every group may have a partly filled row tile."""
    bm, bn = map(int, re.match(r"[STL](\d+)x(\d+)", name).groups())
    rows = M // bm + min(groups, M) if groups else -(-M // bm)
    return rows * -(-N // bn) * MX4_THREADS.get(name, 256)


def test_mx4_kernel_numbers(pg):
    text = open(os.path.join(ROOT, "include", "mx4gemm.h")).read()
    numbers = dict(re.findall(r"MX4GEMM_KERNEL_(\w+) = (\d+)", text))
    assert int(numbers.pop("COUNT")) == len(pg.MX4GEMM_KERNELS)
    assert {n: int(v) for n, v in numbers.items()} == \
        {n: i for i, n in enumerate(pg.MX4GEMM_KERNELS)}


def test_mx4_kernels_whose_tiles_fit_a_launch(pg):
    """A kernel whose tiles a launch does not hold is passed over for one whose
    tiles it does; every kernel is some call's."""
    import random
    rng = random.Random(7)
    size = lambda most: int(2 ** rng.uniform(0, most))  # noqa: E731
    calls = [(524288, 8192, 4096, 65536, 1), (8192, 350000, 32, 1024, 1), (2**30, 1, 32, 0, 1),
             (1, 2**29, 64, 0, 1), (4, 2**30, 64, 0, 1), (16, 2**30, 64, 0, 0)]
    calls += [(size(31), size(31), rng.choice([1, 32, 100, 4096]), rng.choice([0, 0, size(16)]),
               rng.randrange(2)) for _ in range(20000)]
    calls += [(size(14), size(14), 32 * size(9), rng.choice([0, 0, size(8)]), rng.randrange(2))
              for _ in range(20000)]
    refused, seen = 0, set()
    for M, N, K, groups, aligned in calls:
        kernel = pg.mx4gemm_select_kernel(M, N, K, groups, aligned, 256)
        if kernel >= 0:
            name = pg.MX4GEMM_KERNELS[kernel]
            seen.add(name)
            assert mx4_work_items(name, M, N, groups) < 2**32, (M, N, K, groups, aligned, name)
            assert name[0] != "L" or (aligned and K % 32 == 0)
            continue
        refused += 1
        assert kernel == -22
        largest = "L256x256" if aligned and K % 32 == 0 else "T128x128"
        assert mx4_work_items(largest, M, N, groups) >= 2**32, (M, N, K, groups, aligned)
    assert 0 < refused < 20000 and seen == set(pg.MX4GEMM_KERNELS)
    for bad, status in (((-1, 1, 1, 0), -1501), ((1, -1, 1, 0), -1502), ((1, 1, -1, 0), -1503),
                        ((1, 1, 1, 65537), -1604)):
        assert pg.mx4gemm_select_kernel(*bad, 1, 256) == status
    assert pg.mx4gemm_select_kernel(0, 0, 0, 0, 0, 0) >= 0


def test_workspaces(pg):
    torch = pytest.importorskip("torch")
    size = pg.rms_norm_grad_workspace_size
    assert size(0, 100, torch.float32) == 0
    assert 400 <= size(1, 100, torch.float32) <= 16 * 400
    assert 0 < size(1 << 30, 16384, torch.bfloat16) <= 1024 * 16384 * 4
    assert size(4, 16385, torch.float16) == 0 and size(-1, 4, torch.float16) == 0
    size = pg.expert_layer_workspace_size
    assert size(1, 1, 1, 1, torch.float32) > 0
    values = 512 * (768 * 4 + 2048 * 4)  # the inner values and the partial products
    assert values <= size(64, 8, 2048, 768, torch.bfloat16) <= values + 512 * 128
    for bad in ((-1, 1, 4, 4), (1, 0, 4, 4), (2049, 1, 4, 4), (1, 1, -1, 4), (1, 1, 4, 2**20 + 1)):
        assert size(*bad, torch.float32) == 0
    # without dweight the gradient takes none
    assert call(pg, "rms_norm_grad", M=0, dweight=None, workspace=None, workspace_bytes=0) == 0


def test_binding_refuses_host_tensors(pg):
    torch = pytest.importorskip("torch")
    x, q, s = torch.zeros(4, 4), torch.zeros(4, 4, dtype=torch.uint8), torch.zeros(4)
    for bad, name in (
            (lambda: pg.rms_norm(4, 4, x, 4, None, 0, s, 0.0, None, 0, x, 4), "X"),
            (lambda: pg.rms_norm_i8(4, 4, x, 4, None, 0, s, 0.0, None, 0, q, 4, s), "X"),
            (lambda: pg.rms_norm_grad(4, 4, x, 4, x, 4, s, 0.0, None, 0, x, 4, None, None), "dY"),
            (lambda: pg.mx4_quantize_rows(4, 4, x, 4, q, 4, q, 4), "X"),
            (lambda: pg.mx4_dequantize_rows(4, 4, q, 4, q, 4, x, 4), "Q"),
            (lambda: pg.mx4gemm(4, 4, 4, q, 4, q, 4, q, 4, q, 4, None, x, 4), "A"),
            (lambda: pg.mx4gemm_grouped(4, 4, 4, 1, s, q, 4, q, 4, q, 4, 0, q, 4, 0, None, x, 4),
             "offsets"),
            (lambda: pg.expert_layer(1, 1, 1, 4, 4, x, 4, s, None, x, 4, 0, None, x, 4, 0, None, x,
                                     4, None), "X")):
        with pytest.raises(TypeError, match=name + " must be a GPU tensor"):
            bad()


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


def operands(torch, make):
    """Operands of one valid call of each, by name."""
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    M, N, K, G, E, H, F = 4, 6, 200, 2, 3, 40, 72
    w = K // 2
    norm = dict(M=M, K=K, X=make(M, K, dtype=bf), ldx=K, R=make(M, K, dtype=bf), ldr=K,
                weight=make(K), eps=1e-6, H=make(M, K, dtype=bf), ldh=K)
    mx = dict(A=make(M, w, dtype=u8), lda=w, scaleA=make(2, M, 4, dtype=u8), ldsa=M)
    layer = dict(tokens=M, topk=2, experts=E, H=H, F=F, X=make(M, H, dtype=bf), ldx=H,
                 ids=make(M, 2, dtype=i32), weights=make(M, 2))
    tail = dict(out=make(M, H, dtype=bf), ldo=H, workspace=make(1 << 16, dtype=u8))
    return {
        "rms_norm": dict(**norm, Y=make(M, K, dtype=bf), ldy=K),
        "rms_norm_i8": dict(**norm, Q=make(M, K, dtype=torch.int8), ldq=K, scale=make(M)),
        "rms_norm_grad": dict(M=M, K=K, dY=make(M, K, dtype=bf), lddy=K, H=make(M, K, dtype=bf),
                              ldh=K, weight=make(K), eps=0.0, dH=make(M, K, dtype=bf), lddh=K,
                              dX=make(M, K, dtype=bf), lddx=K, dweight=make(K),
                              workspace=make(1 << 16, dtype=u8)),
        "mx4_quantize_rows": dict(M=M, K=K, X=make(M, K), ldx=K, Q=make(M, w, dtype=u8), ldq=w,
                                  scale=make(2, M, 4, dtype=u8), lds=M),
        "mx4_dequantize_rows": dict(M=M, K=K, Q=make(M, w, dtype=u8), ldq=w,
                                    scale=make(2, M, 4, dtype=u8), lds=M, Y=make(M, K), ldy=K),
        "mx4gemm": dict(M=M, N=N, K=K, **mx, B=make(N, w, dtype=u8), ldb=w,
                        scaleB=make(2, N, 4, dtype=u8), ldsb=N, bias=make(N), C=make(M, N), ldc=N),
        "mx4gemm_grouped": dict(M=M, N=N, K=K, groups=G, offsets=make(G + 1, dtype=i32), **mx,
                                B=make(G, N, w, dtype=u8), ldb=w, strideB=N * w,
                                scaleB=make(G, 2, N, 4, dtype=u8), ldsb=N, strideSB=8 * N,
                                bias=make(G, N), C=make(M, N), ldc=N),
        "expert_layer": dict(**layer, W1=make(E, 2 * F, H, dtype=bf), ldw1=H, strideW1=2 * F * H,
                             scale1=None, W2=make(E, H, F, dtype=bf), ldw2=F, strideW2=H * F,
                             scale2=None, **tail),
        "expert_layer i8": dict(**layer, W1=make(E, 2 * F, H, dtype=torch.int8), ldw1=H,
                                strideW1=2 * F * H, scale1=make(E, 2 * F),
                                W2=make(E, H, F, dtype=torch.int8), ldw2=F, strideW2=H * F,
                                scale2=make(E, H), **tail),
        "expert_layer mx4": dict(**layer, W1=make(E, 2 * F, H // 2, dtype=u8), ldw1=H // 2,
                                 strideW1=F * H, scale1=make(E, 1, 2 * F, 4, dtype=u8),
                                 W2=make(E, H, F // 2, dtype=u8), ldw2=F // 2,
                                 strideW2=H * F // 2, scale2=make(E, 1, H, 4, dtype=u8), **tail),
    }


NAMES = ["rms_norm", "rms_norm_i8", "rms_norm_grad", "mx4_quantize_rows", "mx4_dequantize_rows",
         "mx4gemm", "mx4gemm_grouped", "expert_layer", "expert_layer i8", "expert_layer mx4"]


@pytest.mark.parametrize("name", NAMES)
def test_binding_takes_what_it_needs(pg, on_host, name):
    """Every operand exactly as large as the call needs is taken; one element
    short, of another type or with gaps, it is refused, by its name."""
    torch, make = on_host
    fn = getattr(pg, name.split()[0])
    args = operands(torch, make)[name]
    assert len(fn(*args.values())) >= len(args)
    for key, v in args.items():
        if not isinstance(v, torch.Tensor) or key == "workspace":
            continue
        # (Rows at a leading dimension are taken as they lie, whatever the shape.)
        with pytest.raises(ValueError, match="^%s holds" % key):
            fn(*{**args, key: v.reshape(-1)[1:]}.values())
        with pytest.raises(TypeError, match="^%s must be" % key):
            fn(*{**args, key: v.to(torch.float64)}.values())
        with pytest.raises(TypeError, match="^%s must be a GPU tensor" % key):
            fn(*{**args, key: [1.0]}.values())
        optional = key in ("R", "H", "dH", "dweight", "weights", "bias") and \
            (key, name) != ("H", "rms_norm_grad")
        if optional:
            fn(*{**args, key: None}.values())
        else:
            with pytest.raises(TypeError, match="^%s must be a GPU tensor" % key):
                fn(*{**args, key: None}.values())


@pytest.mark.parametrize("name,keys", [
    ("rms_norm", ["weight"]), ("rms_norm_i8", ["weight", "scale"]),
    ("rms_norm_grad", ["weight", "dweight", "workspace"]), ("mx4_quantize_rows", ["scale"]),
    ("mx4_dequantize_rows", ["scale"]), ("mx4gemm", ["scaleA", "scaleB", "bias"]),
    ("mx4gemm_grouped", ["offsets", "scaleA", "scaleB", "bias"]),
    ("expert_layer", ["ids", "weights", "workspace"]),
    ("expert_layer i8", ["scale1", "scale2"]), ("expert_layer mx4", ["scale1", "scale2"])])
def test_binding_refuses_vectors_with_gaps(pg, on_host, name, keys):
    torch, make = on_host
    fn = getattr(pg, name.split()[0])
    args = operands(torch, make)[name]
    for key in keys:
        v = args[key]
        gaps = make(*v.shape[:-1], 2 * v.shape[-1], dtype=v.dtype)[..., :v.shape[-1]] \
            if v.dim() > 1 else make(2 * v.shape[0], dtype=v.dtype)[::2]
        with pytest.raises(ValueError, match="^%s must be contiguous" % key):
            fn(*{**args, key: gaps}.values())


def test_binding_takes_torchs_types_of_four_bits(pg, on_host):
    torch, make = on_host
    if not hasattr(torch, "float4_e2m1fn_x2") or not hasattr(torch, "float8_e8m0fnu"):
        pytest.skip("this torch has no types of 4 bits")
    args = operands(torch, make)["mx4gemm"]
    for key in ("A", "B"):
        args[key] = args[key].view(torch.float4_e2m1fn_x2)
    for key in ("scaleA", "scaleB"):
        args[key] = args[key].view(torch.float8_e8m0fnu)
    pg.mx4gemm(*args.values())


def test_binding_refuses_mixed_types(pg, on_host):
    """Operands that share a type have to, and weights are X's type, int8 or 4-bit
    blocks."""
    torch, make = on_host
    all_args = operands(torch, make)
    for name, key, dtype in (("rms_norm", "R", torch.float16), ("rms_norm", "Y", torch.float32),
                             ("rms_norm_grad", "H", torch.float32),
                             ("rms_norm_grad", "dH", torch.float16),
                             ("expert_layer", "W1", torch.float32),
                             ("expert_layer", "W2", torch.float16),
                             ("expert_layer", "out", torch.float32),
                             ("expert_layer i8", "W2", torch.uint8),
                             ("mx4gemm", "B", torch.int8)):
        args = dict(all_args[name])
        args[key] = args[key].to(dtype)
        with pytest.raises(TypeError, match="^%s must be" % key):
            getattr(pg, name.split()[0])(*args.values())


@pytest.mark.parametrize("name", NAMES)
def test_binding_refuses_sizes_beyond_an_int(pg, on_host, name):
    """2^32 + n and -2^32 + n would reach the library as n."""
    torch, make = on_host
    fn = getattr(pg, name.split()[0])
    args = operands(torch, make)[name]
    for key, v in args.items():
        if isinstance(v, torch.Tensor) or v is None or key == "eps":
            continue
        most = 2**64 if key.startswith("stride") else 2**32
        for bad in (v + most, v - most):
            with pytest.raises((ValueError, TypeError)):
                fn(*{**args, key: bad}.values())


def test_workspace_types(pg, on_host):
    torch, make = on_host
    args = operands(torch, make)["rms_norm_grad"]
    for ws in (1 << 20, b"0" * 4096, torch.zeros(4096)):
        with pytest.raises(TypeError, match="workspace must be a GPU tensor"):
            pg.rms_norm_grad(*{**args, "workspace": ws}.values())
    assert pg.rms_norm_grad(*{**args, "workspace": make(64)}.values())[-1] == 256
    assert pg.rms_norm_grad(*{**args, "workspace": None}.values())[-2:] == (None, 0)


def test_without_torch(pg):
    code = """
import sys
sys.modules["torch"] = None  # imports of it fail
from precision_gemm_amd import *
import precision_gemm_amd as pg
assert all(hasattr(pg, n) for n in pg.__all__)
assert RMS_NORM_GRAD_MAX_K == 16384 and EXPERT_LAYER_MAX_SLOTS == 2048
for call in (lambda: rms_norm(1, 1, None, 1, None, 1, None, 0.0, None, 1, None, 1),
             lambda: mx4_quantize_rows(1, 1, None, 1, None, 1, None, 1)):
    try:
        call()
    except ImportError as e:
        assert "torch" in str(e)
    else:
        raise SystemExit("taken")
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
