"""Calls that reach every kernel of the grouped fp32 products and of the 8-bit
products, and the kernel each is for: test_kernel_choice.py checks without a
GPU that every kernel is among them and is the one chosen on 256 compute units,
test_gpu_kernels.py runs them."""
from collections import namedtuple

# counts: rows of each group; pad: elements between rows; shift: elements before
# the first of each operand.
Grouped = namedtuple("Grouped", "kernel tB counts N K pad shift alpha beta")
Outer = namedtuple("Outer", "kernel counts M N pad shift alpha beta")
# counts None: one product of M rows.
I8 = namedtuple("I8", "kernel M counts N K pad shift out bias")

LEAD, TAIL = 2, 3  # rows before the first group's and behind the last one's
UNEVEN = [1300, 0, 700, 511, 1, 64, 2050, 65, 127, 129, 900, 333, 0, 1024, 700, 288]  # 8192 rows
FIVE = [700, 0, 1, 1023, 576]  # 2300 rows
THREE = [8000, 129, 8300]  # 16429 rows
FEW = [5, 0, 9, 16]

GROUPED = [
    Grouped("S16x16", 0, FEW, 70, 132, 0, 0, 1.0, 0.0),
    Grouped("S16x16", 1, FEW, 70, 133, 3, 1, -0.5, 2.0),
    Grouped("S32x16", 0, [1300], 70, 261, 1, 3, 1.0, 0.0),
    Grouped("S32x16", 1, [600], 100, 132, 0, 0, -0.5, 2.0),
    Grouped("S16x64", 0, [1] * 16, 4096, 260, 0, 0, 1.0, 0.0),
    Grouped("S16x64", 1, [1, 1, 0, 1] * 4, 4099, 133, 2, 1, -0.5, 2.0),
    Grouped("S32x64", 0, [16, 17, 0, 67] * 4, 514, 261, 1, 2, 1.0, 0.0),
    Grouped("S32x64", 1, [16, 17, 0, 67] * 4, 512, 132, 0, 0, -0.5, 2.0),
    Grouped("T64x64", 0, UNEVEN, 2048, 1024, 0, 0, 1.0, 0.0),
    Grouped("T64x64", 1, UNEVEN, 1024, 2048, 0, 0, 1.0, 0.0),
    Grouped("T64x64", 0, FIVE, 516, 132, 4, 4, -0.5, 2.0),
    Grouped("T64x64", 1, FIVE, 514, 132, 8, 4, -0.5, 2.0),
    Grouped("T64x64", 0, FIVE, 512, 4, 0, 0, 1.0, 0.0),
    Grouped("T64x64", 1, FIVE, 513, 20, 0, 0, 1.0, 0.5),
    Grouped("T64x64_ANY", 0, UNEVEN, 2047, 1023, 0, 0, 1.0, 0.0),
    Grouped("T64x64_ANY", 1, UNEVEN, 1025, 2047, 1, 1, 1.0, 0.0),
    Grouped("T64x64_ANY", 0, FIVE, 511, 131, 1, 1, -0.5, 2.0),
    Grouped("T64x64_ANY", 0, FIVE, 513, 17, 2, 3, 1.0, 0.0),
    Grouped("T64x64_ANY", 0, FIVE, 514, 33, 3, 2, 1.0, 0.0),
    Grouped("T64x64_ANY", 0, FIVE, 515, 1, 0, 0, 1.0, 0.5),
    Grouped("T64x64_ANY", 0, FIVE, 512, 48, 0, 1, 1.0, 0.0),
    Grouped("T64x64_ANY", 1, FIVE, 511, 131, 1, 1, -0.5, 2.0),
    Grouped("T64x64_ANY", 1, FIVE, 513, 17, 2, 3, 1.0, 0.0),
    Grouped("T64x64_ANY", 1, FIVE, 514, 33, 3, 2, 1.0, 0.0),
    Grouped("T64x64_ANY", 1, FIVE, 515, 1, 0, 0, 1.0, 0.5),
    Grouped("T64x64_ANY", 1, FIVE, 512, 48, 0, 1, 1.0, 0.0),
    Grouped("T128x128", 0, THREE, 4096, 132, 0, 0, 1.0, 0.0),
    Grouped("T128x128", 1, THREE, 4100, 260, 4, 4, -0.5, 2.0),
    Grouped("T128x128", 0, THREE, 4100, 20, 4, 4, -0.5, 2.0),
    Grouped("T128x128", 1, THREE, 4097, 36, 0, 0, 1.0, 0.0),
]
# A is [rows, 2] and B [groups, 2, 3] here: 1-float loads are for rows that the
# streams' tiles do not fit a launch with.
GROUPED_V1 = Grouped("T64x64_V1", 0, [2**27, 0, 2**27 + 99], 3, 2, 0, 0, 1.0, 0.0)

OUTER = [
    Outer("S16x16", [5, 0, 70], 20, 33, 1, 1, -0.5, 2.0),
    Outer("S16x16", [300, 1], 64, 64, 0, 0, 1.0, 0.0),
    Outer("S32x32", [100, 0, 3, 65], 250, 260, 0, 0, 1.0, 0.0),
    Outer("S32x32", [100, 0, 3, 65], 251, 261, 3, 2, -0.5, 2.0),
    Outer("T64x64", [40, 0, 129, 16, 1, 90], 512, 516, 0, 0, 1.0, 0.0),
    Outer("T64x64", [40, 0, 129, 16, 1, 90], 516, 512, 4, 4, -0.5, 2.0),
    Outer("T64x64_ANY", [40, 0, 129, 16, 1, 90], 511, 513, 0, 0, 1.0, 0.0),
    Outer("T64x64_ANY", [40, 0, 129, 16, 1, 90], 514, 515, 1, 3, -0.5, 2.0),
    Outer("T64x64_ANY", [17, 33, 2, 0, 15], 512, 512, 0, 1, 1.0, 0.0),
    Outer("T128x128", UNEVEN, 1024, 2048, 0, 0, 1.0, 0.0),
    Outer("T128x128", [40, 0, 129, 16, 1, 90] * 2, 2052, 2056, 4, 4, -0.5, 2.0),
    Outer("T128x128_ANY", UNEVEN, 1023, 2047, 0, 0, 1.0, 0.0),
    Outer("T128x128_ANY", [40, 0, 129, 16, 1, 90] * 3, 1025, 2050, 1, 3, -0.5, 2.0),
    Outer("T128x128_ANY", [17, 33, 2, 0, 15, 16] * 3, 1026, 2051, 2, 1, 1.0, 0.0),
]
OUTER_V1 = Outer("T64x64_V1", [1, 0, 2] + [1] * 60 + [0, 7], 1, 2**21 - 1, 0, 0, 1.0, 0.0)

I8_CASES = [
    I8("S16x16", 3, None, 200, 1040, 0, 0, "float32", True),
    I8("S16x16", 9, None, 200, 1041, 0, 0, "bfloat16", False),
    I8("S16x16_W16", 2, None, 500, 8192, 0, 0, "float32", False),
    I8("S16x16_W16", 4, None, 511, 4100, 3, 5, "float16", True),
    I8("S16x32", 16, None, 16400, 272, 0, 0, "float32", False),
    I8("S16x32", 13, None, 16399, 301, 1, 7, "bfloat16", True),
    I8("S16x32", None, [3, 0, 16, 1, 20, 0, 2, 5], 300, 528, 0, 0, "float32", True),
    I8("S16x32", None, [30, 0, 16, 1, 20, 0, 2, 40], 300, 529, 2, 3, "float32", False),
    I8("S32x16", 33, None, 1000, 1024, 0, 0, "float32", True),
    I8("S32x16", 60, None, 1001, 1027, 2, 9, "float16", False),
    I8("S32x32", 64, None, 4000, 528, 0, 0, "float32", False),
    I8("S32x32", 50, None, 4001, 531, 5, 1, "bfloat16", True),
    I8("S32x64", 32, None, 12288, 4096, 0, 0, "float32", True),
    I8("S32x64", 17, None, 12289, 1000, 0, 0, "bfloat16", False),
    I8("S32x64", 29, None, 9000, 513, 7, 3, "float16", True),
    I8("T64x64", 300, None, 900, 1000, 8, 0, "float32", False),
    I8("T64x64", None, [40, 0, 129, 16, 1, 90], 300, 333, 1, 5, "bfloat16", True),
    I8("T128x128", 2000, None, 2100, 1000, 0, 0, "float32", True),
    I8("T128x128", None, UNEVEN, 700, 527, 1, 1, "float16", False),
    # rows on 16-byte boundaries, K that ends within a chunk
    I8("T64x64", 300, None, 900, 1005, 3, 0, "float32", True),
    I8("T128x128", 2000, None, 2100, 1001, 7, 0, "bfloat16", False),
    I8("L32x64", 100, None, 4000, 1040, 0, 0, "float32", True),
    I8("L64x64_R4", 250, None, 4093, 272, 16, 16, "bfloat16", False),
    I8("L64x64", 822, None, 2468, 2064, 0, 0, "float32", True),
    I8("L64x64", 6274, None, 563, 16, 0, 0, "bfloat16", False),
    I8("L64x128", 300, None, 4001, 2064, 0, 0, "float32", False),
    I8("L128x128", 1900, None, 2047, 2048, 0, 0, "float16", True),
    I8("L128x256", 2000, None, 4095, 2032, 0, 0, "float32", True),
    I8("L256x256", 4001, None, 8192, 656, 0, 0, "bfloat16", False),
    I8("L128x256", None, UNEVEN, 8190, 528, 0, 0, "float16", False),
    I8("L256x256", None, UNEVEN, 5998, 1040, 0, 0, "float32", True),
]


def rows(case):
    return LEAD + sum(case.counts) + TAIL


def vec4(case, *extents):
    """Whether operands of these row extents allow 16-byte loads."""
    return (case.pad | case.shift) % 4 == 0 and all(e % 4 == 0 for e in extents)


def grouped_choice(pg, case, cus):
    allowed = vec4(case, case.K, 0 if case.tB else case.N)
    number = pg.sgemm_grouped_select_kernel(case.tB, rows(case), case.N, len(case.counts), allowed,
                                            cus)
    return pg.GROUPED_KERNELS[number] if number >= 0 else number


def outer_choice(pg, case, cus):
    number = pg.sgemm_grouped_outer_select_kernel(case.M, case.N, len(case.counts),
                                                  vec4(case, case.M, case.N), cus)
    return pg.GROUPED_OUTER_KERNELS[number] if number >= 0 else number


def i8_aligned(case):
    return (case.K + case.pad) % 16 == 0 and case.shift % 16 == 0


def i8_choice(pg, case, cus):
    M, groups = (case.M, 0) if case.counts is None else (rows(case), len(case.counts))
    number = pg.i8gemm_select_kernel(M, case.N, case.K, groups, i8_aligned(case), cus)
    return pg.I8GEMM_KERNELS[number] if number >= 0 else number


def name(case):
    return "-".join(str(v) if not isinstance(v, list) else f"{len(v)}x{sum(v)}" for v in case)
