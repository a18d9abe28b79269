"""Every kernel of the grouped fp32 products and of the 8-bit products
(kernel_cases.py) on whole numbers, whose results are exact, and the fp32 ones
on random floats within their roundings. Beside the operands' rows, before the
first and behind the last lies NaN."""
import sys

import numpy as np
import pytest

import kernel_cases as kc

pytestmark = pytest.mark.gpu


def log(msg):
    sys.stdout.write(msg + "\n")
    sys.stdout.flush()


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_gemm_amd as pg
    pg._load()
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    return torch, pg, cus, torch.Generator(device="cuda")


def starts(counts, lead=kc.LEAD):
    return [lead + int(e) for e in np.concatenate([[0], np.cumsum(counts)])]


class Matrix:
    """count x rows x cols floats at the case's pad and shift, NaN around them."""

    def __init__(self, torch, values, pad, shift):
        self.values = values
        n, rows, cols = values.shape
        self.ld = cols + pad
        self.stride = rows * self.ld
        self.store = torch.full((shift + n * self.stride + 8,), torch.nan, device="cuda")
        self.t = self.store[shift:]
        self.view = self.t[:n * self.stride].view(n, rows, self.ld)[:, :, :cols]
        self.view.copy_(values)
        self.before = self.store.clone()

    def only_changed(self, torch, rows):
        """Whether all but the values of these rows is as it was, bit for bit."""
        self.view[:, rows].copy_(self.values[:, rows])
        return torch.equal(self.store.view(torch.int32), self.before.view(torch.int32))


# How the operands of a product over k are filled:
#   small   whole numbers up to 4 in both: every partial sum is exact
#   wide_a  whole numbers of up to 24 bits in the left operand against a right
#           one of 0 and +-1, few enough in each column that sums stay exact:
#           an operand that lost bits on its way would show
#   wide_b  the same the other way round
#   floats  uniform in (-1, 1)
FILLS = ["small", "wide_a", "wide_b", "floats"]


def fill_pair(torch, g, fill, a_shape, b_shape, a_k, b_k, terms):
    """a_k, b_k: which dimension of each runs along k; terms: of a sum over k."""
    whole = lambda shape, most: torch.randint(-most, most + 1, shape, generator=g,  # noqa: E731
                                              device="cuda").float()
    if fill == "small":
        return whole(a_shape, 4), whole(b_shape, 4)
    if fill == "floats":
        return tuple(torch.rand(s, generator=g, device="cuda") * 2 - 1 for s in (a_shape, b_shape))
    wide_shape, shape, k = (a_shape, b_shape, b_k) if fill == "wide_a" else (b_shape, a_shape, a_k)
    other = 3 - k  # (shapes are count x 2 dimensions)
    index = [torch.arange(shape[d], device="cuda").view([-1 if i == d else 1 for i in range(3)])
             for d in range(3)]
    # terms `every` apart, so that each k has one and each row or column has one
    every = min(shape[1], shape[2])
    at = (index[k] - index[other] - 3 * index[0]) % every == 0
    sparse = at.float() * (1 - 2 * (whole(shape, 4) > 0).float())
    most = -(-terms // every)
    return (whole(wide_shape, (1 << 24) // most), sparse) if fill == "wide_a" else \
        (sparse, whole(wide_shape, (1 << 24) // most))


def check(torch, got, a, b, c, case, fill, what):
    """got against alpha a b + beta c in 64 bits. On floats every product goes
    through at most its own rounding, one for each of the other terms and one
    for each of 16 waves' sums; then come three of the epilogue."""
    a, b = a.double().contiguous(), b.double().contiguous()
    want = case.alpha * (a @ b)
    if case.beta:
        want += case.beta * c.double()
    err = (got.double() - want).abs()
    if fill == "floats":
        size = abs(case.alpha) * (a.abs() @ b.abs())
        if case.beta:
            size += abs(case.beta) * c.double().abs()
        tol = 1.01 * (a.shape[1] + 20) * 2.0 ** -24 * size
    else:
        tol = torch.zeros_like(want)
    assert (err <= tol).all(), (what, err.max().item(), int((~(err <= tol)).sum()))


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("case", kc.GROUPED, ids=kc.name)
def test_grouped(env, case, fill):
    torch, pg, cus, g = env
    log(f"[kernels] {case} {fill}")
    assert kc.grouped_choice(pg, case, cus) == case.kernel
    g.manual_seed(case.N * 7 + case.K)
    ends, G, N, K, tB = starts(case.counts), len(case.counts), case.N, case.K, case.tB
    M = kc.rows(case)
    if fill.startswith("wide"):  # (exact without the scalars)
        case = case._replace(alpha=1.0, beta=0.0)
    a, b = fill_pair(torch, g, fill, (1, M, K), (G, N, K) if tB else (G, K, N), 2, 2 if tB else 1,
                     K)
    a[:, :ends[0]], a[:, ends[-1]:] = torch.nan, torch.nan
    A, B = Matrix(torch, a, case.pad, case.shift), Matrix(torch, b, case.pad, case.shift)
    c = torch.randint(-4, 5, (1, M, N), generator=g, device="cuda").float() if case.beta else \
        torch.full((1, M, N), torch.nan, device="cuda")
    C = Matrix(torch, c, case.pad, case.shift)
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    pg.sgemm_grouped(tB, M, N, K, G, off, case.alpha, A.t, A.ld, B.t, B.ld, B.stride, case.beta,
                     C.t, C.ld)
    torch.cuda.synchronize()
    for e in range(G):
        rows = slice(ends[e], ends[e + 1])
        check(torch, C.view[0, rows], a[0, rows], b[e].t() if tB else b[e], c[0, rows], case, fill,
              e)
    assert C.only_changed(torch, slice(ends[0], ends[-1]))


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("case", kc.OUTER, ids=kc.name)
def test_outer(env, case, fill):
    torch, pg, cus, g = env
    log(f"[kernels] {case} {fill}")
    assert kc.outer_choice(pg, case, cus) == case.kernel
    g.manual_seed(case.M * 7 + case.N)
    ends, G, M, N = starts(case.counts), len(case.counts), case.M, case.N
    K = kc.rows(case)
    if fill.startswith("wide"):
        case = case._replace(alpha=1.0, beta=0.0)
    a, b = fill_pair(torch, g, fill, (1, K, M), (1, K, N), 1, 1, max(case.counts))
    for x in (a, b):
        x[:, :ends[0]], x[:, ends[-1]:] = torch.nan, torch.nan
    A, B = Matrix(torch, a, case.pad, case.shift), Matrix(torch, b, case.pad, case.shift)
    c = torch.randint(-4, 5, (G, M, N), generator=g, device="cuda").float() if case.beta else \
        torch.full((G, M, N), torch.nan, device="cuda")
    C = Matrix(torch, c, case.pad, case.shift)
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    pg.sgemm_grouped_outer(M, N, K, G, off, case.alpha, A.t, A.ld, B.t, B.ld, case.beta, C.t, C.ld,
                           C.stride)
    torch.cuda.synchronize()
    for e in range(G):
        rows = slice(ends[e], ends[e + 1])
        check(torch, C.view[e], a[0, rows].t(), b[0, rows], c[e], case, fill, e)
    assert C.only_changed(torch, slice(None))


def test_grouped_rows_beyond_the_streams(env):
    torch, pg, cus, g = env
    case = kc.GROUPED_V1
    log(f"[kernels] {kc.name(case)}")
    assert kc.grouped_choice(pg, case, cus) == case.kernel
    g.manual_seed(1)
    ends = starts(case.counts)
    M, N, K = kc.rows(case), case.N, case.K
    A = torch.empty(M, K, device="cuda").uniform_(-1000, 1000, generator=g).round_()
    B = torch.randint(-4, 5, (3, K, N), generator=g, device="cuda").float()
    C = torch.full((M * N + 5,), torch.nan, device="cuda")
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    pg.sgemm_grouped(0, M, N, K, 3, off, 1.0, A, K, B, N, K * N, 0.0, C, N)
    torch.cuda.synchronize()
    for e in (0, 2):
        for lo in range(ends[e], ends[e + 1], 1 << 24):
            hi = min(lo + (1 << 24), ends[e + 1])
            want = A[lo:hi, :1] * B[e, 0] + A[lo:hi, 1:] * B[e, 1]  # exact
            assert torch.equal(C[lo * N:hi * N].view(-1, N), want), (e, lo)
    assert C[:ends[0] * N].isnan().all() and C[ends[-1] * N:].isnan().all()


def test_outer_outputs_beyond_the_streams(env):
    torch, pg, cus, g = env
    case = kc.OUTER_V1
    log(f"[kernels] {kc.name(case)}")
    assert kc.outer_choice(pg, case, cus) == case.kernel
    g.manual_seed(2)
    ends, G, M, N = starts(case.counts), len(case.counts), case.M, case.N
    K = kc.rows(case)
    A = torch.randint(-1000, 1001, (K, M), generator=g, device="cuda").float()
    B = torch.randint(-1000, 1001, (K, N), generator=g, device="cuda").float()
    C = torch.full((G * N + 5,), torch.nan, device="cuda")
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    pg.sgemm_grouped_outer(M, N, K, G, off, 1.0, A, M, B, N, 0.0, C, N, N)
    torch.cuda.synchronize()
    for e in range(G):
        want = (A[ends[e]:ends[e + 1]] * B[ends[e]:ends[e + 1]]).sum(0)  # exact
        assert torch.equal(C[e * N:(e + 1) * N], want), e
    assert C[G * N:].isnan().all()


@pytest.mark.parametrize("case", kc.I8_CASES, ids=kc.name)
def test_i8(env, case):
    """Sums over k are whole numbers, the scales powers of two and the biases
    whole numbers, so that the conversion to fp32, the sum with the bias and the
    conversion to C's type are the only roundings: equal bits."""
    torch, pg, cus, g = env
    log(f"[kernels] {case}")
    assert kc.i8_choice(pg, case, cus) == case.kernel
    N, K, ld = case.N, case.K, case.K + case.pad
    if case.counts is None:
        ends, G, M = [0, case.M], 1, case.M
    else:
        ends, G, M = starts(case.counts), len(case.counts), kc.rows(case)
    g.manual_seed(M + N + K)

    def rows(n):
        t = torch.randint(-128, 128, (case.shift + n * ld,), generator=g, device="cuda",
                          dtype=torch.int8)[case.shift:]
        return t, t.view(n, ld)[:, :K].double()

    A, a = rows(M)
    B, b = rows(G * N)
    b = b.view(G, N, K)
    power = lambda *s: torch.randint(-9, -3, s, generator=g,  # noqa: E731
                                     device="cuda").float().exp2()
    sA, sB = power(M), power(G, N)
    bias = torch.randint(-50, 51, (G, N), generator=g, device="cuda").float() if case.bias else None
    dt = getattr(torch, case.out)
    C = torch.full((M + 2, N + 3), 7.0, dtype=dt, device="cuda")
    if case.counts is None:
        pg.i8gemm(M, N, K, A, ld, sA, B, ld, sB, bias, C[1:], N + 3)
    else:
        off = torch.tensor(ends, dtype=torch.int32, device="cuda")
        pg.i8gemm_grouped(M, N, K, G, off, A, ld, sA, B, ld, N * ld, sB, bias, C[1:], N + 3)
    torch.cuda.synchronize()
    for e in range(G):
        lo, hi = ends[e], ends[e + 1]
        acc = (a[lo:hi] @ b[e].t().contiguous()).float()
        want = acc.double() * sA[lo:hi, None].double() * sB[e].double()
        if case.bias:
            want = want + bias[e].double()  # exact in 64 bits
        assert torch.equal(C[lo + 1:hi + 1, :N], want.float().to(dt)), e
    assert (C[:ends[0] + 1] == 7).all() and (C[ends[-1] + 1:] == 7).all()
    assert (C[:, N:] == 7).all()
