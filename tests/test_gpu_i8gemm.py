"""The 8-bit integer product and its row quantization against 64-bit values.

The integer sums are exact, so a product's error comes from three fp32
roundings (the sum to fp32, times each scale), the sum with the bias and the
rounding to C's type."""
import sys

import numpy as np
import pytest

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
    return torch, pg


TYPES = ["float32", "float16", "bfloat16"]


def tolerance(torch, dtype, product, bias):
    """|computed - exact| of one element: the fp32 roundings are of numbers no
    larger than |product| + |bias| up to their own roundings (hence 4.1 for 4),
    the last one to `dtype` (half a step, or half the smallest number)."""
    size = product.abs() + bias.abs()
    fp32 = 4.1 * 2.0 ** -24 * size
    if dtype == torch.float32:
        return fp32
    return fp32 + (size + fp32) * torch.finfo(dtype).eps / 2 + \
        torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


class Operand:
    """rows x cols int8 at stride ld, `shift` bytes into its storage."""

    def __init__(self, torch, rng, rows, cols, ld=None, shift=0, groups=1, extreme=False):
        self.ld = max(1, cols if ld is None else ld)
        self.stride = max(1, rows) * self.ld
        n = groups * self.stride + shift
        store = rng.integers(-128, 128, n, dtype=np.int8)
        if extreme:
            store[:] = -128
        self.t = torch.from_numpy(store).cuda()[shift:]
        host = torch.from_numpy(store[shift:shift + groups * self.stride].copy())
        self.host = host.view(groups, max(1, rows), self.ld)[:, :rows, :cols].double()


def product_case(env, M, N, K, dtype="bfloat16", counts=None, first=0, bias=False, lda=None,
                 ldb=None, shift=0, ldc=None, extreme=False, seed=0):
    """One call against 64 bits; counts: rows of each group, from row `first`."""
    torch, pg = env
    log(f"[i8gemm] {M}x{N}x{K} {dtype} counts={counts} first={first} lda={lda} ldb={ldb} "
        f"shift={shift} ldc={ldc}")
    rng = np.random.default_rng(seed + 7 * M + 3 * N + K)
    dt = getattr(torch, dtype)
    G = 1 if counts is None else len(counts)
    A = Operand(torch, rng, M, K, lda, shift, extreme=extreme)
    B = Operand(torch, rng, N, K, ldb, shift, groups=G, extreme=extreme)
    sA = torch.from_numpy(rng.uniform(0.5, 1.5, M).astype(np.float32) / 64)
    sB = torch.from_numpy(rng.uniform(0.5, 1.5, (G, N)).astype(np.float32) / 64)
    bs = torch.from_numpy(rng.standard_normal((G, N)).astype(np.float32)) if bias else None
    ldc = ldc or max(1, N)
    C0 = torch.full((M, ldc), 7.0, dtype=dt)
    C = C0.cuda()
    dA, dB, dbs = sA.cuda(), sB.cuda(), None if bs is None else bs.cuda()
    if counts is None:
        pg.i8gemm(M, N, K, A.t, A.ld, dA, B.t, B.ld, dB, dbs, C, ldc)
        ranges = [(0, M)]
    else:
        ends = np.concatenate([[0], np.cumsum(counts)]) + first
        off = torch.from_numpy(ends.astype(np.int32)).cuda()
        pg.i8gemm_grouped(M, N, K, G, off, A.t, A.ld, dA, B.t, B.ld, B.stride, dB, dbs, C, ldc)
        ranges = [(int(ends[g]), int(ends[g + 1])) for g in range(G)]
    torch.cuda.synchronize()
    got = C.cpu()
    touched = torch.zeros(M, dtype=torch.bool)
    for g, (lo, hi) in enumerate(ranges):
        p = (A.host[0, lo:hi] @ B.host[g].T) * sA[lo:hi, None].double() * sB[g].double()
        b = torch.zeros_like(p) if bs is None else bs[g].double().expand_as(p)
        want, tol = p + b, tolerance(torch, dt, p, b)
        if dt == torch.float16:
            assert (want.abs() < 60000).all()
        err = (got[lo:hi, :N].double() - want).abs()
        assert (err <= tol).all(), (g, err.max().item(), (err / tol).max().item())
        touched[lo:hi] = True
    assert torch.equal(got[:, N:], C0[:, N:])
    assert torch.equal(got[~touched], C0[~touched])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 16, 16), (1, 1000, 512), (2, 33, 48), (3, 64, 64), (5, 257, 80), (8, 128, 4096),
    (15, 96, 112), (16, 100, 128), (17, 64, 256), (31, 31, 31), (32, 192, 1024), (33, 70, 144),
    (48, 320, 96), (63, 65, 160), (64, 64, 2048), (65, 130, 272), (100, 512, 512), (128, 128, 128),
    (129, 255, 384), (200, 300, 400), (256, 256, 64), (257, 513, 192), (512, 384, 1040),
    (700, 900, 528)])
def test_product(env, M, N, K, dtype):
    product_case(env, M, N, K, dtype, bias=(M + N) % 2 == 1)


@pytest.mark.parametrize("K", [1, 2, 15, 17, 31, 33, 63, 65, 127, 129, 255, 257, 1000, 4097])
@pytest.mark.parametrize("M", [1, 20, 150])
def test_product_any_k(env, M, K):
    product_case(env, M, 77, K, "float32", bias=True)


@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (30, 100, 256), (130, 270, 384)])
@pytest.mark.parametrize("pad,shift,cpad", [(16, 0, 0), (48, 16, 3), (1, 0, 1), (0, 1, 0),
                                            (7, 5, 9), (16, 8, 0)])
def test_product_strides(env, M, N, K, pad, shift, cpad):
    """Leading dimensions beyond the row, operands off every alignment, and
    the columns of C behind N left as they were."""
    product_case(env, M, N, K, "bfloat16", lda=K + pad, ldb=K + 2 * pad, shift=shift,
                 ldc=N + cpad)


@pytest.mark.parametrize("M,N", [(1, 48), (33, 40), (300, 290)])
def test_product_largest_sums(env, M, N):
    """Every product 2^14 over the largest K: sums next to 2^31."""
    product_case(env, M, N, 131071, "float32", extreme=True)
    product_case(env, M, N, 131056, "float32", extreme=True)


@pytest.mark.parametrize("M,N,K", [(1, 100, 64), (16, 64, 0), (0, 5, 8), (70, 0, 8)])
def test_product_empty(env, M, N, K):
    product_case(env, M, N, K, "float32", bias=True)
    product_case(env, M, N, K, "float16")


@pytest.mark.parametrize("N,K", [(64, 64), (130, 192), (96, 80), (77, 45)])
@pytest.mark.parametrize("counts,first,extra", [
    ([1], 0, 0), ([0, 0, 3], 0, 0), ([5, 0, 17, 1, 0], 0, 0), ([64, 64], 0, 5),
    ([65, 1, 130, 0, 7], 3, 4), ([0, 0], 0, 6), ([1] * 70, 0, 0), ([300, 2, 0, 129], 1, 1),
    ([3, 0, 1, 2] * 50, 0, 3)])
def test_grouped(env, counts, first, extra, N, K):
    M = first + sum(counts) + extra
    product_case(env, M, N, K, "bfloat16", counts=counts, first=first, bias=len(counts) % 2 == 1)


def test_grouped_strides(env):
    product_case(env, 150, 70, 96, "float32", counts=[20, 100, 0, 30], lda=99, ldb=101, shift=3,
                 ldc=75, bias=True)
    product_case(env, 150, 70, 96, "float16", counts=[20, 100, 0, 30], lda=128, ldb=112, shift=16)


def test_grouped_shared_weights(env):
    """strideB = 0: one B for every group, each with its own scales."""
    torch, pg = env
    g = torch.Generator().manual_seed(3)
    A = torch.randint(-128, 128, (50, 64), generator=g, dtype=torch.int8)
    B = torch.randint(-128, 128, (40, 64), generator=g, dtype=torch.int8)
    sA, sB = torch.rand(50, generator=g), torch.rand(3, 40, generator=g)
    off = torch.tensor([0, 20, 20, 50], dtype=torch.int32)
    C = torch.zeros(50, 40, device="cuda")
    pg.i8gemm_grouped(50, 40, 64, 3, off.cuda(), A.cuda(), 64, sA.cuda(), B.cuda(), 64, 0,
                      sB.cuda(), None, C, 40)
    group = torch.tensor([0] * 20 + [2] * 30)
    p = (A.double() @ B.double().T) * sA[:, None].double() * sB[group].double()
    err = (C.cpu().double() - p).abs()
    assert (err <= tolerance(torch, torch.float32, p, torch.zeros_like(p))).all()


def test_grouped_offsets_out_of_range(env):
    """Offsets outside [0, M] are brought into it, and an end before its start
    makes an empty group: rows outside every group stay as they were."""
    torch, pg = env
    A = torch.ones(8, 16, dtype=torch.int8, device="cuda")
    B = torch.ones(3, 4, 16, dtype=torch.int8, device="cuda")
    one = torch.ones(8, device="cuda")
    sB = torch.tensor([[1.0] * 4, [2.0] * 4, [4.0] * 4], device="cuda")
    for off, want in (([-5, 2, 6, 100], [1, 1, 2, 2, 2, 2, 4, 4]),
                      ([0, 4, 1, 1], [1, 1, 1, 1, 0, 0, 0, 0]),
                      ([9, 9, 9, 9], [0] * 8)):
        C = torch.zeros(8, 4, device="cuda")
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        pg.i8gemm_grouped(8, 4, 16, 3, o, A, 16, one, B, 16, 64, sB, None, C, 4)
        assert C[:, 0].tolist() == [16.0 * w for w in want], off


def test_product_scales_carry_infinity_and_nan(env):
    """Zero, infinite and NaN scales act as numbers do; a NaN bias reaches its
    channel only."""
    torch, pg = env
    inf, nan = float("inf"), float("nan")
    A = torch.tensor([[1] * 16, [0] * 16, [2] * 16, [1] * 16], dtype=torch.int8, device="cuda")
    B = torch.ones(3, 16, dtype=torch.int8, device="cuda")
    sA = torch.tensor([1.0, inf, nan, 0.0], device="cuda")
    sB = torch.tensor([1.0, -1.0, 0.5], device="cuda")
    bias = torch.tensor([0.0, nan, 1.0], device="cuda")
    C = torch.zeros(4, 3, device="cuda")
    pg.i8gemm(4, 3, 16, A, 16, sA, B, 16, sB, bias, C, 3)
    want = torch.tensor([[16, nan, 9], [nan, nan, nan], [nan, nan, nan], [0, nan, 1]])
    assert torch.equal(C.cpu().nan_to_num(-99.0), want.nan_to_num(-99.0))


def test_product_leading_dimensions_past_32_bits(env):
    """Rows 2^31 - 1 bytes apart: offsets beyond 2^32 in A, B and C."""
    torch, pg = env
    ld, K = 2**31 - 1, 96
    A = torch.empty(2 * ld + K, dtype=torch.int8, device="cuda")
    g = torch.Generator().manual_seed(4)
    rows = torch.randint(-128, 128, (3, K), generator=g, dtype=torch.int8)
    for r in range(3):
        A[r * ld:r * ld + K] = rows[r].cuda()
    one = torch.ones(3, device="cuda")
    C = torch.empty(2 * ld + 3, dtype=torch.bfloat16, device="cuda")
    pg.i8gemm(3, 3, K, A, ld, one, A, ld, one, None, C, ld)
    want = rows.double() @ rows.double().T
    for r in range(3):
        got = C[r * ld:r * ld + 3].cpu().double()
        assert ((got - want[r]).abs() <= want[r].abs() * 2.0 ** -8).all()


def test_product_many_row_tiles(env):
    """More rows than 2^16 tiles, one column."""
    torch, pg = env
    M = 64 * 70000 + 3
    A = torch.randint(-3, 4, (M, 16), dtype=torch.int8, device="cuda")
    B = torch.randint(-3, 4, (1, 16), dtype=torch.int8, device="cuda")
    one = torch.ones(M, device="cuda")
    C = torch.zeros(M, 1, device="cuda")
    pg.i8gemm(M, 1, 16, A, 16, one, B, 16, one, None, C, 1)
    assert torch.equal(C[:, 0], (A.float() * B.float()).sum(1))


def test_binding_refuses(env):
    """Short, foreign-typed and missing tensors raise before anything runs."""
    torch, pg = env
    a = torch.zeros(4, 32, dtype=torch.int8, device="cuda")
    s = torch.zeros(4, device="cuda")
    c = torch.zeros(4, 4, device="cuda")
    with pytest.raises(ValueError, match="A holds"):
        pg.i8gemm(5, 4, 32, a, 32, s, a, 32, s, None, c, 4)
    with pytest.raises(ValueError, match="B holds"):
        pg.i8gemm(4, 4, 32, a, 32, s, a, 33, s, None, c, 4)
    with pytest.raises(ValueError, match="bias holds"):
        pg.i8gemm(4, 4, 32, a, 32, s, a, 32, s, s[1:], c, 4)
    with pytest.raises(ValueError, match="C holds"):
        pg.i8gemm(4, 4, 32, a, 32, s, a, 32, s, None, c, 5)
    with pytest.raises(TypeError, match="scaleA must be"):
        pg.i8gemm(4, 4, 32, a, 32, s.half(), a, 32, s, None, c, 4)
    with pytest.raises(TypeError, match="C must be"):
        pg.i8gemm(4, 4, 32, a, 32, s, a, 32, s, None, c.int(), 4)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="offsets holds"):
        pg.i8gemm_grouped(4, 4, 32, 3, off, a, 32, s, a, 32, 0, s, None, c, 4)
    with pytest.raises(ValueError, match="B holds"):
        pg.i8gemm_grouped(4, 2, 32, 2, off, a, 32, s, a, 32, 128, s, None, c, 4)
    with pytest.raises(pg.SgemmError, match="i8gemm: invalid argument 5"):
        pg.i8gemm(4, 4, 32, a, 31, s, a, 32, s, None, c, 4)


# --- quantization ---------------------------------------------------------------------------


def quantize_want(torch, X):
    x = X.double()
    peak = x.abs().amax(1) if X.shape[1] else x.new_zeros(X.shape[0])
    scale = torch.maximum(peak / 127, torch.tensor(2.0 ** -126, dtype=torch.float64)).float()
    return torch.round(x / scale.double()[:, None]).to(torch.int8), scale


def quantize_case(env, X, ldx=None, ldq=None, shift=0):
    torch, pg = env
    M, K = X.shape
    ldx, ldq = ldx or max(1, K), ldq or max(1, K)
    log(f"[quantize] {M}x{K} {X.dtype} ldx={ldx} ldq={ldq} shift={shift}")
    store = torch.full((shift + M * ldx,), 999.0, dtype=X.dtype)
    store[shift:].view(M, ldx)[:, :K] = X
    Q = torch.full((M * ldq + shift,), 55, dtype=torch.int8, device="cuda")
    scale = torch.zeros(M, device="cuda")
    pg.i8_quantize_rows(M, K, store.cuda()[shift:], ldx, Q[shift:], ldq, scale)
    torch.cuda.synchronize()
    got = Q.cpu()[shift:].view(M, ldq)
    want, ws = quantize_want(torch, X)
    assert torch.equal(scale.cpu(), ws)
    assert torch.equal(got[:, :K], want), (got[:, :K] != want).sum()
    assert (got[:, K:] == 55).all() and (Q[:shift] == 55).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [
    (1, 1), (3, 0), (5, 3), (4, 4), (7, 9), (2, 255), (9, 256), (3, 257), (6, 1000), (1, 2048),
    (5, 2049), (3, 4092), (4, 4096), (2, 8190), (2, 16384), (1, 32769), (2, 65537), (1, 100001),
    (300, 64), (1000, 40)])
def test_quantize(env, M, K, dtype):
    torch, _ = env
    g = torch.Generator().manual_seed(M * 100003 + K)
    X = torch.randn(M, K, generator=g) * torch.exp(3 * torch.randn(M, 1, generator=g))
    quantize_case(env, X.to(getattr(torch, dtype)))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_strides(env, dtype):
    torch, _ = env
    g = torch.Generator().manual_seed(1)
    for M, K, ldx, ldq, shift in ((5, 64, 65, 67, 1), (4, 1001, 1003, 1001, 3), (3, 256, 256, 272, 0)):
        quantize_case(env, torch.randn(M, K, generator=g).to(getattr(torch, dtype)), ldx, ldq,
                      shift)


def test_quantize_borders(env):
    """Values on and one last place beside the borders between integers, where
    a rounded quotient would go wrong; ties go to the even integer."""
    torch, _ = env
    g = torch.Generator().manual_seed(2)
    X = torch.empty(64, 768)
    for m in range(64):
        peak = torch.rand(1, generator=g) * 2.0 ** (m - 32) + 2.0 ** (m - 34)
        s = (peak.double() / 127).float()
        k = torch.arange(256).double() - 127.5
        mid = (k.clamp(-126.5, 126.5) * s.double()).float()
        X[m] = torch.cat([mid, torch.nextafter(mid, torch.tensor(torch.inf)),
                          torch.nextafter(mid, torch.tensor(-torch.inf))])
        X[m, 0] = peak
    quantize_case(env, X)
    # a scale of exactly 1: the borders are ties
    T = torch.arange(-127, 127).float() + 0.5
    T = torch.cat([T, torch.tensor([127.0])])[None]
    quantize_case(env, T)


def test_quantize_smallest_and_largest(env):
    torch, _ = env
    tiny = 2.0 ** -149
    X = torch.tensor([[0.0, -0.0, 0.0], [tiny, -tiny, 0.0], [2.0 ** -126, -2.0 ** -127, tiny],
                      [1.5 * 2.0 ** -127, 2.0 ** -127, -3 * 2.0 ** -128],
                      [127 * 2.0 ** -126, 63.5 * 2.0 ** -126, -tiny],
                      [3.4028235e38, -1.7e38, 1e30], [-3.4028235e38, 3.4028235e38, 1.0]])
    quantize_case(env, X)


def test_quantize_infinity_and_nan(env):
    """A row with an infinity or NaN: the scale says so and Q is 0; other rows
    are as ever."""
    torch, pg = env
    for dtype in TYPES:
        X = torch.ones(5, 70, dtype=getattr(torch, dtype))
        X[1, 3], X[2, 69], X[3, 0], X[3, 1] = torch.inf, torch.nan, -torch.inf, torch.nan
        Q = torch.full((5, 70), 9, dtype=torch.int8, device="cuda")
        scale = torch.zeros(5, device="cuda")
        pg.i8_quantize_rows(5, 70, X.cuda(), 70, Q, 70, scale)
        s, q = scale.cpu(), Q.cpu()
        assert s[1] == torch.inf and s[2].isnan() and s[3].isnan()
        assert (q[1:4] == 0).all() and (q[0] == 127).all() and (q[4] == 127).all()


def test_quantize_many_rows(env):
    """More rows than one launch holds of the wave-a-row form would index
    wrongly with 32-bit products of rows and their length."""
    torch, pg = env
    M, K = (1 << 23) + 5, 300
    X = torch.zeros(M, K, dtype=torch.float16, device="cuda")
    X[-1, -1] = 2.0
    X[1 << 23, 7] = -1.0
    Q = torch.empty(M, K, dtype=torch.int8, device="cuda")
    scale = torch.empty(M, device="cuda")
    pg.i8_quantize_rows(M, K, X, K, Q, K, scale)
    assert Q[-1, -1].item() == 127 and Q[1 << 23, 7].item() == -127
    assert int(torch.count_nonzero(Q)) == 2
    assert scale[-1].item() == np.float32(2.0) / np.float32(127.0)


# --- streams and graphs ---------------------------------------------------------------------


def test_other_stream_and_graph(env):
    """Quantization and products on a side stream, captured and replayed with
    new inputs and eager work in between."""
    torch, pg = env
    M, N, K, G = 70, 96, 128, 3
    X = torch.randn(M, K, device="cuda")
    B = torch.randint(-127, 128, (G, N, K), dtype=torch.int8, device="cuda")
    sB = torch.rand(G, N, device="cuda")
    off = torch.tensor([0, 30, 31, 70], dtype=torch.int32, device="cuda")

    def buffers():
        return (torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"),
                torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda"))

    def work(Q, s, C, D, stream=None):
        pg.i8_quantize_rows(M, K, X, K, Q, K, s, stream=stream)
        pg.i8gemm(M, N, K, Q, K, s, B, K, sB, None, C, N, stream=stream)
        pg.i8gemm_grouped(M, N, K, G, off, Q, K, s, B, K, N * K, sB, None, D, N, stream=stream)

    side = torch.cuda.Stream()
    eager, other, captured = buffers(), buffers(), buffers()
    work(*eager)
    side.wait_stream(torch.cuda.current_stream())
    work(*other, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        work(*captured)
    for rep in range(4):
        X.copy_(torch.randn(M, K, device="cuda") * (rep + 1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        work(*eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, captured)), rep


@pytest.mark.parametrize("M,N", [(1, 40), (16, 70), (20, 64), (60, 2000), (500, 300)])
def test_products_without_k(env, M, N):
    """K = 0: the bias, or 0; A and B are not read."""
    product_case(env, M, N, 0, "bfloat16", bias=True)
    product_case(env, M, N, 0, "float32", counts=[M - 1, 0, 1], bias=True)
    torch, pg = env
    s, c = torch.ones(M + N, device="cuda"), torch.full((M, N), 3.0, device="cuda")
    e = torch.empty(0, dtype=torch.int8, device="cuda")
    pg.i8gemm(M, N, 0, e, 1, s, e, 1, s, None, c, N)
    assert (c == 0).all()


@pytest.mark.parametrize("K", list(range(1, 50)) + [63, 65, 79, 81, 127, 129, 143, 145])
def test_row_ends(env, K):
    """Rows that end anywhere in a 16-byte chunk, with other bytes behind them
    and at every alignment, through each kernel that takes them."""
    for M, N in ((1, 33), (40, 40), (70, 150)):
        product_case(env, M, N, K, "float32", lda=K + K % 7, ldb=K + 3, shift=K % 16)
    product_case(env, 2000, 2100, K, "bfloat16", lda=K + 1, ldb=K + 2, shift=5)


# --- large products: every tile of the dispatch, against 64-bit products on the GPU -------------


def large_case(env, M, N, K, dtype, counts=None, first=0, extra=0, bias=True, ldc_pad=0):
    torch, pg = env
    log(f"[i8gemm large] {M}x{N}x{K} {dtype} counts={counts}")
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    dt, G = getattr(torch, dtype), 1 if counts is None else len(counts)
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda",  # noqa: E731
                                  dtype=torch.int8)
    A, B = i8(M, K), i8(G, N, K)
    sA = torch.rand(M, generator=g, device="cuda") / 64
    sB = torch.rand(G, N, generator=g, device="cuda") / 64
    bs = torch.randn(G, N, generator=g, device="cuda") if bias else None
    ldc = N + ldc_pad
    C = torch.full((M, ldc), 7.0, dtype=dt, device="cuda")
    if counts is None:
        pg.i8gemm(M, N, K, A, K, sA, B, K, sB, bs, C, ldc)
        ends = [0, M]
    else:
        ends = [int(e) for e in np.concatenate([[0], np.cumsum(counts)]) + first]
        off = torch.tensor(ends, dtype=torch.int32, device="cuda")
        pg.i8gemm_grouped(M, N, K, G, off, A, K, sA, B, K, N * K, sB, bs, C, ldc)
    for e in range(G):
        lo, hi = ends[e], ends[e + 1]
        p = (A[lo:hi].double() @ B[e].double().t().contiguous()) * sA[lo:hi, None].double() * \
            sB[e].double()
        b = bs[e].double().expand_as(p) if bias else torch.zeros_like(p)
        err = (C[lo:hi, :N].double() - p - b).abs()
        assert (err <= tolerance(torch, dt, p, b)).all(), (e, err.max().item())
    assert (C[:, N:] == 7).all() and (C[:ends[0]] == 7).all() and (C[ends[-1]:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [
    (200, 2048, 1024), (250, 4093, 272), (5000, 512, 512), (500, 4096, 2048), (1001, 4090, 2064),
    (2000, 4095, 2032), (4000, 4090, 2064), (4001, 8192, 144), (700, 16384, 1008),
    (33, 16384, 528), (16, 16400, 272), (3, 5000, 4112), (1, 4100, 4096), (64, 4096, 1040)])
def test_product_large(env, M, N, K, dtype):
    large_case(env, M, N, K, dtype, bias=M % 2 == 0, ldc_pad=M % 3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,N,K", [
    ([1990, 0, 2010], 3800, 2064), ([300] * 16, 2048, 528), ([129, 7, 0, 255, 256, 257, 1] * 4, 2050, 1040),
    ([16] * 50 + [0] * 14, 2048, 512), ([2, 9, 0, 31, 1] * 20, 1030, 272), ([1] * 300, 520, 144)])
def test_grouped_large(env, counts, N, K, dtype):
    large_case(env, sum(counts) + 9, N, K, dtype, counts=counts, first=4, bias=len(counts) % 2 == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K,counts", [
    (4001, 8192, 656, None), (8000, 8190, 1024, None), (4100, 16000, 784, None),
    (0, 8192, 656, [3000, 1, 0, 2000, 255, 257, 500]), (0, 8190, 1040, [256, 512, 1024, 3000, 129]),
    (0, 4096, 2048, [500] * 16 + [1] * 16)])
def test_more_tiles_than_compute_units(env, M, N, K, counts, dtype):
    """Several rounds of 256 x 256 tiles: whole ones, ragged ones, and tiles
    whose lower waves have no rows."""
    large_case(env, M or sum(counts) + 9, N, K, dtype, counts=counts, first=4 if counts else 0,
               bias=N % 4 == 2)


def test_large_products_repeat(env):
    """The same call again and again gives the same bits, with other work on
    the memory in between."""
    torch, pg = env
    M, N, K = 4001, 8192, 1040
    A = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda")
    B = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda")
    sA, sB = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    C = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pg.i8gemm(M, N, K, A, K, sA, B, K, sB, None, C[0], N)
    for _ in range(20):
        C[1].fill_(1.0)
        pg.i8gemm(M, N, K, A, K, sA, B, K, sB, None, C[1], N)
        assert torch.equal(C[0], C[1])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_borders_of_the_smallest_scales(env, dtype):
    """The same for scales from 2^-126 to 2^-124, of which half is not always a
    number: a tie is told from the values beside it all the same."""
    torch, _ = env
    g = torch.Generator().manual_seed(3)
    X = torch.empty(256, 768)
    for m in range(256):
        peak = (127 * (1 + 3 * torch.rand(1, generator=g).double()) * 2.0 ** -126).float()
        s = (peak.double() / 127).float()
        k = torch.arange(256).double() - 127.5
        mid = (k.clamp(-126.5, 126.5) * s.double()).float()
        X[m] = torch.cat([mid, torch.nextafter(mid, torch.tensor(torch.inf)),
                          torch.nextafter(mid, torch.tensor(-torch.inf))])
        X[m, 0] = peak
    quantize_case(env, X.to(getattr(torch, dtype)))


def test_rows_that_only_the_largest_tiles_hold(env):
    """2^30 rows: 2^31 work-items in 256 x 256 tiles, more than a launch holds
    in any other."""
    torch, pg = env
    M, K = 1 << 30, 16
    log(f"[i8gemm] {M}x1x{K}")
    A = torch.empty(M, K, dtype=torch.int8, device="cuda")
    A.view(-1).view(torch.int64).random_(generator=torch.Generator(device="cuda").manual_seed(1))
    B = torch.tensor([[1, -2, 3, -4, 5, -6, 7, -8, 9, 10, -11, 12, 13, 14, -15, 127]],
                     dtype=torch.int8, device="cuda")
    one = torch.ones(M, device="cuda")
    C = torch.full((M + 1,), 7.0, device="cuda")
    pg.i8gemm(M, 1, K, A, K, one, B, K, one, None, C, 1)
    torch.cuda.synchronize()
    for lo in range(0, M, 1 << 26):
        a = A[lo:lo + (1 << 26)]
        want = torch.zeros(a.shape[0], device="cuda")
        for k in range(K):  # whole numbers below 2^24
            want += a[:, k].float() * float(B[0, k])
        assert torch.equal(C[lo:lo + (1 << 26)], want), lo
    assert C[M].item() == 7


def test_groups_that_only_larger_tiles_hold(env):
    """Few rows a group would stream, in more tiles than a launch holds."""
    torch, pg = env
    G, M, N, K = 1024, 8192, 350000, 16
    log(f"[i8gemm grouped] {M}x{N}x{K} groups={G}")
    g = torch.Generator(device="cuda").manual_seed(2)
    A = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    cut = torch.randint(0, M + 1, (G - 1,), generator=g, device="cuda").sort().values
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), M)]).int()
    sA = 2.0 ** torch.randint(-3, 4, (M,), generator=g, device="cuda").float()
    sB = 2.0 ** torch.randint(-3, 4, (G, N), generator=g, device="cuda").float()
    C = torch.full((M, N), 7.0, dtype=torch.float32, device="cuda")
    pg.i8gemm_grouped(M, N, K, G, off, A, K, sA, B, K, 0, sB, None, C, N)
    torch.cuda.synchronize()
    group = torch.repeat_interleave(torch.arange(G, device="cuda"), off.diff().long())
    b = B.float().t().contiguous()
    for lo in range(0, M, 512):  # sums below 2^24, scales powers of two: exact
        rows = slice(lo, lo + 512)
        want = torch.zeros(512, N, device="cuda")
        for k in range(K):
            want += A[rows, k, None].float() * b[k]
        want *= sA[rows, None]
        want *= sB[group[rows]]
        assert torch.equal(C[rows], want), lo
