"""Tokens sorted by expert and back, their gradients, the grouped fp32 products
and a layer made of them, against 64-bit values.

Tolerances count roundings: 2^-24 of the value for each fp32 operation, half a
step of the type for the last rounding."""
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


def half_step(torch, dtype, size):
    """Half a step of dtype at numbers up to `size`, or of its smallest ones."""
    f = torch.finfo(dtype)
    return size * f.eps / 2 + f.smallest_normal * f.eps / 2


def sort_want(ids, experts):
    flat = np.asarray(ids).reshape(-1)
    held = np.flatnonzero((flat >= 0) & (flat < experts))
    order = held[np.argsort(flat[held], kind="stable")]
    row = np.full(flat.size, -1, np.int32)
    row[order] = np.arange(order.size, dtype=np.int32)
    offsets = np.zeros(experts + 1, np.int32)
    offsets[1:] = np.cumsum(np.bincount(flat[held].astype(np.int64), minlength=experts))
    return offsets, row


def run_sort(env, ids, experts):
    torch, pg = env
    tokens, topk = ids.shape
    d = torch.from_numpy(np.ascontiguousarray(ids)).cuda()
    offsets = torch.full((experts + 3,), -7, dtype=torch.int32, device="cuda")
    row = torch.full((tokens * topk + 2,), -9, dtype=torch.int32, device="cuda")
    need = pg.expert_sort_workspace_size(tokens, topk, experts)
    ws = torch.full((need + 64,), 0x5a, dtype=torch.uint8, device="cuda")
    log(f"[sort] tokens={tokens} topk={topk} experts={experts} {ids.dtype} ws={need}")
    pg.expert_sort(tokens, topk, experts, d, offsets, row, ws[:need] if need else None)
    torch.cuda.synchronize()
    assert offsets[experts + 1:].tolist() == [-7, -7] and row[tokens * topk:].tolist() == [-9, -9]
    assert (ws[need:] == 0x5a).all()
    return offsets[:experts + 1].cpu().numpy(), row[:tokens * topk].cpu().numpy()


@pytest.mark.parametrize("idtype", [np.int32, np.int64])
@pytest.mark.parametrize("tokens,topk,experts", [
    (0, 2, 5), (1, 1, 1), (1, 8, 8), (3, 2, 1024), (63, 1, 4), (64, 1, 2), (65, 3, 7), (500, 2, 8),
    (511, 4, 64), (1024, 2, 128), (1025, 2, 127), (4097, 1, 1000), (5000, 8, 256), (20000, 6, 1024),
    (70001, 8, 60), (300000, 4, 16)])
def test_sort(env, tokens, topk, experts, idtype):
    rng = np.random.default_rng(tokens + topk)
    ids = rng.integers(0, experts, (tokens, topk)).astype(idtype)
    for got, want in zip(run_sort(env, ids, experts), sort_want(ids, experts)):
        assert np.array_equal(got, want)


@pytest.mark.parametrize("tokens", [7, 3000, 90000])
def test_sort_skewed_and_absent(env, tokens):
    """One expert for all, ids outside the range, no id inside it."""
    rng = np.random.default_rng(tokens)
    E = 33
    one = np.full((tokens, 3), 17, np.int32)
    some = rng.integers(-3, E + 4, (tokens, 3)).astype(np.int64)
    some[rng.random(some.shape) < 0.3] = -1
    some[0, 0], some[-1, -1] = 2**31 + 5, -2**40 + 2
    none = np.full((tokens, 3), -1, np.int32)
    last = np.full((tokens, 3), E - 1, np.int32)
    for ids in (one, some, none, last, np.full((tokens, 3), E, np.int32),
                np.full((tokens, 3), np.iinfo(np.int32).min, np.int32)):
        for got, want in zip(run_sort(env, ids, E), sort_want(ids, E)):
            assert np.array_equal(got, want)


class Rows:
    """rows x cols at stride ld, `shift` elements into its storage, with NaN
    everywhere else; `host` in 64 bits."""

    def __init__(self, torch, dtype, rows, cols, g, pad=0, shift=0, fill=None):
        self.ld, self.rows, self.cols, self.shift = max(1, cols + pad), rows, cols, shift
        n = shift + rows * self.ld
        if dtype == torch.int8:
            store = torch.full((n,), 77, dtype=dtype)
            values = torch.randint(-128, 128, (rows, cols), generator=g, dtype=torch.int8)
        else:
            store = torch.full((n,), torch.nan, dtype=dtype)
            values = torch.randn(rows, cols, generator=g).to(dtype)
        if fill is not None:
            values = torch.full((rows, cols), fill, dtype=dtype)
        store[shift:].view(rows, self.ld)[:, :cols] = values
        self.before = store.clone()
        self.values = values
        self.host = values.double()
        self.full = store.cuda()
        self.t = self.full[shift:]

    def now(self):
        return self.full.cpu()[self.shift:].view(self.rows, self.ld)[:, :self.cols]

    def untouched(self, torch, mask=None):
        """Everything but the values (and the rows that `mask` leaves out) is
        as it was, bit for bit."""
        a, b = self.full.cpu().clone(), self.before.clone()
        for x in (a, b):
            v = x[self.shift:].view(self.rows, self.ld)[:, :self.cols]
            if mask is None:
                v.zero_()
            else:
                v[~mask] = 0
        size = a.element_size()
        view = {1: torch.int8, 2: torch.int16, 4: torch.int32}[size]
        return torch.equal(a.view(view), b.view(view))


def routing(torch, tokens, topk, experts, seed, absent=0.2):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts, (tokens, topk))
    ids[rng.random(ids.shape) < absent] = -1
    if tokens > 2:
        ids[tokens // 2] = -1  # a token without any expert
    _, row = sort_want(ids, experts)
    rows = torch.from_numpy(row).view(tokens, topk)
    return rows, rows.cuda()


SHAPES = [(1, 1, 1, 1), (1, 8, 2048, 16), (5, 2, 3, 4), (9, 3, 8, 3), (33, 2, 20, 8),
          (17, 9, 100, 12), (64, 4, 257, 5), (7, 20, 1000, 30), (100, 1, 4099, 6), (40, 6, 512, 64),
          (3, 2, 10007, 4), (260, 2, 16, 7)]


@pytest.mark.parametrize("dtype", TYPES + ["int8"])
@pytest.mark.parametrize("tokens,topk,cols,experts", SHAPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 3)])
def test_gather(env, tokens, topk, cols, experts, dtype, pad, shift):
    torch, pg = env
    dt, g = getattr(torch, dtype), torch.Generator().manual_seed(cols)
    rows, d_rows = routing(torch, tokens, topk, experts, cols)
    log(f"[gather] {tokens}x{topk}x{cols} {dtype} pad={pad} shift={shift}")
    X = Rows(torch, dt, tokens, cols, g, pad, shift)
    Y = Rows(torch, dt, tokens * topk, cols, g, 2 * pad, shift)
    pg.expert_gather(tokens, topk, cols, X.t, X.ld, d_rows, Y.t, Y.ld)
    torch.cuda.synchronize()
    written = torch.zeros(tokens * topk, dtype=torch.bool)
    held = rows >= 0
    written[rows[held].long()] = True
    want = Y.values.clone()
    want[rows[held].long()] = X.values[held.nonzero()[:, 0]]
    assert torch.equal(Y.now(), want)
    assert Y.untouched(torch, ~written)


def combine_want(torch, Y, rows, weights, tokens, cols):
    """The sum and the sum of magnitudes, in 64 bits."""
    out = torch.zeros(tokens, cols, dtype=torch.float64)
    size = torch.zeros(tokens, cols, dtype=torch.float64)
    for j in range(rows.shape[1]):
        has = rows[:, j] >= 0
        term = weights[has, j, None].double() * Y[rows[has, j].long()]
        out[has] += term
        size[has] += term.abs()
    return out, size


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,topk,cols,experts", SHAPES)
@pytest.mark.parametrize("pad,shift,weighted", [(0, 0, True), (5, 3, True), (3, 0, False)])
def test_combine(env, tokens, topk, cols, experts, dtype, pad, shift, weighted):
    torch, pg = env
    dt, g = getattr(torch, dtype), torch.Generator().manual_seed(cols + 1)
    rows, d_rows = routing(torch, tokens, topk, experts, cols + 1)
    log(f"[combine] {tokens}x{topk}x{cols} {dtype} pad={pad} shift={shift} weighted={weighted}")
    Y = Rows(torch, dt, tokens * topk, cols, g, pad, shift)
    used = torch.zeros(tokens * topk, dtype=torch.bool)
    used[rows[rows >= 0].long()] = True
    Y.t.view(-1)[:tokens * topk * Y.ld].view(-1, Y.ld)[(~used).cuda()] = torch.nan  # never read
    w = torch.randn(tokens, topk, generator=g)
    out = Rows(torch, dt, tokens, cols, g, 2 * pad, shift)
    pg.expert_combine(tokens, topk, cols, Y.t, Y.ld, d_rows, w.cuda() if weighted else None,
                      out.t, out.ld)
    torch.cuda.synchronize()
    want, size = combine_want(torch, Y.host, rows, w if weighted else torch.ones_like(w), tokens,
                              cols)
    # topk fused steps of at most one rounding of a partial sum each
    fp32 = 1.01 * topk * 2.0 ** -24 * size
    tol = fp32 + half_step(torch, dt, want.abs() + fp32)
    assert ((out.now().double() - want).abs() <= tol).all()
    assert out.untouched(torch)
    assert (out.now()[(rows < 0).all(1)] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,topk,cols,experts", SHAPES)
@pytest.mark.parametrize("pad,shift,weighted", [(0, 0, True), (5, 3, True), (3, 0, False)])
def test_combine_grad(env, tokens, topk, cols, experts, dtype, pad, shift, weighted):
    torch, pg = env
    dt, g = getattr(torch, dtype), torch.Generator().manual_seed(cols + 2)
    rows, d_rows = routing(torch, tokens, topk, experts, cols + 2)
    log(f"[combine_grad] {tokens}x{topk}x{cols} {dtype} pad={pad} shift={shift}")
    slots = tokens * topk
    dout = Rows(torch, dt, tokens, cols, g, pad, shift)
    Y = Rows(torch, dt, slots, cols, g, pad, shift)
    dY = Rows(torch, dt, slots, cols, g, 2 * pad, shift)
    dY2 = Rows(torch, dt, slots, cols, g, 2 * pad, shift)
    w = torch.randn(tokens, topk, generator=g)
    used = torch.zeros(slots, dtype=torch.bool)
    used[rows[rows >= 0].long()] = True
    Y.t[:slots * Y.ld].view(-1, Y.ld)[(~used).cuda()] = torch.nan
    dw = torch.full((slots + 3,), 5.0, device="cuda")
    d_w = w.cuda() if weighted else None
    pg.expert_combine_grad(tokens, topk, cols, dout.t, dout.ld, Y.t, Y.ld, d_rows, d_w, dY.t,
                           dY.ld, dw)
    pg.expert_combine_grad(tokens, topk, cols, dout.t, dout.ld, None, 0, d_rows, d_w, dY2.t,
                           dY2.ld, None)
    torch.cuda.synchronize()
    ww = w if weighted else torch.ones_like(w)
    want_dY = torch.zeros(slots, cols, dtype=torch.float64)
    want_dw = torch.zeros(tokens, topk, dtype=torch.float64)
    size_dw = torch.zeros(tokens, topk, dtype=torch.float64)
    for j in range(topk):
        has = rows[:, j] >= 0
        r = rows[has, j].long()
        want_dY[r] = ww[has, j, None].double() * dout.host[has]
        prod = dout.host[has] * Y.host[r]
        want_dw[has, j], size_dw[has, j] = prod.sum(1), prod.abs().sum(1)
    # dY: the fp32 product, then the type
    fp32 = 2.0 ** -24 * want_dY.abs() + 2.0 ** -150
    tol = fp32 + half_step(torch, dt, want_dY.abs() + fp32)
    for d in (dY, dY2):
        err = (d.now().double() - want_dY).abs()
        assert (err[used] <= tol[used]).all()
        assert d.untouched(torch, ~used)
    # dweights: cols fused steps and the sum over the lanes, in any order
    err = (dw[:slots].cpu().view(tokens, topk).double() - want_dw).abs()
    assert (err <= 1.01 * cols * 2.0 ** -24 * size_dw).all()
    assert (dw[:slots].cpu().view(tokens, topk)[rows < 0] == 0).all()
    assert dw[slots:].tolist() == [5.0] * 3


def test_gradients_against_differences(env):
    """<dout, combine(gather(X))> moves as the gradients say, in fp32 (the
    function is linear in X and in the weights, so a step of any size will do
    and only roundings are left)."""
    torch, pg = env
    T, k, H, E = 40, 3, 70, 9
    rows, d_rows = routing(torch, T, k, E, 5)
    g = torch.Generator().manual_seed(6)
    X, w, dout = (torch.randn(*s, generator=g).cuda() for s in ((T, H), (T, k), (T, H)))
    dX, dw = torch.randn(T, H, generator=g).cuda(), torch.randn(T, k, generator=g).cuda()

    def forward(x, weights):
        y = torch.zeros(T * k, H, device="cuda")
        pg.expert_gather(T, k, H, x, H, d_rows, y, H)
        out = torch.empty(T, H, device="cuda")
        pg.expert_combine(T, k, H, y, H, d_rows, weights, out, H)
        return y, out

    y, out = forward(X, w)
    dY, gw = torch.zeros(T * k, H, device="cuda"), torch.empty(T, k, device="cuda")
    pg.expert_combine_grad(T, k, H, dout, H, y, H, d_rows, w, dY, H, gw)
    gX = torch.empty(T, H, device="cuda")
    pg.expert_combine(T, k, H, dY, H, d_rows, None, gX, H)
    dot = lambda a, b: float((a.double() * b.double()).sum())  # noqa: E731
    size = float((dout.abs().double() * 9).sum()) * k
    assert abs(dot(dout, forward(X + dX, w)[1] - out) - dot(gX, dX)) <= 1e-5 * size
    assert abs(dot(dout, forward(X, w + dw)[1] - out) - dot(gw, dw)) <= 1e-5 * size


def test_nan_stays_in_its_token(env):
    """A NaN in one token's expert rows reaches that token only; one in a row
    that no slot names reaches none; a weight of 0 does not hide it."""
    torch, pg = env
    rows = torch.tensor([[0, 2], [1, -1], [3, 4]], dtype=torch.int32, device="cuda")
    Y = torch.ones(6, 33, device="cuda")
    Y[2, 5], Y[5] = torch.nan, torch.nan
    w = torch.tensor([[1.0, 0.0], [2.0, torch.nan], [0.5, 0.5]], device="cuda")
    out = torch.empty(3, 33, device="cuda")
    pg.expert_combine(3, 2, 33, Y, 33, rows, w, out, 33)
    assert out[0].isnan().nonzero().flatten().tolist() == [5]
    assert (out[1] == 2).all() and (out[2] == 1).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,topk,cols", [(300, 4, 2047), (50, 3, 1030), (2000, 2, 9),
                                              (20, 16, 515), (6, 64, 130), (33, 1, 2049)])
def test_rows_that_end_anywhere(env, tokens, topk, cols, dtype):
    """Rows whose last 16 bytes overlap the chunk before them: every element
    counted once, from unaligned rows too."""
    for pad, shift in ((0, 0), (1, 1), (2, 5)):
        test_gather(env, tokens, topk, cols, 11, dtype, pad, shift)
        test_combine(env, tokens, topk, cols, 11, dtype, pad, shift, True)
        test_combine_grad(env, tokens, topk, cols, 11, dtype, pad, shift, True)


def test_rows_outside_the_range_count_as_absent(env):
    torch, pg = env
    rows = torch.tensor([[0, 4], [2**31 - 1, 1]], dtype=torch.int32, device="cuda")
    X = torch.ones(2, 8, device="cuda")
    Y = torch.zeros(4, 8, device="cuda")
    pg.expert_gather(2, 2, 8, X, 8, rows, Y, 8)
    assert Y[:, 0].tolist() == [1, 1, 0, 0]
    out = torch.empty(2, 8, device="cuda")
    pg.expert_combine(2, 2, 8, Y, 8, rows, None, out, 8)
    assert out[:, 0].tolist() == [1, 1]
    dw = torch.full((2, 2), 3.0, device="cuda")
    pg.expert_combine_grad(2, 2, 8, X, 8, Y, 8, rows, None, torch.empty(4, 8, device="cuda"), 8, dw)
    assert dw.tolist() == [[8, 0], [0, 8]]


def test_rows_past_32_bits(env):
    """Sorted rows beyond 2^32 bytes."""
    torch, pg = env
    T, k, H = 3, 2, 24
    ld = 2**30 - 3
    rows = torch.tensor([[4, 0], [5, -1], [1, 2]], dtype=torch.int32, device="cuda")
    X = torch.randn(T, H, device="cuda").bfloat16()
    Y = torch.empty(5 * ld + H, dtype=torch.bfloat16, device="cuda")
    pg.expert_gather(T, k, H, X, H, rows, Y, ld)
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    pg.expert_combine(T, k, H, Y, ld, rows, None, out, H)
    for t, j in ((0, 0), (1, 0), (2, 1)):
        r = int(rows[t, j])
        assert torch.equal(Y[r * ld:r * ld + H], X[t])
    assert torch.equal(out[0], (2 * X[0].float()).bfloat16()) and torch.equal(out[1], X[1])
    dY = torch.empty(5 * ld + H, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(T, k, device="cuda")
    pg.expert_combine_grad(T, k, H, out, H, Y, ld, rows, None, dY, ld, dw)
    assert torch.equal(dY[5 * ld:5 * ld + H], out[1])
    assert dw[1, 1].item() == 0 and dw[1, 0].item() > 0


# --- grouped products -----------------------------------------------------------------------


def ends_of(counts, first):
    return (np.concatenate([[0], np.cumsum(counts)]) + first).astype(np.int32)


def grouped_case(env, tB, counts, N, K, first=0, extra=0, alpha=1.0, beta=0.0, pad=0, shift=0,
                 integers=True):
    """integers: small whole numbers, whose sums are exact in fp32."""
    torch, pg = env
    M, G = first + sum(counts) + extra, len(counts)
    log(f"[grouped] tB={tB} counts={counts} N={N} K={K} first={first} alpha={alpha} beta={beta} "
        f"pad={pad} shift={shift}")
    rng = np.random.default_rng(N * 31 + K)

    def make(rows, cols, groups=1):
        ld = max(1, cols + pad)
        n = shift + groups * rows * ld
        v = rng.integers(-4, 5, n) if integers else rng.uniform(-1, 1, n)
        t = torch.from_numpy(v.astype(np.float32)).cuda()[shift:]
        return t, ld, t.cpu().view(groups, rows, ld)[:, :, :cols].double()

    A, lda, hA = make(M, K)
    B, ldb, hB = make(N if tB else K, K if tB else N, G)
    C, ldc, hC = make(M, N)
    before = C.cpu().clone()
    ends = ends_of(counts, first)
    pg.sgemm_grouped(tB, M, N, K, G, torch.from_numpy(ends).cuda(), alpha, A, lda, B, ldb,
                     (N if tB else K) * ldb, beta, C, ldc)
    torch.cuda.synchronize()
    got, was = C.cpu().view(M, ldc), before.view(M, ldc)
    touched = torch.zeros(M, dtype=torch.bool)
    for g in range(G):
        lo, hi = int(ends[g]), int(ends[g + 1])
        b = hB[g].T if tB else hB[g]
        want = alpha * (hA[0, lo:hi] @ b) + (beta * hC[0, lo:hi] if beta else 0)
        err = (got[lo:hi, :N].double() - want).abs()
        if integers:
            assert (err == 0).all(), (g, err.max().item())
        else:
            S = abs(alpha) * (hA[0, lo:hi].abs() @ b.abs()) + abs(beta) * hC[0, lo:hi].abs()
            assert (err <= 2e-6 * max(K, 1) * S).all()
        touched[lo:hi] = True
    assert torch.equal(got[~touched], was[~touched]) and torch.equal(got[:, N:], was[:, N:])


COUNTS = [([1], 0, 0), ([0, 0, 3], 0, 0), ([5, 0, 17, 1, 0], 2, 3), ([64, 64], 0, 5),
          ([65, 1, 130, 0, 7], 3, 4), ([0, 0], 0, 6), ([1] * 70, 0, 0), ([300, 2, 0, 129], 1, 1),
          ([3, 0, 1, 2] * 40, 0, 3), ([600, 700], 0, 0)]


@pytest.mark.parametrize("tB", [0, 1])
@pytest.mark.parametrize("counts,first,extra", COUNTS)
@pytest.mark.parametrize("N,K", [(64, 64), (132, 96), (20, 260), (77, 45), (1, 1), (200, 16)])
def test_sgemm_grouped(env, tB, counts, first, extra, N, K):
    grouped_case(env, tB, counts, N, K, first, extra, alpha=-2.0 if N == 132 else 1.0,
                 beta=0.5 if K == 260 else 0.0)


@pytest.mark.parametrize("tB", [0, 1])
def test_sgemm_grouped_strides_and_floats(env, tB):
    for pad, shift in ((4, 0), (4, 4), (3, 0), (0, 1), (8, 3)):
        grouped_case(env, tB, [30, 0, 100, 5], 68, 44, pad=pad, shift=shift, beta=2.0)
        grouped_case(env, tB, [30, 0, 100, 5], 68, 44, pad=pad, shift=shift, integers=False,
                     alpha=0.7, beta=-0.3)
    grouped_case(env, tB, [100, 140], 256, 2048, integers=False)
    grouped_case(env, tB, [9, 0, 2], 260, 4096, integers=False)


@pytest.mark.parametrize("K,alpha,beta", [(0, 1.0, 0.0), (0, 1.0, 0.5), (16, 0.0, 0.0),
                                          (16, 0.0, 2.0), (0, 1.0, 1.0)])
def test_sgemm_grouped_without_product(env, K, alpha, beta):
    grouped_case(env, 0, [30, 0, 100, 5], 68, K, 2, 3, alpha=alpha, beta=beta)


def outer_case(env, counts, M, N, first=0, extra=0, alpha=1.0, beta=0.0, pad=0, shift=0,
               cpad=0, integers=True):
    torch, pg = env
    K, G = first + sum(counts) + extra, len(counts)
    log(f"[outer] counts={counts} M={M} N={N} first={first} alpha={alpha} beta={beta} pad={pad} "
        f"shift={shift}")
    rng = np.random.default_rng(N * 31 + M)

    def make(n):
        v = rng.integers(-4, 5, n) if integers else rng.uniform(-1, 1, n)
        return torch.from_numpy(v.astype(np.float32))

    lda, ldb, ldc = max(1, M + pad), max(1, N + pad), max(1, N + pad)
    A, B = make(shift + K * lda), make(shift + K * ldb)
    C = make(shift + G * (M * ldc + cpad))
    dA, dB, dC = A.cuda()[shift:], B.cuda()[shift:], C.cuda()[shift:]
    ends = ends_of(counts, first)
    # rows that belong to no group are not read
    hA, hB = A[shift:].view(K, lda)[:, :M].double(), B[shift:].view(K, ldb)[:, :N].double()
    out = torch.ones(K, dtype=torch.bool)
    out[int(ends[0]):int(ends[-1])] = False
    dA.view(K, lda)[out.cuda()] = torch.nan
    pg.sgemm_grouped_outer(M, N, K, G, torch.from_numpy(ends).cuda(), alpha, dA, lda, dB, ldb,
                           beta, dC, ldc, M * ldc + cpad)
    torch.cuda.synchronize()
    got = dC.cpu().view(G, M * ldc + cpad)
    was = C[shift:].view(G, M * ldc + cpad)
    for g in range(G):
        lo, hi = int(ends[g]), int(ends[g + 1])
        x, c0 = got[g, :M * ldc].view(M, ldc), was[g, :M * ldc].view(M, ldc)
        want = alpha * (hA[lo:hi].T @ hB[lo:hi]) + (beta * c0[:, :N].double() if beta else 0)
        err = (x[:, :N].double() - want).abs()
        if integers:
            assert (err == 0).all(), (g, err.max().item())
        else:
            S = abs(alpha) * (hA[lo:hi].abs().T @ hB[lo:hi].abs()) + \
                abs(beta) * c0[:, :N].abs().double()
            assert (err <= 2e-6 * max(hi - lo, 1) * S).all()
        assert torch.equal(x[:, N:], c0[:, N:])
    assert torch.equal(got[:, M * ldc:], was[:, M * ldc:])


@pytest.mark.parametrize("counts,first,extra", COUNTS)
@pytest.mark.parametrize("M,N", [(64, 64), (132, 96), (20, 260), (77, 45), (1, 1), (200, 16)])
def test_sgemm_grouped_outer(env, counts, first, extra, M, N):
    outer_case(env, counts, M, N, first, extra, alpha=-2.0 if M == 132 else 1.0,
               beta=0.5 if N == 260 else 0.0)


def test_sgemm_grouped_outer_strides_and_floats(env):
    for pad, shift in ((4, 0), (4, 4), (3, 0), (0, 1), (8, 3)):
        outer_case(env, [30, 0, 100, 5], 68, 44, pad=pad, shift=shift, beta=2.0, cpad=5)
        outer_case(env, [30, 0, 100, 5], 68, 44, pad=pad, shift=shift, integers=False, alpha=0.7,
                   beta=-0.3)
    outer_case(env, [1000, 0, 3000], 256, 192, integers=False)


@pytest.mark.parametrize("alpha,beta", [(0.0, 0.0), (0.0, 2.0), (0.0, 1.0)])
def test_sgemm_grouped_outer_without_product(env, alpha, beta):
    outer_case(env, [3, 0, 7], 40, 20, 1, 2, alpha=alpha, beta=beta)
    outer_case(env, [0, 0], 40, 20, 0, 2, alpha=1.0, beta=beta)


def test_offsets_out_of_range(env):
    """Offsets outside the rows are brought into them, and an end before its
    start makes an empty group: whatever the array holds, other memory is left
    alone."""
    torch, pg = env
    A, B = torch.ones(8, 16, device="cuda"), torch.ones(3, 16, 4, device="cuda")
    B[1], B[2] = 2, 4
    for off, want in (([-5, 2, 6, 100], [1, 1, 2, 2, 2, 2, 4, 4]),
                      ([0, 4, 1, 1], [1, 1, 1, 1, 0, 0, 0, 0]), ([9, 9, 9, 9], [0] * 8),
                      ([2**31 - 1, -2**31, 2**31 - 1, 0], None)):
        store = torch.zeros(10, 4, device="cuda")
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        pg.sgemm_grouped(0, 8, 4, 16, 3, o, 1.0, A, 16, B, 4, 64, 0.0, store[1:], 4)
        if want is not None:
            assert store[1:9, 0].tolist() == [16.0 * w for w in want], off
        assert (store[0] == 0).all() and (store[9] == 0).all()
        C = torch.full((5, 16, 4), 7.0, device="cuda")
        pg.sgemm_grouped_outer(16, 4, 8, 3, o, 1.0, A, 16, torch.ones(8, 4, device="cuda"), 4, 0.0,
                               C[1:], 4, 64)
        if want is not None:
            rows = [want.count(w) for w in (1, 2, 4)]
            assert C[1:4, 0, 0].tolist() == rows, off
        assert (C[0] == 7).all() and (C[4] == 7).all()


@pytest.mark.parametrize("N,K", [(4, 4), (5, 7), (6, 33), (63, 65), (65, 18), (66, 47), (67, 50),
                                 (129, 130), (200, 1001), (191, 259)])
def test_products_of_any_extent(env, N, K):
    """Extents off 4 and 64 in every position, at every 4-byte alignment, and
    nothing read outside the operands (NaN lies around them)."""
    counts = [70, 0, 130, 1, 64]
    for pad, shift in ((0, 0), (1, 1), (2, 3), (5, 2)):
        grouped_case(env, 0, counts, N, K, 1, 2, pad=pad, shift=shift)
        grouped_case(env, 1, counts, N, K, 1, 2, pad=pad, shift=shift, beta=0.5)
        outer_case(env, counts, N, K, 1, 2, pad=pad, shift=shift, alpha=-2.0)


@pytest.mark.parametrize("tB", [0, 1])
def test_nan_around_the_operands(env, tB):
    """What lies beside rows, before the first and behind the last, is NaN."""
    torch, pg = env
    M, N, K, G = 150, 67, 45, 2
    off = torch.tensor([0, 80, 150], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(3)

    def make(groups, rows, cols, lead):
        ld = cols + 3
        store = torch.full((lead + groups * rows * ld,), torch.nan)
        v = torch.randint(-4, 5, (groups, rows, cols), generator=g).float()
        store[lead:].view(groups, rows, ld)[:, :, :cols] = v
        return store.cuda()[lead:], ld, v.double()

    for lead in (0, 1, 6):
        A, lda, hA = make(1, M, K, lead)
        B, ldb, hB = make(G, N if tB else K, K if tB else N, lead)
        D, ldd, hD = make(1, M, N, lead)
        C = torch.full((M, N), torch.nan, device="cuda")
        pg.sgemm_grouped(tB, M, N, K, G, off, 1.0, A, lda, B, ldb, (N if tB else K) * ldb, 0.0, C, N)
        W = torch.full((G, K, N), torch.nan, device="cuda")
        pg.sgemm_grouped_outer(K, N, M, G, off, 1.0, A, lda, D, ldd, 0.0, W, N, K * N)
        for e, (lo, hi) in enumerate(((0, 80), (80, 150))):
            b = hB[e].T if tB else hB[e]
            assert torch.equal(C[lo:hi].cpu().double(), hA[0, lo:hi] @ b)
            assert torch.equal(W[e].cpu().double(), hA[0, lo:hi].T @ hD[0, lo:hi])


@pytest.mark.parametrize("groups", [65, 129, 1000])
def test_many_groups(env, groups):
    """More groups than a wave has lanes: several a lane."""
    rng = np.random.default_rng(groups)
    counts = [int(c) for c in rng.integers(0, 4, groups)]
    grouped_case(env, 0, counts, 36, 24, 1, 2)
    grouped_case(env, 1, counts, 20, 17)
    outer_case(env, counts, 24, 20, 1, 2)
    grouped_case(env, 0, [c * 40 for c in counts[:70]], 64, 32)


def test_sgemm_grouped_large_offsets(env):
    """Rows and weights beyond 2^32 bytes."""
    torch, pg = env
    ld, K, N = (1 << 21) - 1, 20, 12
    M = 1100  # M * ld * 4 bytes > 2^33
    A = torch.empty(M * ld, device="cuda")
    C = torch.empty(M * ld, device="cuda")
    v = A.as_strided((M, K), (ld, 1))
    v.copy_(torch.randint(-4, 5, (M, K), device="cuda").float())
    stride = 1 << 30
    B = torch.empty(2 * stride + 20 * 12, device="cuda")
    for g in range(3):
        B[g * stride:g * stride + 240] = torch.randint(-4, 5, (240,), device="cuda").float()
    off = torch.tensor([0, 400, 500, M], dtype=torch.int32, device="cuda")
    pg.sgemm_grouped(0, M, N, K, 3, off, 1.0, A, ld, B, N, stride, 0.0, C, ld)
    for g, (lo, hi) in enumerate(((0, 400), (400, 500), (500, M))):
        b = B[g * stride:g * stride + 240].view(K, N).double()
        assert torch.equal(C.as_strided((M, N), (ld, 1))[lo:hi].double(), v[lo:hi].double() @ b)


# --- together -------------------------------------------------------------------------------


def test_layer_forward_and_backward(env):
    """A layer of experts, one fp32 product each, from the router's choice to
    the gradients of the tokens, the weights of the sum and the experts."""
    torch, pg = env
    T, k, E, H, F = 150, 2, 6, 40, 52
    rng = np.random.default_rng(8)
    ids = rng.integers(0, E, (T, k))
    ids[:, 1] = (ids[:, 0] + 1 + rng.integers(0, E - 1, T)) % E
    ids[-5:] = -1
    g = torch.Generator().manual_seed(9)
    X, w, W = torch.randn(T, H, generator=g), torch.rand(T, k, generator=g), \
        torch.randn(E, H, F, generator=g)
    dout = torch.randn(T, F, generator=g)

    x64, w64, W64 = (t.double().requires_grad_() for t in (X, w, W))
    parts = []
    for t in range(T):
        s = torch.zeros(F, dtype=torch.float64)
        for j in range(k):
            if ids[t, j] >= 0:
                s = s + w64[t, j] * (x64[t] @ W64[ids[t, j]])
        parts.append(s)
    out64 = torch.stack(parts)
    out64.backward(dout.double())

    cu = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    d = {n: t.cuda() for n, t in (("X", X), ("w", w), ("W", W), ("dout", dout))}
    d_ids = torch.from_numpy(ids).cuda()
    off, row = cu(E + 1).int(), cu(T, k).int()
    xs, y, out = cu(T * k, H), cu(T * k, F), cu(T, F)
    dy, dxs, dX, dw, dW = cu(T * k, F), cu(T * k, H), cu(T, H), cu(T, k), cu(E, H, F)
    S = T * k

    def forward():
        pg.expert_sort(T, k, E, d_ids, off, row, None)
        pg.expert_gather(T, k, H, d["X"], H, row, xs, H)
        pg.sgemm_grouped(0, S, F, H, E, off, 1.0, xs, H, d["W"], F, H * F, 0.0, y, F)
        pg.expert_combine(T, k, F, y, F, row, d["w"], out, F)

    def backward():
        pg.expert_combine_grad(T, k, F, d["dout"], F, y, F, row, d["w"], dy, F, dw)
        pg.sgemm_grouped(1, S, H, F, E, off, 1.0, dy, F, d["W"], F, H * F, 0.0, dxs, H)
        pg.sgemm_grouped_outer(H, F, S, E, off, 1.0, xs, H, dy, F, 0.0, dW, F, H * F)
        pg.expert_combine(T, k, H, dxs, H, row, None, dX, H)

    def check():
        for got, want in ((out, out64), (dX, x64.grad), (dw, w64.grad), (dW, W64.grad)):
            want = want.detach()
            err = (got.cpu().double() - want).abs().max().item()
            # sums of at most T terms of this size, one rounding each, twice over
            assert err <= 2 * T * 2.0 ** -24 * max(1.0, want.abs().max().item()), err

    forward()
    backward()
    torch.cuda.synchronize()
    check()
    first = [t.clone() for t in (out, dX, dw, dW)]

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward()
        backward()
    for rep in range(4):
        for t in (off, row, xs, y, out, dy, dxs, dX, dw, dW):
            t.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (out, dX, dw, dW))), rep
        torch.ones(1000, device="cuda").sum().item()


def test_layer_in_8_bits(env):
    """The serving form: tokens quantized, sorted, multiplied in 8 bits by
    expert and summed, against the same steps in 64 bits."""
    torch, pg = env
    T, k, E, H, F = 90, 3, 10, 128, 96
    g = torch.Generator().manual_seed(11)
    X = torch.randn(T, H, generator=g).bfloat16()
    W = torch.randint(-127, 128, (E, F, H), generator=g, dtype=torch.int8)
    sW = torch.rand(E, F, generator=g) / 64
    score = torch.randn(T, E, generator=g)
    ids = torch.topk(score, k, dim=1).indices
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    S = T * k
    cu = lambda dt, *s: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    q, sx = cu(torch.int8, T, H), cu(torch.float32, T)
    qs, ss = cu(torch.int8, S, H), cu(torch.float32, S)
    off, row = cu(torch.int32, E + 1), cu(torch.int32, T, k)
    y, out = cu(torch.bfloat16, S, F), cu(torch.bfloat16, T, F)
    dW, dsW, dw, dids, dX = W.cuda(), sW.cuda(), w.cuda(), ids.cuda(), X.cuda()

    pg.i8_quantize_rows(T, H, dX, H, q, H, sx)
    pg.expert_sort(T, k, E, dids, off, row, None)
    pg.expert_gather(T, k, H, q, H, row, qs, H)
    pg.expert_gather(T, k, 1, sx, 1, row, ss, 1)
    pg.i8gemm_grouped(S, F, H, E, off, qs, H, ss, dW, H, F * H, dsW, None, y, F)
    pg.expert_combine(T, k, F, y, F, row, dw, out, F)
    torch.cuda.synchronize()

    scale = (X.double().abs().amax(1) / 127).float().double()
    qw = torch.round(X.double() / scale[:, None])
    want = torch.zeros(T, F, dtype=torch.float64)
    tol = torch.zeros(T, F, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            v = (qw[t] @ W[e].double().T) * scale[t] * sW[e].double()
            want[t] += w[t, j].double() * v
            # fp32 roundings of the product, bf16 of y, fp32 of the sum
            tol[t] += w[t, j].double() * v.abs() * ((4.1 + 1.01 * k) * 2.0 ** -24 + 1.01 * 2.0 ** -8)
    tol = tol + (want.abs() + tol) * 2.0 ** -8
    assert ((out.cpu().double() - want).abs() <= tol).all()


def test_two_streams_at_once(env):
    """Sorts with a workspace each and products on two streams do not disturb
    each other."""
    torch, pg = env
    T, k, E, H = 40000, 4, 64, 32
    rng = np.random.default_rng(12)
    jobs = []
    for i in range(2):
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
        jobs.append((sort_want(ids, E), torch.from_numpy(ids).cuda(),
                     torch.zeros(E + 1, dtype=torch.int32, device="cuda"),
                     torch.zeros(T * k, dtype=torch.int32, device="cuda"),
                     torch.zeros(pg.expert_sort_workspace_size(T, k, E), dtype=torch.uint8,
                                 device="cuda"),
                     torch.randn(T, H, device="cuda"), torch.zeros(T * k, H, device="cuda"),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for _, ids, off, row, ws, X, Y, s in jobs:
            pg.expert_sort(T, k, E, ids, off, row, ws, stream=s)
            pg.expert_gather(T, k, H, X, H, row, Y, H, stream=s)
    torch.cuda.synchronize()
    for (offsets, rows), _, off, row, _, X, Y, _ in jobs:
        assert np.array_equal(off.cpu().numpy(), offsets)
        assert np.array_equal(row.cpu().numpy(), rows)
        assert torch.equal(Y[row.long()], X.repeat_interleave(k, 0))


def test_binding_refuses(env):
    torch, pg = env
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    off, row = ids.new_zeros(9), ids.new_zeros(8)
    x, y = torch.zeros(4, 8, device="cuda"), torch.zeros(8, 8, device="cuda")
    with pytest.raises(ValueError, match="offsets holds"):
        pg.expert_sort(4, 2, 9, ids, off, row, None)
    with pytest.raises(ValueError, match="row_of_slot holds"):
        pg.expert_sort(4, 2, 8, ids, off, row[1:], None)
    with pytest.raises(TypeError, match="ids must be"):
        pg.expert_sort(4, 2, 8, ids.short(), off, row, None)
    with pytest.raises(ValueError, match="Y holds"):
        pg.expert_gather(4, 2, 8, x, 8, row, x, 8)
    with pytest.raises(TypeError, match="Y must be"):
        pg.expert_gather(4, 2, 8, x, 8, row, y.half(), 8)
    with pytest.raises(ValueError, match="weights holds"):
        pg.expert_combine(4, 2, 8, y, 8, row, x[3, 1:], x, 8)
    with pytest.raises(pg.SgemmError, match="expert_combine_grad: invalid argument 7"):
        pg.expert_combine_grad(4, 2, 8, x, 8, None, 8, row, None, y, 8, x[0])
    big = torch.zeros(20000, 8, dtype=torch.int32, device="cuda")
    with pytest.raises(pg.SgemmError, match="expert_sort: invalid argument 8"):
        pg.expert_sort(20000, 8, 8, big, off, big, None)
    with pytest.raises(ValueError, match="B holds"):
        pg.sgemm_grouped(0, 4, 8, 8, 2, off, 1.0, x, 8, y, 8, 64, 0.0, x, 8)
    with pytest.raises(ValueError, match="C holds"):
        pg.sgemm_grouped_outer(8, 8, 4, 2, off, 1.0, x, 8, x, 8, 0.0, y, 8, 64)


@pytest.mark.parametrize("M,N,counts", [(1, 1, [5, 0, 70]), (1, 33, [300]), (2, 2, [40, 3]),
                                        (3, 70, [16, 17, 15]), (33, 1, [129]), (47, 31, [0, 64, 0]),
                                        (16, 500, [1000]), (64, 64, [2049]), (65, 130, [33, 31])])
def test_outer_products_of_few_tiles(env, M, N, counts):
    """Tiles smaller than 64 x 64, and rows that end in every part of a block."""
    for pad, shift in ((0, 0), (3, 1)):
        outer_case(env, counts, M, N, 1, 2, pad=pad, shift=shift)
        outer_case(env, counts, M, N, 1, 2, pad=pad, shift=shift, alpha=0.5, beta=-1.0)


@pytest.mark.parametrize("tB", [0, 1])
@pytest.mark.parametrize("M,N,K", [(17, 1, 64), (33, 3, 7), (40, 100, 1000), (100, 65, 17),
                                   (300, 20, 333), (64, 130, 2049)])
def test_products_of_few_tiles(env, M, N, K, tB):
    grouped_case(env, tB, [M], N, K, 1, 2)
    grouped_case(env, tB, [M], N, K, 1, 2, pad=1, shift=1, alpha=0.5, beta=-1.0)
    grouped_case(env, tB, [M, 0, 5], N, K, 1, 2, pad=3, shift=2)


def test_the_most_groups(env):
    """65536 groups, most of them empty, around row and column ends."""
    torch, pg = env
    G, M, N, K = 65536, 70, 33, 5
    rng = np.random.default_rng(1)
    owner = np.sort(rng.choice(G, M))
    owner[0], owner[-1] = 0, G - 1
    off = torch.from_numpy(np.searchsorted(owner, np.arange(G + 1)).astype(np.int32)).cuda()
    A = rng.integers(-8, 9, (M, K)).astype(np.float32)
    B = rng.integers(-8, 9, (G, K, N)).astype(np.float32)
    log(f"[grouped] G={G} M={M} N={N} K={K}")
    C = torch.full((M, N), torch.nan, device="cuda")
    pg.sgemm_grouped(0, M, N, K, G, off, 1.0, torch.from_numpy(A).cuda(), K,
                     torch.from_numpy(B).cuda(), N, K * N, 0.0, C, N)
    want = np.stack([A[m] @ B[owner[m]] for m in range(M)])  # exact: small whole numbers
    assert np.array_equal(C.cpu().numpy(), want)
