"""The norms at the ends of fp32's range, over more rows than one launch takes, and
gradients whose sums are exact."""
import sys

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
    yield torch, pg
    torch.cuda.empty_cache()


def norms(env, rows, w, eps):
    """Y, Q, scale, dX and dweight of fp32 rows, dY and dH of ones."""
    torch, pg = env
    M, K = rows.shape
    X, W, one = rows.cuda(), w.cuda(), torch.ones(M, K).cuda()
    Y, dX, dw = torch.full((M, K), 7.0).cuda(), torch.full((M, K), 7.0).cuda(), torch.zeros(K).cuda()
    Q, s = torch.full((M, K), 9, dtype=torch.int8).cuda(), torch.zeros(M).cuda()
    ws = torch.zeros(max(1, pg.rms_norm_grad_workspace_size(M, K, X.dtype)), dtype=torch.uint8).cuda()
    pg.rms_norm(M, K, X, K, None, 0, W, eps, None, 0, Y, K)
    pg.rms_norm_i8(M, K, X, K, None, 0, W, eps, None, 0, Q, K, s)
    pg.rms_norm_grad(M, K, one, K, X, K, W, eps, one, K, dX, K, dw, ws)
    return [t.cpu() for t in (Y, Q, s, dX, dw)]


@pytest.mark.parametrize("K", [64, 1024, 16384])
def test_large_rows(env, K):
    """The largest power of two whose squares' sum is a number, and the next one."""
    torch, _ = env
    log(f"[norm ends] K={K}")
    half = (K.bit_length() - 1) // 2  # K = 4^half
    rows = torch.stack([torch.full((K,), 2.0 ** (63 - half)), torch.full((K,), 2.0 ** (64 - half))])
    w = torch.linspace(0.5, 2, K)
    Y, Q, s, dX, dw = norms(env, rows, w, 1e-6)
    # rstd is a power of two, and exact
    assert torch.equal(Y[0], w) and bool((Y[1] == 0).all())
    step = (w.double().max() / 127).float().double()  # (a power of two below the row's)
    assert torch.equal(Q[0].double(), torch.round(w.double() / step)) and torch.equal(Q[0], Q[1])
    assert abs(s[0].item() * 127 / 2 - 1) <= 2.0 ** -22 and s[1] == 0
    # 1 + rstd (w - mean w): rstd is below half a step of 1; and 1 + 0
    assert bool((dX == 1).all())
    assert bool((dw - 1).abs().max() <= 2.0 ** -22)  # (of the second row nothing)


def test_no_epsilon(env):
    """eps = 0: rows of zeros, of squares that underflow, and of the least that do not."""
    torch, _ = env
    K = 64
    rows = torch.zeros(4, K)
    rows[1, ::2] = 2.0 ** -76
    rows[2] = 2.0 ** -74
    rows[3] = 3.0
    w = torch.ones(K)
    Y, Q, s, dX, dw = norms(env, rows, w, 0.0)
    assert bool(Y[0].isnan().all())
    assert bool((Y[1, ::2] == float("inf")).all()) and bool(Y[1, 1::2].isnan().all())
    assert torch.equal(Y[2], w) and torch.equal(Y[3], w)
    assert bool((Q[0] == 0).all()) and bool((Q[1, ::2] == 127).all()) and bool((Q[1, 1::2] == 0).all())
    assert bool((Q[2:] == 127).all()) and bool((s[:2] == float("inf")).all())
    assert float((s[2:] * 127 - 1).abs().max()) <= 2.0 ** -22
    assert not bool(dX[:2].isfinite().any()) and not bool(dw.isfinite().any())
    # the gradient along a row is none, of an even row's ones all
    assert float((dX[2:] - 1).abs().max()) <= 2.0 ** -20


@pytest.mark.parametrize("i8", [False, True])
def test_many_rows(env, i8):
    """More rows than one launch takes (2^26 of a column): the second launch's are
    those of a call of their own."""
    torch, pg = env
    first, more, K = 1 << 26, 300, 1
    M = first + more
    log(f"[many rows] {M}x{K} i8={i8}")
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(M, K, generator=g, device="cuda", dtype=torch.float16)
    R = torch.randn(M, K, generator=g, device="cuda", dtype=torch.float16)
    w = torch.full((K,), 1.5).cuda()
    H = torch.full((M + 64, K), 7.0, device="cuda", dtype=torch.float16)
    out = torch.full((M + 64, K), 77, device="cuda", dtype=torch.int8 if i8 else torch.float16)
    scale = torch.full((M + 64,), 7.0).cuda()

    def call(m, x, r, h, o, s):
        if i8:
            pg.rms_norm_i8(m, K, x, K, r, K, w, 1e-6, h, K, o, K, s)
        else:
            pg.rms_norm(m, K, x, K, r, K, w, 1e-6, h, K, o, K)

    call(M, X, R, H, out, scale)
    for lo, n in ((0, 300), (first - 200, 200), (first, more)):
        x, r = X[lo:lo + n].clone(), R[lo:lo + n].clone()
        h, o, s = torch.zeros_like(x), torch.zeros(n, K, dtype=out.dtype).cuda(), torch.zeros(n).cuda()
        call(n, x, r, h, o, s)
        assert torch.equal(H[lo:lo + n], h) and torch.equal(out[lo:lo + n], o)
        assert torch.equal(H[lo:lo + n], x + r) and bool(o.any())
        if i8:
            assert torch.equal(scale[lo:lo + n], s) and bool(s.any())
    assert bool((H[M:] == 7).all()) and bool((out[M:] == 77).all()) and bool((scale[M:] == 7).all())
    assert not bool((H[:M] == 7).all())


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("M,K", [(1, 1), (33, 64), (300, 1024), (1030, 8192), (2, 16384), (5000, 2048),
                                 (20000, 300), (16385, 40), (70, 129)])
def test_exact_gradients(env, M, K, dtype):
    """Rows of 1 and -1 with eps = 0 have rstd 1, and whole dY and dH make every sum a
    whole number (below 2^24): dweight, and dX where K is a power of two, are
    compared for equality, so that no row or column can be lost or taken twice."""
    torch, pg = env
    log(f"[exact gradients] {M}x{K} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(M + K)
    dt = getattr(torch, dtype)
    h = 1 - 2 * torch.randint(0, 2, (M, K), generator=g, device="cuda").double()
    dy, dh = (torch.randint(-8, 9, (M, K), generator=g, device="cuda").double() for _ in range(2))
    w = torch.exp2(torch.randint(-1, 2, (K,), generator=g, device="cuda").float())
    dX, dw = torch.full((M, K), 7.0, dtype=dt).cuda(), torch.full((K,), 7.0).cuda()
    ws = torch.full((pg.rms_norm_grad_workspace_size(M, K, dt),), 255, dtype=torch.uint8).cuda()
    pg.rms_norm_grad(M, K, dy.to(dt), K, h.to(dt), K, w, 0.0, dh.to(dt), K, dX, K, dw, ws)
    assert torch.equal(dw.double(), (dy * h).sum(0))
    if K & (K - 1) == 0:
        wdy = dy * w.double()
        want = dh + wdy - h * (wdy * h).sum(1, keepdim=True) / K
        assert torch.equal(dX, want.to(dt))
