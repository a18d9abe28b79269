"""The norm with the residual's addition, its 8-bit output and its gradients
against 64-bit values.

Tolerances: a sum of K squares or products in fp32, in up to 64 terms a thread
and a tree over the threads, is within (64 + 12) 2^-24 of the sum of the
magnitudes; a division, root, product or conversion rounds by at most half a
step (2^-24 in fp32)."""
import sys

import pytest

pytestmark = pytest.mark.gpu
TYPES = ["float32", "float16", "bfloat16"]
SUM = 80 * 2.0 ** -24  # of a sum of up to 2^16 terms, relative to the magnitudes' sum


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


def matrix(torch, g, rows, cols, dtype, ld=None, shift=0, size=1.0):
    """(tensor `shift` elements into its storage, rows `ld` apart; its values)"""
    ld = max(1, cols) if ld is None else ld
    store = (size * torch.randn(max(1, rows) * ld + shift, generator=g)).to(dtype)
    host = store[shift:].view(max(1, rows), ld)[:rows, :cols]
    return store.cuda()[shift:], host, ld


def half_step(torch, dtype, v):
    """Most that rounding `v` to `dtype` moves it."""
    f = torch.finfo(dtype)
    return v.abs() * f.eps / 2 + f.smallest_normal * f.eps / 2


def reference(torch, x, r, w, eps, dtype):
    h = x if r is None else (x.float() + r.float()).to(dtype)
    hd, wd = h.double(), w.double()
    rstd = 1 / (hd.square().sum(1) / max(1, h.shape[1]) + eps).sqrt()
    t = (hd * wd).float()
    return h, rstd, t


def run_norm(env, M, K, dtype, residual=True, keep=True, lds=(0, 0, 0, 0), shift=0, eps=1e-5,
             size=1.0, seed=0, i8=True):
    torch, pg = env
    log(f"[norm] {M}x{K} {dtype} residual={residual} keep={keep} lds={lds} shift={shift} i8={i8}")
    g = torch.Generator().manual_seed(1000 * M + K + seed)
    dt = getattr(torch, dtype)
    dx, x, ldx = matrix(torch, g, M, K, dt, max(1, K) + lds[0], shift, size)
    dr, r, ldr = matrix(torch, g, M, K, dt, max(1, K) + lds[1], shift, size)
    w = 1 + 0.5 * torch.randn(K, generator=g)
    ldh, ldo = max(1, K) + lds[2], max(1, K) + lds[3]
    H = torch.full((M, ldh), 7.0, dtype=dt, device="cuda")
    R = (dr, ldr) if residual else (None, 0)
    h, rstd, t = reference(torch, x, r if residual else None, w, eps, dt)
    kept = (H, ldh) if keep else (None, 0)
    if i8:
        Q = torch.full((M, ldo), 77, dtype=torch.int8, device="cuda")
        scale = torch.full((M,), 7.0, device="cuda")
        pg.rms_norm_i8(M, K, dx, ldx, *R, w.cuda(), eps, *kept, Q, ldo, scale)
        s = (t.abs().amax(1).double() / 127).float().clamp_min(2.0 ** -126)
        want = torch.round(t.double() / s.double()[:, None])
        torch.cuda.synchronize()
        assert torch.equal(Q[:, :K].cpu().double(), want)
        assert bool((Q[:, K:] == 77).all())
        exact = s.double() * rstd
        # the sum, the mean, the root, its reciprocal and the product with s
        assert bool(((scale.cpu().double() - exact).abs() <= exact * (SUM / 2 + 5 * 2.0 ** -24)).all())
    else:
        Y = torch.full((M, ldo), 7.0, dtype=dt, device="cuda")
        pg.rms_norm(M, K, dx, ldx, *R, w.cuda(), eps, *kept, Y, ldo)
        torch.cuda.synchronize()
        exact = t.double() * rstd[:, None]
        off = (Y[:, :K].cpu().double() - exact).abs()
        allowed = exact.abs() * (SUM / 2 + 5 * 2.0 ** -24)
        assert bool((off <= allowed + half_step(torch, dt, exact.abs() + allowed)).all())
        assert bool((Y[:, K:] == 7).all())
    if keep:
        assert torch.equal(H[:, :K].cpu(), h) and bool((H[:, K:] == 7).all())


SIZES = [(1, 1), (3, 5), (1, 64), (33, 63), (70, 129), (5, 1000), (4, 4096), (37, 2047), (2, 8200),
         (3, 16384), (2, 33000), (1, 140000)]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", SIZES)
def test_sizes(env, M, K, dtype, i8):
    if K > 2 ** 16:
        # more terms a thread: 140000 / (1024 threads) in chunks, up to 144
        K = 140000
    run_norm(env, M, K, dtype, i8=i8)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(3, 8192), (3, 8193), (5, 14915), (3, 20001), (2, 32768)])
def test_long_rows(env, M, K, dtype, i8):
    run_norm(env, M, K, dtype, i8=i8)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("residual,keep", [(False, False), (False, True), (True, False)])
def test_without_parts(env, residual, keep, i8):
    run_norm(env, 9, 513, "bfloat16", residual, keep, i8=i8)
    run_norm(env, 2, 70000, "bfloat16", residual, keep, i8=i8)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_alignment(env, dtype, i8):
    run_norm(env, 13, 257, dtype, lds=(1, 3, 2, 5), shift=1, i8=i8)
    run_norm(env, 6, 4096, dtype, lds=(8, 0, 1, 7), shift=3, i8=i8)


@pytest.mark.parametrize("K", [40, 4096, 70000])
@pytest.mark.parametrize("alias", ["X", "R"])
def test_sum_in_place(env, alias, K):
    """H may be X or R."""
    torch, pg = env
    g = torch.Generator().manual_seed(K)
    x, r = (torch.randn(5, K, generator=g).bfloat16() for _ in range(2))
    w = torch.randn(K, generator=g).cuda()
    out = []
    for into in (None, alias):
        X, R = x.cuda(), r.cuda()
        H = torch.empty_like(X) if into is None else X if into == "X" else R
        Q, s, Y = torch.zeros(5, K, dtype=torch.int8).cuda(), torch.zeros(5).cuda(), torch.empty_like(X)
        pg.rms_norm_i8(5, K, X, K, R, K, w, 1e-6, H, K, Q, K, s)
        X2, R2 = x.cuda(), r.cuda()
        H2 = torch.empty_like(X) if into is None else X2 if into == "X" else R2
        pg.rms_norm(5, K, X2, K, R2, K, w, 1e-6, H2, K, Y, K)
        out.append([v.cpu() for v in (H, Q, s, H2, Y)])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_special_rows(env):
    """Rows of zeros, of subnormal, huge and non-finite values."""
    torch, pg = env
    K = 100
    rows = torch.ones(7, K)
    rows[0] = 0
    rows[1] = 2.0 ** -140
    rows[2, 5] = float("inf")
    rows[3, 7] = float("nan")
    rows[4] = 2.0 ** 70
    rows[5] = torch.arange(K) - 50.0
    w = torch.linspace(0.5, 2, K)
    X, W = rows.cuda(), w.cuda()
    Q, s = torch.full((7, K), 9, dtype=torch.int8).cuda(), torch.zeros(7).cuda()
    Y = torch.zeros(7, K).cuda()
    pg.rms_norm_i8(7, K, X, K, None, 0, W, 1e-6, None, 0, Q, K, s)
    pg.rms_norm(7, K, X, K, None, 0, W, 1e-6, None, 0, Y, K)
    Q, s, Y = Q.cpu(), s.cpu(), Y.cpu()
    assert bool((Q[0] == 0).all()) and abs(s[0].item() / (2.0 ** -126 * 1e3) - 1) < 1e-6
    assert bool((Q[1] == 0).all())  # below half of the least step
    assert bool((Q[2] == 0).all()) and bool(s[2].isnan()) and bool((Q[3] == 0).all()) and bool(s[3].isnan())
    assert bool(Y[2, 5].isnan()) and bool((Y[2, :5] == 0).all()) and bool(Y[3].isnan().all())
    assert bool((Y[4] == 0).all()) and s[4] == 0  # squares beyond fp32
    assert bool((Y[6] - w * (1 / (1 + 1e-6) ** 0.5)).abs().max() < 1e-6)


def run_grad(env, M, K, dtype, with_dh=True, with_dw=True, lds=(0, 0, 0, 0), shift=0, eps=1e-5,
             seed=0):
    torch, pg = env
    log(f"[norm grad] {M}x{K} {dtype} dh={with_dh} dw={with_dw} lds={lds} shift={shift}")
    g = torch.Generator().manual_seed(31 * M + K + seed)
    dt = getattr(torch, dtype)
    ddy, dy, lddy = matrix(torch, g, M, K, dt, max(1, K) + lds[0], shift)
    dh_, h, ldh = matrix(torch, g, M, K, dt, max(1, K) + lds[1], shift)
    ddh, dh, lddh = matrix(torch, g, M, K, dt, max(1, K) + lds[2], shift)
    w = 1 + 0.5 * torch.randn(K, generator=g)
    lddx = max(1, K) + lds[3]
    dX = torch.full((max(1, M), lddx), 7.0, dtype=dt, device="cuda")
    dw = torch.full((K,), 7.0, device="cuda") if with_dw else None
    need = pg.rms_norm_grad_workspace_size(M, K, dt)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if with_dw else None
    pg.rms_norm_grad(M, K, ddy, lddy, dh_, ldh, w.cuda(), eps, ddh if with_dh else None, lddh, dX,
                     lddx, dw, ws)
    torch.cuda.synchronize()
    x, gy, wd = h.double(), dy.double(), w.double()
    rstd = 1 / (x.square().sum(1, keepdim=True) / K + eps).sqrt()
    along = (wd * gy * x).sum(1, keepdim=True) / K * rstd ** 2
    base = dh.double() if with_dh else torch.zeros_like(x)
    want = base + rstd * (wd * gy - x * along)
    # the sums' errors, and a few roundings of each term
    size = base.abs() + rstd * ((wd * gy).abs() + x.abs() * along.abs())
    spread = rstd * x.abs() * rstd ** 2 * (wd * gy * x).abs().sum(1, keepdim=True) / K
    allowed = size * (2 * SUM + 10 * 2.0 ** -24) + spread * SUM
    if M:
        off = (dX[:M, :K].cpu().double() - want).abs()
        assert bool((off <= allowed + half_step(torch, dt, want.abs() + allowed)).all())
    assert bool((dX[:, K:] == 7).all())
    if with_dw:
        terms = gy * x * rstd
        want = terms.sum(0)
        # up to M / 1024 + 1 rows a group in turn, then up to 16384 / 32 groups in turn and 32
        steps = M // 1024 + 2 + 512 + 32
        allowed = terms.abs().sum(0) * (steps * 2.0 ** -24 + SUM / 2 + 6 * 2.0 ** -24)
        assert bool(((dw.cpu().double() - want).abs() <= allowed).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (3, 5), (40, 64), (33, 129), (500, 1000), (5, 513),
                                 (1100, 2048), (7, 4096), (9, 5003), (1030, 8192), (3, 16384),
                                 (5, 12001)])
def test_gradients(env, M, K, dtype):
    run_grad(env, M, K, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_parts(env, dtype):
    run_grad(env, 17, 300, dtype, with_dh=False)
    run_grad(env, 17, 300, dtype, with_dw=False)
    run_grad(env, 17, 300, dtype, lds=(1, 3, 2, 5), shift=1)
    run_grad(env, 0, 300, dtype)  # dweight is 0


def test_gradients_against_differences(env):
    """Central differences of sum(dY * Y) + sum(dH * H) in fp64."""
    torch, pg = env
    M, K, eps = 3, 40, 1e-5
    g = torch.Generator().manual_seed(5)
    h, dy, dh = (torch.randn(M, K, generator=g) for _ in range(3))
    w = torch.randn(K, generator=g)

    def loss(h, w):
        y = h * w / (h.square().mean(1, keepdim=True) + eps).sqrt()
        return ((y * dy.double()) + h * dh.double()).sum()

    dX, dw = torch.zeros(M, K).cuda(), torch.zeros(K).cuda()
    ws = torch.empty(pg.rms_norm_grad_workspace_size(M, K, torch.float32), dtype=torch.uint8).cuda()
    pg.rms_norm_grad(M, K, dy.cuda(), K, h.cuda(), K, w.cuda(), eps, dh.cuda(), K, dX, K, dw, ws)
    step = 1e-4
    for m, k in ((0, 0), (1, 17), (2, 39)):
        d = torch.zeros(M, K, dtype=torch.float64)
        d[m, k] = step
        fd = (loss(h.double() + d, w.double()) - loss(h.double() - d, w.double())) / (2 * step)
        assert abs(fd - dX[m, k].item()) < 1e-5 * (1 + abs(fd))
    for k in (0, 21):
        d = torch.zeros(K, dtype=torch.float64)
        d[k] = step
        fd = (loss(h.double(), w.double() + d) - loss(h.double(), w.double() - d)) / (2 * step)
        assert abs(fd - dw[k].item()) < 1e-5 * (1 + abs(fd))


@pytest.mark.parametrize("K", [48, 2048, 9000])
@pytest.mark.parametrize("alias", ["dY", "dH"])
def test_gradient_in_place(env, alias, K):
    torch, pg = env
    g = torch.Generator().manual_seed(K)
    M = 1500
    dy, h, dh = (torch.randn(M, K, generator=g).half() for _ in range(3))
    w = torch.randn(K, generator=g).cuda()
    ws = torch.empty(pg.rms_norm_grad_workspace_size(M, K, torch.float16), dtype=torch.uint8).cuda()
    out = []
    for into in (None, alias):
        dY, dH, H = dy.cuda(), dh.cuda(), h.cuda()
        dX = torch.empty_like(H) if into is None else dY if into == "dY" else dH
        dw = torch.zeros(K).cuda()
        pg.rms_norm_grad(M, K, dY, K, H, K, w, 1e-6, dH, K, dX, K, dw, ws)
        out.append((dX.cpu(), dw.cpu()))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_captured_with_its_product(env):
    """Norm, 8-bit product, norm and gradient in one graph, replayed with the
    program's own work between."""
    torch, pg = env
    M, K, N = 9, 256, 96
    g = torch.Generator().manual_seed(3)
    x, r = (torch.randn(M, K, generator=g).bfloat16() for _ in range(2))
    X, R, w = x.cuda(), r.cuda(), torch.randn(K, generator=g).cuda()
    H = torch.zeros_like(X)
    Q, s = torch.zeros(M, K, dtype=torch.int8).cuda(), torch.zeros(M).cuda()
    B = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sB = torch.rand(N, generator=g).cuda()
    C = torch.zeros(M, N, dtype=torch.bfloat16).cuda()
    Y, dX, dw = torch.zeros_like(X), torch.zeros_like(X), torch.zeros(K).cuda()
    ws = torch.empty(pg.rms_norm_grad_workspace_size(M, K, X.dtype), dtype=torch.uint8).cuda()

    def step():
        pg.rms_norm_i8(M, K, X, K, R, K, w, 1e-6, H, K, Q, K, s)
        pg.i8gemm(M, N, K, Q, K, s, B, K, sB, None, C, N)
        pg.rms_norm(M, K, H, K, None, 0, w, 1e-6, None, 0, Y, K)
        pg.rms_norm_grad(M, K, Y, K, H, K, w, 1e-6, R, K, dX, K, dw, ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        X.copy_((x * (i + 1)).bfloat16())
        for t in (H, Q, s, C, Y, dX, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (H, Q, s, C, Y, dX, dw)]
        for t in (H, Q, s, C, Y, dX, dw):
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (H, Q, s, C, Y, dX, dw)))
    # and the product is that of the norm's values
    h = H.cpu().double()
    y = h * w.cpu().double() / (h.square().mean(1, keepdim=True) + 1e-6).sqrt()
    want = y @ (B.cpu().double() * sB.cpu().double()[:, None]).T
    # every value is off by half a step of its row at most
    step_ = (y.abs().amax(1, keepdim=True) / 127 / 2) * (B.cpu().double().abs() * sB.cpu().double()[:, None]).sum(1)
    assert bool(((C.cpu().double() - want).abs() <= 1.01 * step_ + want.abs() * 2.0 ** -7).all())
