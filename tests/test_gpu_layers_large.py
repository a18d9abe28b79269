"""The norms, the 4-bit calls and the experts' layer on operands past 2^31
elements or bytes, and on more rows than one launch takes: the places that an
offset of 32 bits would miss are checked against 64-bit values."""
import sys

import pytest

from test_gpu_mx4gemm import Operand, packed, value

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


def far_rows(torch, rows, ld):
    """A matrix of `rows` on the GPU, `ld` elements apart."""
    t = torch.zeros((len(rows) - 1) * ld + rows.shape[1], dtype=rows.dtype, device="cuda")
    view = t.as_strided(rows.shape, (ld, 1))
    view.copy_(rows)
    return t, view


def test_rows_far_apart(env):
    """Rows 2^30 + 16 elements apart: the third starts past 2^31."""
    torch, pg = env
    ld, M, K = 2**30 + 16, 3, 200
    g = torch.Generator().manual_seed(1)
    x = torch.randn(M, K, generator=g).half()
    w = torch.ones(K).cuda()
    log("[far rows] norm")
    X, _ = far_rows(torch, x, ld)
    H, h = far_rows(torch, torch.zeros(M, K, dtype=torch.float16), ld)
    near, Y, Yn = torch.zeros(M, K).half().cuda(), torch.zeros(M, K).half().cuda(), \
        torch.zeros(M, K).half().cuda()
    pg.rms_norm(M, K, X, ld, X, ld, w, 1e-6, H, ld, Y, K)
    pg.rms_norm(M, K, x.cuda(), K, x.cuda(), K, w, 1e-6, near, K, Yn, K)
    assert torch.equal(Y, Yn) and torch.equal(h, near) and bool(Y[2].any())
    dw, dwn, dXn = torch.zeros(K).cuda(), torch.zeros(K).cuda(), torch.zeros(M, K).half().cuda()
    ws = torch.empty(pg.rms_norm_grad_workspace_size(M, K, X.dtype), dtype=torch.uint8).cuda()
    pg.rms_norm_grad(M, K, x.cuda(), K, near, K, w, 1e-6, x.cuda(), K, dXn, K, dwn, ws)
    pg.rms_norm_grad(M, K, X, ld, H, ld, w, 1e-6, X, ld, X, ld, dw, ws)
    assert torch.equal(X.as_strided((M, K), (ld, 1)), dXn) and torch.equal(dw, dwn)
    del X, H, h
    log("[far rows] 4 bits")
    X, _ = far_rows(torch, x, ld)
    Q, q = far_rows(torch, torch.zeros(M, K // 2, dtype=torch.uint8), ld)
    s, sn = (torch.zeros(2, M, 4, dtype=torch.uint8).cuda() for _ in range(2))
    qn = torch.zeros(M, K // 2, dtype=torch.uint8).cuda()
    pg.mx4_quantize_rows(M, K, X, ld, Q, ld, s, M)
    pg.mx4_quantize_rows(M, K, x.cuda(), K, qn, K // 2, sn, M)
    assert torch.equal(q, qn) and torch.equal(s, sn) and bool(qn[2].any())
    pg.mx4_dequantize_rows(M, K, Q, ld, s, M, X, ld)
    pg.mx4_dequantize_rows(M, K, qn, K // 2, sn, M, Y, K)
    assert torch.equal(X.as_strided((M, K), (ld, 1)), Y)


def test_many_rows(env):
    """More rows than one launch of the rounding takes."""
    torch, pg = env
    K, n, times = 40, 1000, 1100
    g = torch.Generator().manual_seed(2)
    x = torch.randn(n, K, generator=g).half().cuda()
    X, M = x.repeat(times, 1), n * times
    Q, S = torch.zeros(M, K // 2, dtype=torch.uint8).cuda(), torch.zeros(1, M, 4, dtype=torch.uint8).cuda()
    Y = torch.zeros(M, K).cuda()
    pg.mx4_quantize_rows(M, K, X, K, Q, K // 2, S, M)
    pg.mx4_dequantize_rows(M, K, Q, K // 2, S, M, Y, K)
    q, s = Q[:n], S[:, :n]
    assert bool(q.any()) and torch.equal(Q, q.repeat(times, 1)) and torch.equal(S, s.repeat(1, times, 1))
    assert torch.equal(Y, Y[:n].repeat(times, 1)) and bool(Y.any())


@pytest.mark.parametrize("M", [3, 40, 300])
def test_weights_past_2_31_bytes(env, M):
    """The last channels of 600000 x 8192 in 4 bits (2.46 GB)."""
    torch, pg = env
    N, K, last = 600000, 8192, 48
    log(f"[mx4gemm] {M}x{N}x{K}")
    g = torch.Generator().manual_seed(M)
    A, B = Operand(torch, g, M, K), Operand(torch, g, last, K)
    W = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    SW = torch.full((K // 128, N, 4), 127, dtype=torch.uint8, device="cuda")
    W[N - last:] = B.t.view(last, K // 2)
    SW[:, N - last:] = B.s[0]
    C = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    pg.mx4gemm(M, N, K, A.t, K // 2, A.s, M, W, K // 2, SW, N, None, C, N)
    want = A.host[0] @ B.host[0].T
    size = A.host[0].abs() @ B.host[0].abs().T
    tol = size * ((K // 64 + 1) * 2.0 ** -19 + 20 * 2.0 ** -24)
    tol = tol + (want.abs() + tol) * 2.0 ** -8
    assert bool(((C[:, N - last:].cpu().double() - want).abs() <= tol).all())
    assert bool((C[:, :N - last] == 0).all())


@pytest.mark.parametrize("kind", ["same", "i8", "mx4"])
def test_experts_past_2_32_bytes(env, kind):
    """An expert whose weights start beyond 2^32 bytes."""
    torch, pg = env
    T, E, H, F = 2, 5, 256, 160
    dt = torch.bfloat16
    g = torch.Generator().manual_seed(3)
    from test_gpu_expert_layer import Weights
    near1, near2 = Weights(torch, g, 1, 2 * F, H, kind, dt), Weights(torch, g, 1, H, F, kind, dt)
    stride = 2**30 + 64 if kind == "same" else 2**31 + 64  # elements; bytes of the others
    far1 = torch.zeros((E - 1) * stride + 2 * F * near1.ld, dtype=near1.t.dtype, device="cuda")
    far2 = torch.zeros((E - 1) * stride + H * near2.ld, dtype=near2.t.dtype, device="cuda")
    far1[(E - 1) * stride:] = near1.t[:2 * F * near1.ld]
    far2[(E - 1) * stride:] = near2.t[:H * near2.ld]
    s1 = s2 = None
    if kind != "same":
        s1 = torch.cat([torch.zeros_like(near1.scale)] * (E - 1) + [near1.scale])
        s2 = torch.cat([torch.zeros_like(near2.scale)] * (E - 1) + [near2.scale])
    x = torch.randn(T, H, generator=g).to(dt).cuda()
    outs = []
    for e, n, w1, d1, sc1, w2, d2, sc2 in (
            (0, 1, near1.t, near1.stride, near1.scale, near2.t, near2.stride, near2.scale),
            (E - 1, E, far1, stride, s1, far2, stride, s2)):
        out = torch.zeros(T, H, dtype=dt).cuda()
        ws = torch.zeros(pg.expert_layer_workspace_size(T, 1, H, F, dt), dtype=torch.uint8).cuda()
        ids = torch.full((T, 1), e, dtype=torch.int32).cuda()
        pg.expert_layer(T, 1, n, H, F, x, H, ids, None, w1, near1.ld, d1, sc1, w2, near2.ld, d2, sc2,
                        out, H, ws)
        outs.append(out.float())
    # Both are the same sums; the number of experts may spread K over more waves.
    assert bool(outs[0].any())
    assert float((outs[0] - outs[1]).abs().max()) <= 2.0 ** -7 * float(outs[0].abs().max())


def test_values_of_the_helpers():
    """The 4-bit helpers these tests share with those of the products."""
    import torch
    code = torch.tensor([[1, 15, 7]])
    assert packed(torch, code).tolist() == [[0xf1, 0x07]]
    assert value(torch, code, torch.tensor([[128]]), 3).tolist() == [[1.0, -12.0, 12.0]]
