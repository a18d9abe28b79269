"""Values of the experts' layer that are known exactly: what each sum holds is a
number of fp32, so the outputs are compared for equality."""
import sys

import pytest

pytestmark = pytest.mark.gpu
TYPES = ["float32", "float16", "bfloat16"]
KINDS = ["same", "i8", "mx4"]
LEVELS = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


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


def weights(torch, w, kind, dt):
    """E x rows x K weights of 0, 1 and -1 in a kind's form: tensor, row, stride, scale."""
    E, rows, K = w.shape
    if kind == "same":
        return w.to(dt).cuda(), K, rows * K, None
    if kind == "i8":
        return w.to(torch.int8).cuda(), K, rows * K, torch.ones(E, rows).cuda()
    code = torch.zeros(E, rows, (K + 1) // 2 * 2, dtype=torch.int64)
    code[..., :K] = 2 * w.abs().long() + 8 * (w < 0).long()
    width = code.shape[2] // 2
    scale = torch.full((E, (K + 127) // 128, rows, 4), 127, dtype=torch.uint8).cuda()
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8).cuda(), width, rows * width, \
        scale


def run(env, x, ids, E, w1, w2, kind):
    torch, pg = env
    dt = x.dtype
    (T, H), k, F = x.shape, ids.shape[1], w2.shape[2]
    W1, ld1, st1, s1 = weights(torch, w1, kind, dt)
    W2, ld2, st2, s2 = weights(torch, w2, kind, dt)
    out = torch.full((T, H), 7.0, dtype=dt).cuda()
    ws = torch.full((pg.expert_layer_workspace_size(T, k, H, F, dt),), 255, dtype=torch.uint8).cuda()
    pg.expert_layer(T, k, E, H, F, x.cuda(), H, ids.int().cuda(), None, W1, ld1, st1, s1, W2, ld2,
                    st2, s2, out, H, ws)
    return out.cpu()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H,F", [(1, 1, 1, 64, 64), (1, 8, 16, 4160, 96), (3, 2, 8, 200, 102),
                                       (16, 2, 20, 960, 480), (64, 8, 64, 64, 416),
                                       (40, 1, 2, 130, 2080)])
def test_inner_values_keep_24_bits(env, T, k, E, H, F, dtype, kind):
    """Inner values that differ in bits 18 to 24 alone, and outputs that are their
    differences. The gate is 64, whose sigmoid is 1 in fp32; the inner values are
    64 (64.25 + 2^-11 to 2^-17) and 64 * 64.25, each a number of 24 bits, every
    product with a weight of 1 or -1 too, and so are the sums in any order: of an
    output's two inner values, and of their slots."""
    torch, _ = env
    log(f"[24 bits] T={T} k={k} E={E} H={H} F={F} {dtype} {kind}")
    g = torch.Generator().manual_seed(T + H)
    x = torch.zeros(T, H)
    x[:, 0] = x[:, 1] = 64
    x[:, 9] = 0.25
    for i in range(7):
        x[:, 2 + i] = 2.0 ** -(11 + i)
    w1, w2 = torch.zeros(E, 2 * F, H), torch.zeros(E, H, F)
    w1[:, :F, 0] = 1
    w1[:, F:, 1] = w1[:, F:, 9] = 1
    which = torch.randint(0, 7, (E, F // 2), generator=g)
    w1[:, F:F + 2 * (F // 2):2] += torch.nn.functional.one_hot(2 + which, H)
    pair = torch.randint(0, F // 2, (E, H), generator=g)
    w2.scatter_(2, 2 * pair[..., None], 1.0)
    w2.scatter_(2, 2 * pair[..., None] + 1, -1.0)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    each = 2.0 ** -(5 + torch.gather(which, 1, pair).double())
    want = torch.zeros(T, H, dtype=torch.float64)
    for j in range(k):
        want += each[ids[:, j]]
    dt = getattr(torch, dtype)
    got = run(env, x.to(dt), ids, E, w1, w2, kind)
    assert torch.equal(got, want.to(dt))
