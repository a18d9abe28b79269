"""4-bit products whose sums are exact, compared for equality over long rows: with
scales of 1 a product is a multiple of 1/4 of at most 36, and the sums of random
signs stay below 2^13, far from where an instruction drops anything (2^-22 of the
largest). A single k lost, doubled or swapped would show."""
import sys

import pytest

from test_gpu_mx4gemm import LEVELS, packed

pytestmark = pytest.mark.gpu
SIZES = [("S16x16", 7, 300, 8190), ("S16x32", 9, 16400, 8192), ("S32x16", 45, 600, 8159),
         ("S32x32", 40, 4000, 8192), ("S32x64", 20, 10000, 8190), ("T64x64", 300, 2000, 8191),
         ("T128x128", 2050, 2060, 8190), ("L64x64", 300, 2000, 8192),
         ("L64x128", 1000, 4000, 8160), ("L128x128", 1000, 4000, 4096),
         ("L128x128_R2", 2000, 4100, 8192), ("L128x256", 2050, 2060, 2144),
         ("L256x256", 4001, 8192, 4128)]


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_gemm_amd as pg
    pg._load()
    yield torch, pg
    torch.cuda.empty_cache()


def rows(torch, g, n, K):
    """n rows of K: bytes (16-byte rows where K allows the fast kernels), their
    values, and scales of 1 with NaN's behind the last block."""
    code = torch.randint(0, 16, (n, K), generator=g, device="cuda")
    level = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64).cuda()
    scale = torch.full((-(-K // 128), n, 4), 127, dtype=torch.uint8).cuda()
    if -(-K // 32) % 4:
        scale[-1, :, -(-K // 32) % 4:] = 255
    return packed(torch, code, odd=7), level[code], scale


@pytest.mark.parametrize("name,M,N,K", SIZES)
def test_sums_of_long_rows(env, name, M, N, K):
    torch, pg = env
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    chosen = pg.MX4GEMM_KERNELS[pg.mx4gemm_select_kernel(M, N, K, 0, K % 32 == 0, cus)]
    sys.stdout.write(f"[mx4gemm] {M}x{N}x{K} {chosen}\n")
    sys.stdout.flush()
    if cus == 256:
        assert chosen == name
    g = torch.Generator(device="cuda").manual_seed(K + M)
    A, a, sA = rows(torch, g, M, K)
    B, b, sB = rows(torch, g, N, K)
    C = torch.full((M, N), 7.0).cuda()
    width = A.shape[1]
    pg.mx4gemm(M, N, K, A, width, sA, M, B, width, sB, N, None, C, N)
    want = torch.mm(a, b.t().contiguous())
    assert float(want.abs().max()) < 2.0 ** 13
    assert torch.equal(C.double(), want)


@pytest.mark.parametrize("K", [2048, 2050])
def test_sums_of_groups(env, K):
    torch, pg = env
    M, N, groups = 1200, 520, 9
    g = torch.Generator(device="cuda").manual_seed(K)
    A, a, sA = rows(torch, g, M, K)
    B, b, sB = rows(torch, g, groups * N, K)
    ends = [3, 3, 50, 51, 400, 401, 900, 900, 1100, 1190]
    off = torch.tensor(ends, dtype=torch.int32).cuda()
    words, width = sB.shape[0], A.shape[1]
    sB = sB.view(words, groups, N, 4).transpose(0, 1).contiguous()
    C = torch.full((M, N), 7.0).cuda()
    pg.mx4gemm_grouped(M, N, K, groups, off, A, width, sA, M, B, width, N * width, sB, N,
                       4 * words * N, None, C, N)
    want = torch.full((M, N), 7.0, dtype=torch.float64).cuda()
    for e, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        if hi > lo:
            want[lo:hi] = torch.mm(a[lo:hi], b[e * N:(e + 1) * N].t().contiguous())
    assert torch.equal(C.double(), want)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_every_element_with_every_scale(env, dtype):
    """The way back of all 16 codes and 256 scale bytes; beyond the type's range it
    is infinite."""
    torch, pg = env
    from test_gpu_mx4gemm import value
    dt = getattr(torch, dtype)
    code = torch.arange(16).repeat(256, 2)
    byte = torch.arange(256)[:, None]
    scale = torch.zeros(1, 256, 4, dtype=torch.uint8)
    scale[0, :, 0] = byte[:, 0].to(torch.uint8)
    Y = torch.zeros(256, 32, dtype=dt).cuda()
    pg.mx4_dequantize_rows(256, 32, packed(torch, code).cuda(), 16, scale.cuda(), 256, Y, 32)
    want = value(torch, code, byte, 32).to(dt)
    assert torch.equal(Y.cpu().isnan(), want.isnan()) and bool(want[255].isnan().all())
    assert torch.equal(Y.cpu()[:255], want[:255])
    assert bool(want[253, [6, 7]].isinf().all()) and bool(want[254, 4:8].isinf().all())
