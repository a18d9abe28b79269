"""Grouped products whose offsets decrease, with so many rows in so many groups
that their tiles, counted one by one, would pass 2^31."""
import sys

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["mx4gemm_grouped", "i8gemm_grouped", "sgemm_grouped"])
def test_counts_of_tiles_stay_in_range(call):
    """Offsets 0, M, 0, M, ...: every second group holds all rows. All groups share
    one B, so a row's value does not depend on whose it is, and the first group
    alone has a tile for every row."""
    import torch
    import precision_gemm_amd as pg
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M, groups = (1 << 23) + 128, 65536
    sys.stdout.write(f"[{call}] M={M} groups={groups}\n")
    sys.stdout.flush()
    g = torch.Generator(device="cuda").manual_seed(1)
    off = torch.zeros(groups + 1, dtype=torch.int32).cuda()
    off[1::2] = M
    C = torch.full((M + 64,), 7.0).cuda()
    if call == "sgemm_grouped":
        a = torch.randint(-100, 100, (M,), generator=g, device="cuda").float()
        b = torch.tensor([3.0]).cuda()
        pg.sgemm_grouped(1, M, 1, 1, groups, off, 1.0, a, 1, b, 1, 0, 0.0, C, 1)
        want = 3 * a
    elif call == "i8gemm_grouped":
        a = torch.randint(-100, 100, (M,), generator=g, device="cuda", dtype=torch.int8)
        b = torch.tensor([3], dtype=torch.int8).cuda()
        one = torch.ones(max(M, groups)).cuda()
        pg.i8gemm_grouped(M, 1, 1, groups, off, a, 1, one, b, 1, 0, one, None, C, 1)
        want = 3 * a.float()
    else:
        a = torch.randint(0, 256, (M,), generator=g, device="cuda", dtype=torch.uint8)
        b = torch.tensor([2 + 16 * 12], dtype=torch.uint8).cuda()  # 1 and -2
        sa, sb = (torch.full((n, 4), 127, dtype=torch.uint8).cuda() for n in (M, 1))
        pg.mx4gemm_grouped(M, 1, 2, groups, off, a, 1, sa, M, b, 1, 0, sb, 1, 0, None, C, 1)
        level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6]).cuda()
        level = torch.cat([level, -level])
        want = level[(a & 15).long()] - 2 * level[(a >> 4).long()]
    assert torch.equal(C[:M], want) and bool((C[M:] == 7).all())
