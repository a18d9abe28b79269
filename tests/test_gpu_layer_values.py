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


class Blocks:
    """A 4-bit layer: random codes, and a scale byte of all blocks of W1's gate, its
    other part and W2."""

    def __init__(self, torch, g, E, H, F, gate=126, other=126, down=126):
        self.torch, self.E, self.H, self.F = torch, E, H, F
        self.c1 = torch.randint(0, 16, (E, 2 * F, H + H % 2), generator=g)
        self.c2 = torch.randint(0, 16, (E, H, F + F % 2), generator=g)
        self.s1 = torch.full((E, (H + 127) // 128, 2 * F, 4), gate, dtype=torch.uint8)
        self.s1[:, :, F:] = other
        self.s2 = torch.full((E, (F + 127) // 128, H, 4), down, dtype=torch.uint8)

    def run(self, pg, x, ids, mix=None):
        torch, E, H, F = self.torch, self.E, self.H, self.F
        w1, w2 = ((c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8).cuda()
                  for c in (self.c1, self.c2))
        d1, d2 = w1.shape[2], w2.shape[2]
        T, k = ids.shape
        out = torch.full((T, H), 7.0, dtype=x.dtype).cuda()
        ws = torch.full((pg.expert_layer_workspace_size(T, k, H, F, x.dtype),), 255,
                        dtype=torch.uint8).cuda()
        pg.expert_layer(T, k, E, H, F, x.cuda(), H, ids.int().cuda(),
                        None if mix is None else mix.cuda(), w1, d1, 2 * F * d1, self.s1.cuda(), w2,
                        d2, H * d2, self.s2.cuda(), out, H, ws)
        return out.cpu()


def some_tokens(torch, g, T, H, dt):
    """Tokens of 0.5 to 2 (either sign), each a bf16 number, so that they can be scaled."""
    x = 0.5 + 1.5 * torch.rand(T, H, generator=g)
    return (x * (1 - 2 * torch.randint(0, 2, (T, H), generator=g))).bfloat16().to(dt)


# even rows of one and of several words, the whole-sum kernel, ragged rows
BLOCK_SIZES = [(1, 2, 4, 64, 96), (1, 8, 16, 4160, 96), (20, 2, 3, 320, 160), (5, 2, 3, 130, 75)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,k,E,H,F", BLOCK_SIZES)
def test_ends_of_the_scales(env, T, k, E, H, F, dtype):
    """Blocks of 2^-127 (whose elements are subnormal bf16) and of 2^125, the largest
    that the rounding writes, give what blocks of about 1 give with the other
    operand scaled by the inverse power of two. To the bit, but where W2's are
    subnormal: an instruction drops what lies below 2^-22 of the largest of what it
    adds, whose size it takes from the exponents' fields, and a subnormal factor's
    field, that of 2^-126, is up to four times its value of 2^-128 and more. So each
    of the instructions, three of 32 k, drops up to 2^-20 of the magnitudes' sum on
    either side. (W1's products, of 8 and 2 bits, lose nothing at all: they are
    multiples of 2^-9 of the scales, and all sums below 2^15 of them.)"""
    torch, pg = env
    g = torch.Generator().manual_seed(H)
    dt = getattr(torch, dtype)
    x = some_tokens(torch, g, T, H, dt)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    log(f"[ends of the scales] T={T} k={k} E={E} H={H} F={F} {dtype}")
    b = Blocks(torch, g, E, H, F, 120, 120)
    want = b.run(pg, x, ids)
    assert bool(want.isfinite().all()) and bool((want != 0).any(1).all())
    for byte, power in ((0, 120), (1, 119)):
        b.s1[:] = byte
        assert torch.equal(b.run(pg, x * 2.0 ** power, ids), want)
    b.s1[:] = 252
    want = b.run(pg, x * 2.0 ** -125, ids)
    b.s1[:] = 127
    assert torch.equal(b.run(pg, x, ids), want) and bool(want.isfinite().all())
    # W2, with inner values scaled by W1's other part: by 2^126 from those of 2^-18 and less
    b.s1[:, :, :F] = 120
    b.s1[:, :, F:] = 100
    b.s2[:] = 126
    want = b.run(pg, x, ids)
    b.s1[:, :, F:] = 226
    b.s2[:] = 0
    level = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64)
    w1, w2 = level[b.c1[..., :H]], level[b.c2[..., :F]] / 2
    size = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for e in ids[t].tolist():
            s = w1[e] @ x[t].double()
            gate, up = s[:F] * 2.0 ** -7, s[F:] * 2.0 ** -27
            size[t] += w2[e].abs() @ (gate * torch.sigmoid(gate) * up).abs()
    allowed = 2 * 3 * -(-F // 32) * 2.0 ** -20 * size + want.double().abs() * torch.finfo(dt).eps
    got = b.run(pg, x, ids)
    assert bool(((got.double() - want.double()).abs() <= allowed).all())
    assert bool((want != 0).any(1).all())
    b.s1[:, :, F:] = 100
    b.s2[:] = 252
    assert torch.equal(b.run(pg, x, ids, torch.full((T, k), 2.0 ** -126)), want)


@pytest.mark.parametrize("T,k,E,H,F", BLOCK_SIZES)
def test_blocks_of_nan(env, T, k, E, H, F):
    """A block with the scale NaN spoils the outputs it is part of: all of the tokens
    that name its expert, of W2 their row's, and no others."""
    torch, pg = env
    g = torch.Generator().manual_seed(F)
    x = some_tokens(torch, g, T, H, torch.bfloat16)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    e = ids[0, 0].item()
    named = (ids == e).any(1)
    b = Blocks(torch, g, E, H, F, 120, 120)
    want = b.run(pg, x, ids)
    assert bool(want.isfinite().all())
    for row in (F // 2, F + F // 3):
        b.s1[e, 0, row, 1] = 255
        got = b.run(pg, x, ids)
        assert bool(got[named].isnan().all()) and torch.equal(got[~named], want[~named])
        b.s1[e, 0, row, 1] = 120
    b.s2[e, 0, H // 2, 1] = 255
    got = b.run(pg, x, ids)
    bad = torch.zeros(T, H, dtype=torch.bool)
    bad[named, H // 2] = True
    assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,F", [(33, 48), (64, 65), (161, 97)])
def test_unused_halves_of_bytes(env, H, F, dtype):
    """The high half of an odd row's last byte is no element: whatever it and a large
    scale would make, it counts for nothing."""
    torch, pg = env
    g = torch.Generator().manual_seed(H + F)
    T, k, E = 4, 2, 3
    x = some_tokens(torch, g, T, H, getattr(torch, dtype))
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    b = Blocks(torch, g, E, H, F, 122, 122)
    for c, s, K in ((b.c1, b.s1, H), (b.c2, b.s2, F)):
        if K % 2:  # the last block holds one element, a zero
            c[:, :, K - 1] = 0
            s[:, -1, :, K // 32 % 4] = 254
            c[:, :, K] = 0
    want = b.run(pg, x, ids)
    assert bool(want.isfinite().all()) and bool(want.any())
    for c, K in ((b.c1, H), (b.c2, F)):
        if K % 2:
            c[:, :, K] = torch.randint(5, 8, c[:, :, K].shape, generator=g)
    assert torch.equal(b.run(pg, x, ids), want)


@pytest.mark.parametrize("T,k,E,H,F", BLOCK_SIZES)
def test_blocks_beyond_the_range(env, T, k, E, H, F):
    """An element whose value is 2^128 counts as an infinity; 3 * 2^126, which both of
    the last scale bytes can make, as what it is."""
    torch, pg = env
    g = torch.Generator().manual_seed(H)
    x = some_tokens(torch, g, T, H, torch.bfloat16)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    e = ids[0, 0].item()
    named = (ids == e).any(1)
    b = Blocks(torch, g, E, H, F, 120, 120)
    f = F + F // 2  # a row whose second block is one element; no other row sees it
    b.c1[:, :, 40] = b.c1[:, f, 32:64] = 0

    def with_element(byte, code, token):
        b.s1[e, 0, f, 1], b.c1[e, f, 40] = byte, code
        x[:, 40] = token
        return b.run(pg, x, ids)

    want = with_element(127, 5, 1.0)
    assert bool(want.isfinite().all())
    for byte, code in ((253, 5), (254, 3)):
        assert torch.equal(with_element(byte, code, 2.0 ** -126), want)
    for byte, code in ((253, 6), (254, 4)):
        got = with_element(byte, code, 2.0 ** -126)
        assert not bool(got[named].isfinite().any()) and torch.equal(got[~named], want[~named])
