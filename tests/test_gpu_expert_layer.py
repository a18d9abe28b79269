"""The experts' layer of a few tokens against 64-bit values.

Tolerances: a product's sum over K runs in the matrix units over 8 waves, each
instruction of 4 k (fp32) or 32 k adding to the sum so far with an error of at
most 2^-22 of the magnitudes' sum, and the waves' sums are added (8 roundings).
The inner values carry 16 bits (fp32 layers: 24) and one or two roundings of
exp, the quotient and the product."""
import sys

import pytest

pytestmark = pytest.mark.gpu
TYPES = ["float32", "float16", "bfloat16"]
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


class Weights:
    """E x rows x K weights of a kind, rows `pad` elements (bytes) apart."""

    def __init__(self, torch, g, E, rows, K, kind, dt, pad=0, shift=0):
        size = K ** -0.5
        self.scale = None
        if kind == "mx4":
            width = (K + 1) // 2
            code = torch.randint(0, 16, (E, rows, 2 * width), generator=g)
            nb, words = -(-K // 32), -(-K // 128)
            near = 127 - max(1, round((K ** 0.5)).bit_length())
            byte = torch.randint(near - 1, near + 2, (E, rows, nb), generator=g)
            s = torch.full((E, words, rows, 4), 255, dtype=torch.uint8)
            for b in range(nb):
                s[:, b // 4, :, b % 4] = byte[:, :, b].to(torch.uint8)
            self.scale = s.cuda()
            level = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64)
            self.host = level[code[..., :K]] * \
                (2.0 ** (byte.double() - 127)).repeat_interleave(32, -1)[..., :K]
            w = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
        elif kind == "i8":
            w = torch.randint(-128, 128, (E, rows, K), generator=g, dtype=torch.int8)
            s = (0.5 + torch.rand(E, rows, generator=g)) * size / 64
            self.scale = s.cuda()
            self.host = w.double() * s.double()[..., None]
        else:
            w = (torch.randn(E, rows, K, generator=g) * size).to(dt)
            self.host = w.double()
        width = w.shape[2]
        self.ld = max(1, width + pad)
        self.stride = rows * self.ld + pad
        store = torch.zeros(shift + E * self.stride + 1, dtype=w.dtype)
        if width and rows:
            view = store[shift:].as_strided((E, rows, width), (self.stride, self.ld, 1),
                                            shift)
            view.copy_(w)
        self.t = store.cuda()[shift:]


def layer_case(env, T, k, E, H, F, dtype="bfloat16", kind="same", ids=None, mix=True, pads=(0, 0, 0, 0),
               shift=0, ids64=False, seed=0, x=None):
    torch, pg = env
    log(f"[layer] T={T} k={k} E={E} H={H} F={F} {dtype} {kind} mix={mix} pads={pads} shift={shift}")
    g = torch.Generator().manual_seed(seed + T + 10 * k + H + 3 * F)
    dt = getattr(torch, dtype)
    if x is None:
        x = torch.randn(T, H, generator=g).to(dt)
    ldx, ldo = H + pads[0], H + pads[1]
    xs = torch.zeros(shift + T * ldx, dtype=dt)
    xs[shift:].view(T, ldx)[:, :H] = x
    X = xs.cuda()[shift:]
    if ids is None:
        ids = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    ids = ids.to(torch.int64 if ids64 else torch.int32).contiguous()
    weights = torch.rand(T, k, generator=g) + 0.1
    W1 = Weights(torch, g, E, 2 * F, H, kind, dt, pads[2], shift)
    W2 = Weights(torch, g, E, H, F, kind, dt, pads[3], shift)
    out = torch.full((T, ldo), 7.0, dtype=dt, device="cuda")
    ws = torch.full((pg.expert_layer_workspace_size(T, k, H, F, dt),), 255, dtype=torch.uint8).cuda()
    pg.expert_layer(T, k, E, H, F, X, ldx, ids.cuda(), weights.cuda() if mix else None, W1.t, W1.ld,
                    W1.stride, W1.scale, W2.t, W2.ld, W2.stride, W2.scale, out, ldo, ws)
    torch.cuda.synchronize()
    per = 4 if kind == "same" and dtype == "float32" else 32
    error = lambda K: ((K // (8 * per) + 2) * (4 if per == 4 else 1) + 12) * 2.0 ** -22  # noqa: E731
    keep = 2.0 ** -22 if dtype == "float32" else 2.0 ** -16
    want = torch.zeros(T, H, dtype=torch.float64)
    allowed = torch.zeros(T, H, dtype=torch.float64)
    size = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        v = x[t].double()
        for j in range(k):
            e = ids[t, j].item()
            if not 0 <= e < E:
                continue
            m = weights[t, j].double().item() if mix else 1.0
            s, ds = W1.host[e] @ v, error(H) * (W1.host[e].abs() @ v.abs())
            gate, up, dg, du = s[:F], s[F:], ds[:F], ds[F:]
            silu = gate * torch.sigmoid(gate)
            a = silu * up
            # |silu'| < 1.1
            da = 1.1 * dg * up.abs() + silu.abs() * du + 1.1 * dg * du + a.abs() * (8 * 2.0 ** -24 + keep)
            y = W2.host[e] @ a
            sy = W2.host[e].abs() @ a.abs()
            want[t] += m * y
            size[t] += m * sy
            allowed[t] += m * (W2.host[e].abs() @ da + error(F) * sy)
    allowed += (k + 2) * 2.0 ** -24 * size
    f = torch.finfo(dt)
    allowed += (want.abs() + allowed) * f.eps / 2 + f.smallest_normal * f.eps / 2
    got = out.cpu().double()
    worst = ((got[:, :H] - want).abs() - allowed).max().item()
    assert worst <= 0, worst
    assert bool((got[:, H:] == 7).all())
    return out


KINDS = ["same", "i8", "mx4"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H,F", [(1, 1, 1, 1, 1), (1, 2, 4, 64, 48), (3, 2, 8, 200, 100),
                                       (16, 4, 8, 128, 257), (5, 8, 64, 512, 256),
                                       (33, 2, 3, 96, 40), (1, 8, 128, 1024, 384)])
def test_layer(env, T, k, E, H, F, dtype, kind):
    layer_case(env, T, k, E, H, F, dtype, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H,F", [(16, 2, 20, 960, 480), (64, 8, 64, 64, 416),
                                       (64, 8, 128, 64, 800), (64, 8, 128, 1600, 32),
                                       (1, 8, 16, 4160, 96), (2, 4, 8, 4160, 1056),
                                       (8, 1, 2, 2080, 1312)])
def test_every_tile(env, T, k, E, H, F, dtype, kind):
    """Sizes at which the choice of tiles, of waves that share one and of the second
    kernel falls each way."""
    layer_case(env, T, k, E, H, F, dtype, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", TYPES)
def test_odd_rows(env, dtype, kind):
    """Rows off any boundary, odd lengths, gaps between rows and experts."""
    layer_case(env, 4, 2, 5, 129, 67, dtype, kind, pads=(3, 5, 1, 7), shift=1)
    layer_case(env, 2, 3, 4, 255, 127, dtype, kind, pads=(1, 0, 3, 0), shift=0)


@pytest.mark.parametrize("kind", KINDS)
def test_many_rows_of_one_expert(env, kind):
    """More columns than one pass takes, an expert named twice by a token, experts
    that nobody names, int64 ids."""
    torch, _ = env
    ids = torch.zeros(100, 2, dtype=torch.int64)
    ids[:, 1] = torch.arange(100) % 3 * 3
    layer_case(env, 100, 2, 7, 80, 50, "bfloat16", kind, ids=ids, ids64=True)
    ids = torch.full((50, 1), 2)
    layer_case(env, 50, 1, 3, 64, 33, "float16", kind, ids=ids)
    ids = torch.zeros(20, 1, dtype=torch.int64)
    layer_case(env, 20, 1, 1, 64, 33, "float32", kind, ids=ids, mix=False)


@pytest.mark.parametrize("ids64", [False, True])
def test_slots_without_expert(env, ids64):
    torch, _ = env
    ids = torch.tensor([[0, -1], [-1, -1], [9, 2], [3, 3], [4, 2 ** 31 - 1], [-2 ** 31, 1]])
    out = layer_case(env, 6, 2, 4, 72, 40, "float32", ids=ids, ids64=ids64)
    assert bool((out[1, :72] == 0).all()) and bool((out[4, :72] == 0).all())
    out = layer_case(env, 3, 1, 4, 72, 40, "bfloat16", ids=torch.full((3, 1), -1), ids64=ids64)
    assert bool((out == 0).all())


def test_most_slots(env):
    """EXPERT_LAYER_MAX_SLOTS of them over 1024 experts."""
    torch, pg = env
    layer_case(env, 256, 8, 1024, 40, 24, "float16", "i8")
    layer_case(env, 2048, 1, 300, 24, 40, "bfloat16", "same")


def test_empty(env):
    torch, pg = env
    x = torch.ones(3, 8).cuda()
    out = torch.full((3, 8), 7.0).cuda()
    ids = torch.zeros(3, 1, dtype=torch.int32).cuda()
    ws = torch.zeros(1 << 16, dtype=torch.uint8).cuda()
    # no inner values: the sum over none
    pg.expert_layer(3, 1, 2, 8, 0, x, 8, ids, None, x, 8, 0, None, x, 1, 0, None, out, 8, ws)
    assert bool((out == 0).all())
    out.fill_(7)
    w = torch.ones(64).cuda()  # (the weights of one expert, shared)
    pg.expert_layer(0, 1, 2, 8, 4, x, 8, ids, None, w, 8, 0, None, w, 4, 0, None, out, 8, ws)
    pg.expert_layer(3, 1, 2, 0, 4, x, 8, ids, None, w, 8, 0, None, w, 4, 0, None, out, 8, ws)
    assert bool((out == 7).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_stay_with_their_token(env, dtype):
    """A token with an infinity or NaN spoils no other."""
    torch, pg = env
    T, H, F, E = 5, 64, 48, 2
    g = torch.Generator().manual_seed(1)
    dt = getattr(torch, dtype)
    x = torch.randn(T, H, generator=g).to(dt)
    x[1, 3], x[3, 60] = float("inf"), float("nan")
    ids = torch.tensor([[0], [0], [0], [0], [1]]).int().cuda()
    for kind in KINDS:
        W1 = Weights(torch, g, E, 2 * F, H, kind, dt)
        W2 = Weights(torch, g, E, H, F, kind, dt)
        outs = []
        for v in (x, torch.nan_to_num(x, 0, 0, 0)):
            out = torch.zeros(T, H, dtype=dt).cuda()
            ws = torch.zeros(pg.expert_layer_workspace_size(T, 1, H, F, dt), dtype=torch.uint8).cuda()
            pg.expert_layer(T, 1, E, H, F, v.cuda(), H, ids, None, W1.t, W1.ld, W1.stride, W1.scale,
                            W2.t, W2.ld, W2.stride, W2.scale, out, H, ws)
            outs.append(out.cpu())
        assert torch.equal(outs[0][[0, 2, 4]], outs[1][[0, 2, 4]])
        assert bool(outs[0][3].isnan().all()) and not bool(outs[0][1].isfinite().any())


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_subnormal_weights(env, dtype):
    """Weights below the type's normal numbers count as what they are."""
    torch, pg = env
    T, H, F = 3, 64, 48
    g = torch.Generator().manual_seed(2)
    dt = getattr(torch, dtype)
    small = 2.0 ** -17 if dtype == "float16" else 2.0 ** -129
    x = (torch.randn(T, H, generator=g) * (2.0 ** 12 if dtype == "float16" else 2.0 ** 124)).to(dt)
    w1 = (torch.randn(2 * F, H, generator=g) * small).to(dt)
    w2 = (torch.randn(H, F, generator=g) * small).to(dt)
    ids = torch.zeros(T, 1, dtype=torch.int32).cuda()
    weight = min(1 / small, 2.0 ** 100)
    mix = torch.full((T, 1), weight).cuda()
    out = torch.zeros(T, H, dtype=dt).cuda()
    ws = torch.zeros(pg.expert_layer_workspace_size(T, 1, H, F, dt), dtype=torch.uint8).cuda()
    pg.expert_layer(T, 1, 1, H, F, x.cuda(), H, ids, mix, w1.cuda(), H, 0, None, w2.cuda(), F, 0,
                    None, out, H, ws)
    s = x.double() @ w1.double().T
    a = s[:, :F] * torch.sigmoid(s[:, :F]) * s[:, F:]
    want = a @ w2.double().T * weight
    size = a.abs() @ w2.double().abs().T * weight
    f = torch.finfo(dt)
    # The sums' errors are those of test_layer at these sizes: 14 * 2^-22 of magnitudes
    # (some 8 times a value here) twice, and the inner values' 2^-16.
    allowed = size * (2.0 ** -16 + 2 * 8 * 14 * 2.0 ** -22) + want.abs() * f.eps
    assert float(w1.double().abs().max()) < f.smallest_normal * 4 and bool(out.any())
    assert bool(((out.cpu().double() - want).abs() <= allowed).all())


@pytest.mark.parametrize("kind", KINDS)
def test_graph_and_streams(env, kind):
    """Captured after a norm and replayed with other ids between; the same on two
    streams with a workspace each; calls repeat their bits."""
    torch, pg = env
    T, k, E, H, F = 12, 4, 16, 256, 128
    g = torch.Generator().manual_seed(9)
    dt = torch.bfloat16
    W1, W2 = Weights(torch, g, E, 2 * F, H, kind, dt), Weights(torch, g, E, H, F, kind, dt)
    X, R, w = torch.randn(T, H, generator=g).to(dt).cuda(), torch.randn(T, H, generator=g).to(dt).cuda(), \
        torch.ones(H).cuda()
    ids = torch.zeros(T, k, dtype=torch.int32).cuda()
    mix = torch.rand(T, k, generator=g).cuda()
    size = pg.expert_layer_workspace_size(T, k, H, F, dt)

    def buffers():
        return torch.zeros_like(X), torch.zeros_like(X), torch.zeros_like(X), \
            torch.full((size,), 255, dtype=torch.uint8).cuda()

    def step(Hs, Y, out, ws):
        pg.rms_norm(T, H, X, H, R, H, w, 1e-6, Hs, H, Y, H)
        pg.expert_layer(T, k, E, H, F, Y, H, ids, mix, W1.t, W1.ld, W1.stride, W1.scale, W2.t, W2.ld,
                        W2.stride, W2.scale, out, H, ws)

    a, b = buffers(), buffers()
    step(*a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*a)
    for i in range(4):
        ids.copy_(torch.rand(T, E, generator=g).argsort(1)[:, :k].int())
        a[2].zero_()
        a[3].fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = a[2].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(*b)
        step(*a)
        torch.cuda.synchronize()
        assert torch.equal(got, a[2]) and torch.equal(got, b[2]) and bool(got.any())


@pytest.mark.parametrize("kind", ["same", "i8", "mx4"])
def test_next_to_the_sorted_path(env, kind):
    """expert_sort, expert_gather, sgemm_grouped and expert_combine give the same
    layer from the weights' values."""
    torch, pg = env
    T, k, E, H, F = 10, 2, 6, 160, 96
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, H, generator=g)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k].int().contiguous()
    mix = torch.rand(T, k, generator=g)
    W1, W2 = Weights(torch, g, E, 2 * F, H, kind, torch.float32), Weights(torch, g, E, H, F, kind,
                                                                          torch.float32)
    out = torch.zeros(T, H).cuda()
    ws = torch.zeros(pg.expert_layer_workspace_size(T, k, H, F, torch.float32), dtype=torch.uint8).cuda()
    X, I, Mx = x.cuda(), ids.cuda(), mix.cuda()
    pg.expert_layer(T, k, E, H, F, X, H, I, Mx, W1.t, W1.ld, W1.stride, W1.scale, W2.t, W2.ld, W2.stride,
                    W2.scale, out, H, ws)
    S = T * k
    off, row = torch.zeros(E + 1, dtype=torch.int32).cuda(), torch.zeros(S, dtype=torch.int32).cuda()
    xs, y, z, o2 = (torch.zeros(s).cuda() for s in ((S, H), (S, 2 * F), (S, H), (T, H)))
    w1, w2 = W1.host.float().cuda(), W2.host.float().cuda()
    pg.expert_sort(T, k, E, I, off, row, None)
    pg.expert_gather(T, k, H, X, H, row, xs, H)
    pg.sgemm_grouped(1, S, 2 * F, H, E, off, 1.0, xs, H, w1, H, 2 * F * H, 0.0, y, 2 * F)
    a = (torch.nn.functional.silu(y[:, :F]) * y[:, F:]).contiguous()
    pg.sgemm_grouped(1, S, H, F, E, off, 1.0, a, F, w2, F, H * F, 0.0, z, H)
    pg.expert_combine(T, k, H, z, H, row, Mx, o2, H)
    # both are within 2^-17 of the sum of magnitudes, which is some 40 times a typical value
    assert float((out - o2).abs().max()) <= 2.0 ** -16 * 40 * float(o2.abs().max())
