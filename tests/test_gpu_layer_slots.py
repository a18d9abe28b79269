"""The experts' layer with the most slots, and its groups of slots behind the 512
whose ids a wave holds, against 64-bit values; experts far apart, to the bit."""
import pytest

from test_gpu_expert_layer import Weights, layer_case, log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_gemm_amd as pg
    pg._load()
    yield torch, pg
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["same", "i8", "mx4"])
@pytest.mark.parametrize("ids64", [False, True])
def test_all_slots_of_one_expert(env, kind, ids64):
    """2048 slots, 128 groups of 16."""
    torch, _ = env
    layer_case(env, 2048, 1, 1, 40, 24, "bfloat16", kind, ids=torch.zeros(2048, 1), ids64=ids64)
    layer_case(env, 256, 8, 3, 40, 24, "float32", kind, ids=torch.full((256, 8), 2), ids64=ids64)


@pytest.mark.parametrize("kind", ["same", "mx4"])
@pytest.mark.parametrize("ids64", [False, True])
def test_groups_behind_the_held_ids(env, kind, ids64):
    """1500 slots: three experts with hundreds each, one with 16 slots among the
    first 512 and its other groups behind them, one with all of its 33 behind them,
    and slots without an expert on either side."""
    torch, _ = env
    g = torch.Generator().manual_seed(4)
    ids = torch.tensor([5, 70, 99])[torch.randint(0, 3, (1500,), generator=g)]
    ids[torch.randperm(512, generator=g)[:16]] = 33
    late = 512 + torch.randperm(988, generator=g)
    ids[late[:45]] = 33
    ids[late[45:78]] = 0
    ids[late[78:90]] = -1
    ids[late[90:100]] = 100
    ids[torch.nonzero(ids[:512] == 5)[:7, 0]] = -3
    layer_case(env, 1500, 1, 100, 40, 24, "float16", kind, ids=ids[:, None], ids64=ids64)
    layer_case(env, 500, 3, 100, 40, 24, "float32", kind, ids=ids.view(500, 3), ids64=ids64)


@pytest.mark.parametrize("kind", ["same", "i8", "mx4"])
def test_far_experts_to_the_bit(env, kind):
    """Six tokens through the experts 1 and 4 of five, side by side and 2^31 + 64
    bytes apart: the same kernels with the same split, so the same bits."""
    torch, pg = env
    T, E, H, F = 6, 5, 256, 160
    dt = torch.bfloat16
    g = torch.Generator().manual_seed(3)
    W1, W2 = Weights(torch, g, E, 2 * F, H, kind, dt), Weights(torch, g, E, H, F, kind, dt)
    x = torch.randn(T, H, generator=g).to(dt).cuda()
    ids = torch.tensor([[4], [1], [4], [4], [1], [4]], dtype=torch.int32).cuda()
    stride = 2 ** 30 + 64 if kind == "same" else 2 ** 31 + 64  # elements; bytes of the others
    log(f"[far experts] {kind}")
    far = []
    for W, rows in ((W1, 2 * F), (W2, H)):
        t = torch.zeros((E - 1) * stride + rows * W.ld, dtype=W.t.dtype, device="cuda")
        for e in range(E):
            t[e * stride:e * stride + rows * W.ld] = W.t[e * W.stride:e * W.stride + rows * W.ld]
        far.append(t)
    outs = []
    for w1, d1, w2, d2 in ((W1.t, W1.stride, W2.t, W2.stride), (far[0], stride, far[1], stride)):
        out = torch.zeros(T, H, dtype=dt).cuda()
        ws = torch.zeros(pg.expert_layer_workspace_size(T, 1, H, F, dt), dtype=torch.uint8).cuda()
        pg.expert_layer(T, 1, E, H, F, x, H, ids, None, w1, W1.ld, d1, W1.scale, w2, W2.ld, d2,
                        W2.scale, out, H, ws)
        outs.append(out)
    assert bool(outs[0].any(1).all()) and torch.equal(*outs)
