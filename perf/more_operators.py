"""Norms, 4-bit products and the mixture layer of a few tokens, as measured cases:
each in a plain torch form and through the calls of this package.

  norm     the residual's addition, the root-mean-square norm and its rounding to 8-bit
           integers with a scale a row (rms_norm_i8)
  train    the same norm in the input's type and its gradients (rms_norm, rms_norm_grad)
  round    rows to 4-bit floating point, blocks of 32 sharing a power of two, and back
           (mx4_quantize_rows, mx4_dequantize_rows)
  product  C = A B^T + bias, A and B in those blocks (mx4gemm), or with the rows of A
           sorted by expert and one B an expert (mx4gemm_grouped)
  layer    out = sum_j w_j W2_e (silu(W1g_e x) * (W1u_e x)) over a token's experts
           (expert_layer): weights in the tokens' type, in 8-bit integers with a scale a
           channel, or in the 4-bit blocks

A 4-bit value is sign, two bits of exponent and one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4 or
6; element k of a row is the low (even k) or high half of byte k / 2. A block's scale is
2^(byte - 127); four blocks' bytes stand together, then the rows, then the next four.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
DEVICE = "cuda"
EPS = 1e-6


def listed():
    return [
        # the tokens of a small decode step before an 8-bit projection: the latency of a call
        {"name": "norm_decode", "op": "norm", "M": 4, "K": 4096, "type": "bf16"},
        # a batch of prompts before an 8-bit projection
        {"name": "norm_prompt", "op": "norm", "M": 16384, "K": 4096, "type": "bf16"},
        # a small training batch in fp32 with a width of 1000
        {"name": "train_small", "op": "train", "M": 500, "K": 1000, "type": "fp32"},
        # a training batch
        {"name": "train_batch", "op": "train", "M": 16384, "K": 2048, "type": "bf16"},
        # a few tokens' activations in 4 bits
        {"name": "round_decode", "op": "round", "M": 16, "K": 4096, "type": "bf16"},
        # a batch of prompts in fp32, rows that end inside a block
        {"name": "round_prompt", "op": "round", "M": 8192, "K": 4092, "type": "fp32"},
        # one token through a square projection: the weights' bytes and the latency of a call
        {"name": "product_token", "op": "product", "M": 1, "N": 4096, "K": 4096, "groups": 0,
         "out": "bf16", "bias": False},
        # a prompt of odd length through a wide projection
        {"name": "product_prompt", "op": "product", "M": 4001, "N": 8192, "K": 4096, "groups": 0,
         "out": "fp16", "bias": True},
        # a batch of prompts over 32 experts, unevenly loaded
        {"name": "product_experts", "op": "product", "M": 16384, "N": 4096, "K": 2048,
         "groups": 32, "out": "fp32", "bias": False},
        # one token through 8 of 128 experts
        {"name": "layer_token", "op": "layer", "T": 1, "topk": 8, "E": 128, "H": 2048, "F": 768,
         "type": "bf16", "weights": "same"},
        # a decode step of 16 sequences, 4 of 64 experts in 8 bits
        {"name": "layer_i8", "op": "layer", "T": 16, "topk": 4, "E": 64, "H": 2048, "F": 1024,
         "type": "fp16", "weights": "i8"},
        # a decode step of 64 sequences, 8 of 128 experts in 4 bits
        {"name": "layer_mx4", "op": "layer", "T": 64, "topk": 8, "E": 128, "H": 2048, "F": 768,
         "type": "bf16", "weights": "mx4"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "train", "round", "product", "product", "layer", "layer"])
    types = ["fp32", "fp16", "bf16"]
    if op in ("norm", "train", "round"):
        case = {"op": op, "M": _log(rng, 1, 32768),
                "K": _log(rng, 1, 8192 if op == "train" else 16384), "type": rng.choice(types)}
        while case["M"] * case["K"] > 1 << 25:
            case["M"] = (case["M"] + 1) // 2
        return case
    if op == "product":
        groups = rng.choice([0, 0, _log(rng, 2, 128)])
        case = {"op": op, "M": _log(rng, 1, 16384), "N": _log(rng, 16, 8192),
                "K": _log(rng, 16, 8192), "groups": groups, "out": rng.choice(types),
                "bias": rng.random() < 0.3}
        if rng.random() < 0.7:  # most models' widths are multiples of 64
            case["N"] = -(-case["N"] // 64) * 64
            case["K"] = -(-case["K"] // 64) * 64
        while case["M"] * case["N"] * case["K"] > 1 << 36:
            case["M"] = (case["M"] + 1) // 2
        while max(groups, 1) * case["N"] * case["K"] > 1 << 28:
            case["groups"] = groups = max(groups // 2, 1)
        return case
    E = _log(rng, 2, 128)
    case = {"op": op, "T": _log(rng, 1, 64), "topk": rng.randint(1, min(8, E)), "E": E,
            "H": _log(rng, 64, 4096), "F": _log(rng, 64, 4096), "type": rng.choice(types),
            "weights": rng.choice(["same", "i8", "mx4"])}
    if rng.random() < 0.7:
        case["H"] = -(-case["H"] // 64) * 64
        case["F"] = -(-case["F"] // 64) * 64
    while case["E"] * case["H"] * case["F"] > 1 << 27:
        case["F"] = (case["F"] + 1) // 2
    return case


# --- inputs --------------------------------------------------------------------------------


def _counts(rows, groups, g):
    """Rows of each group: a router's uneven load, some groups without any."""
    share = torch.exp(0.7 * torch.randn(groups, generator=g, device=DEVICE))
    which = torch.multinomial(share, rows, replacement=True, generator=g)
    return torch.bincount(which, minlength=groups)


def _mx4(groups, rows, K, size, g):
    """Rows in blocks as weights and activations give them: bell-shaped values of about
    `size`, and scales around it. Packed bytes [groups, rows, K / 2] and scales [groups, K /
    128, rows, 4], both rounded up."""
    near = (2.2 * torch.randn(1 << 17, generator=g, device=DEVICE)).abs()
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEVICE)
    code = torch.bucketize(near, border)
    code += 8 * torch.randint(0, 2, code.shape, generator=g, device=DEVICE)
    pool = (code[0::2] + 16 * code[1::2]).to(torch.uint8)
    width = (K + 1) // 2
    packed = torch.empty(groups * rows * width, dtype=torch.uint8, device=DEVICE)
    for i in range(0, packed.numel(), 1 << 26):
        part = packed[i:i + (1 << 26)]
        part.copy_(pool[torch.randint(0, 1 << 16, part.shape, generator=g, device=DEVICE,
                                      dtype=torch.int32)])
    packed = packed.view(groups, rows, width)
    if K % 2:
        packed[:, :, -1] &= 15
    middle = 127 + round(math.log2(size / 2.2))
    scale = torch.randint(middle - 1, middle + 2, (groups, (K + 127) // 128, rows, 4),
                          generator=g, device=DEVICE, dtype=torch.uint8)
    return packed, scale


def _ids(case, g):
    """topk different experts of every token, uneven over the experts."""
    T, k, E = case["T"], case["topk"], case["E"]
    liking = 0.7 * torch.randn(E, generator=g, device=DEVICE)
    score = liking + torch.randn(T, E, generator=g, device=DEVICE)
    ids = torch.topk(score, k, dim=1).indices.to(torch.int32)
    return ids.contiguous(), torch.softmax(torch.randn(T, k, generator=g, device=DEVICE), 1)


def _weights(case, rows, K, g):
    """Experts' weights [E, rows, K] and their scales."""
    E, size = case["E"], 1 / math.sqrt(K)
    if case["weights"] == "mx4":
        return _mx4(E, rows, K, size, g)
    i8 = case["weights"] == "i8"
    w = torch.empty(E, rows, K, dtype=torch.int8 if i8 else DTYPES[case["type"]], device=DEVICE)
    flat = w.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i:i + (1 << 26)]
        v = torch.randn(part.numel(), generator=g, device=DEVICE)
        part.copy_(v.mul_(40).round_().clamp_(-127, 127) if i8 else v.mul_(size))
    if not i8:
        return w, None
    return w, (0.5 + torch.rand(E, rows, generator=g, device=DEVICE)) * (size / 40)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    s = dict(case)
    randn = lambda *shape: torch.randn(shape, generator=g, device=DEVICE)  # noqa: E731
    if case["op"] in ("norm", "train", "round"):
        M, K, dt = case["M"], case["K"], DTYPES[case["type"]]
        # a few channels of a model's activations are much larger than the others
        large = 1 + 20 * (torch.rand(K, generator=g, device=DEVICE) < 0.01)
        s["X"] = (randn(M, K) * large).to(dt)
        if case["op"] == "round":
            s["Q"] = torch.zeros(M, (K + 1) // 2, dtype=torch.uint8, device=DEVICE)
            s["scale"] = torch.zeros((K + 127) // 128, M, 4, dtype=torch.uint8, device=DEVICE)
            s["Y"] = torch.zeros(M, K, dtype=dt, device=DEVICE)
            return s
        s["R"] = randn(M, K).to(dt)
        s["weight"] = 1 + 0.2 * randn(K)
        s["H"] = torch.zeros(M, K, dtype=dt, device=DEVICE)
        if case["op"] == "norm":
            s["Q"] = torch.zeros(M, K, dtype=torch.int8, device=DEVICE)
            s["scale"] = torch.zeros(M, device=DEVICE)
        else:
            s["dY"], s["dH"] = randn(M, K).to(dt), randn(M, K).to(dt)
            s["Y"], s["dX"] = torch.zeros_like(s["H"]), torch.zeros_like(s["H"])
            s["dweight"] = torch.zeros(K, device=DEVICE)
            # more than the gradient asks for at any of these sizes
            s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEVICE)
    elif case["op"] == "product":
        M, N, K, G = case["M"], case["N"], case["K"], case["groups"]
        A, sA = _mx4(1, M, K, 1.0, g)
        s["A"], s["sA"] = A[0], sA[0]
        s["B"], s["sB"] = _mx4(max(G, 1), N, K, 1 / math.sqrt(K), g)
        s["biases"] = randn(max(G, 1), N) if case["bias"] else None
        s["C"] = torch.zeros(M, N, dtype=DTYPES[case["out"]], device=DEVICE)
        if G:
            counts = _counts(M, G, g)
            s["offsets"] = torch.zeros(G + 1, dtype=torch.int32, device=DEVICE)
            s["offsets"][1:] = torch.cumsum(counts, 0)
    else:
        T, H, F, dt = case["T"], case["H"], case["F"], DTYPES[case["type"]]
        s["ids"], s["mix"] = _ids(case, g)
        s["X"] = randn(T, H).to(dt)
        s["W1"], s["scale1"] = _weights(case, 2 * F, H, g)
        s["W2"], s["scale2"] = _weights(case, H, F, g)
        s["out"] = torch.zeros(T, H, dtype=dt, device=DEVICE)
        # more than the layer asks for at any of these sizes
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEVICE)
    return s


# --- the calls of this package -------------------------------------------------------------


def _run_own(s):
    import precision_gemm_amd as pg
    if s["op"] == "norm":
        M, K = s["M"], s["K"]
        pg.rms_norm_i8(M, K, s["X"], K, s["R"], K, s["weight"], EPS, s["H"], K, s["Q"], K,
                       s["scale"])
        return {"H": s["H"], "Q": s["Q"], "scale": s["scale"]}
    if s["op"] == "train":
        M, K = s["M"], s["K"]
        pg.rms_norm(M, K, s["X"], K, s["R"], K, s["weight"], EPS, s["H"], K, s["Y"], K)
        pg.rms_norm_grad(M, K, s["dY"], K, s["H"], K, s["weight"], EPS, s["dH"], K, s["dX"], K,
                         s["dweight"], s["workspace"])
        return {"H": s["H"], "Y": s["Y"], "dX": s["dX"], "dweight": s["dweight"]}
    if s["op"] == "round":
        M, K, width = s["M"], s["K"], s["Q"].shape[1]
        pg.mx4_quantize_rows(M, K, s["X"], K, s["Q"], width, s["scale"], M)
        pg.mx4_dequantize_rows(M, K, s["Q"], width, s["scale"], M, s["Y"], K)
        return s["Y"]
    if s["op"] == "product":
        M, N, K, G, width = s["M"], s["N"], s["K"], s["groups"], s["A"].shape[1]
        if G:
            pg.mx4gemm_grouped(M, N, K, G, s["offsets"], s["A"], width, s["sA"], M, s["B"], width,
                               N * width, s["sB"], N, s["sB"].stride(0), s["biases"], s["C"], N)
        else:
            pg.mx4gemm(M, N, K, s["A"], width, s["sA"], M, s["B"], width, s["sB"], N, s["biases"],
                       s["C"], N)
        return s["C"]
    H, F = s["H"], s["F"]
    w1, w2 = s["W1"].shape[2], s["W2"].shape[2]
    pg.expert_layer(s["T"], s["topk"], s["E"], H, F, s["X"], H, s["ids"], s["mix"], s["W1"], w1,
                    2 * F * w1, s["scale1"], s["W2"], w2, H * w2, s["scale2"], s["out"], H,
                    s["workspace"])
    return s["out"]


# --- the plain forms -----------------------------------------------------------------------


def _values(packed, scale, K):
    """Packed bytes [..., rows, K / 2] and scales [..., K / 128, rows, 4] as fp32."""
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=packed.device)
    level = torch.cat([level, -level])
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)[..., :K]
    power = (scale.to(torch.int32) << 23).view(torch.float32)
    power = power.transpose(-3, -2).flatten(-2).repeat_interleave(32, -1)[..., :K]
    return level[code.int()] * power


def _place(group, groups):
    """The place of every row within its group, and the rows of the largest group; `group`
    need not be sorted."""
    order = torch.sort(group, stable=True).indices
    counts = torch.bincount(group, minlength=groups)
    first = torch.cumsum(counts, 0) - counts
    place = torch.empty_like(group)
    place[order] = torch.arange(group.numel(), device=group.device) - first[group[order]]
    return place, max(1, int(counts.max()))


def _normed(s):
    h = (s["X"].float() + s["R"].float()).to(s["X"].dtype)
    f = h.float()
    rstd = torch.rsqrt((f * f).mean(1, keepdim=True) + EPS)
    return h, f, rstd


def _run_plain(s):
    if s["op"] == "norm":
        h, f, rstd = _normed(s)
        t = f * s["weight"]
        # both quotients in 64 bits: in 32 they round onto the border between two integers
        step = (t.abs().amax(1).double() / 127).float().clamp_min(torch.finfo(torch.float32).tiny)
        q = torch.round(t.double() / step.double()[:, None])
        return {"H": h, "Q": q.to(torch.int8), "scale": step * rstd[:, 0]}
    if s["op"] == "train":
        h, f, rstd = _normed(s)
        y = f * s["weight"] * rstd
        dy = s["dY"].float()
        wdy = dy * s["weight"]
        dx = s["dH"].float() + rstd * (wdy - f * rstd * rstd * (wdy * f).mean(1, keepdim=True))
        dt = h.dtype
        return {"H": h, "Y": y.to(dt), "dX": dx.to(dt), "dweight": (dy * f * rstd).sum(0)}
    if s["op"] == "round":
        M, K = s["M"], s["K"]
        x = torch.nn.functional.pad(s["X"].float(), (0, -K % 32)).view(M, -1, 32)
        power = torch.exp2(torch.frexp(x.abs().amax(2, keepdim=True)).exponent - 3.0)
        v = x.abs() / power
        # steps of a half below 2, of one below 4, of two from there on; ties to the even code
        v = torch.where(v < 2, torch.round(2 * v) / 2,
                        torch.where(v < 4, torch.round(v), 2 * torch.round(v / 2)))
        return (v.clamp_max(6) * power * x.sign()).flatten(1)[:, :K].to(s["X"].dtype)
    if s["op"] == "product":
        K, G = s["K"], s["groups"]
        a, b = _values(s["A"], s["sA"], K), _values(s["B"], s["sB"], K)
        if not G:
            c = torch.mm(a, b[0].t())
            if s["bias"]:
                c = c + s["biases"]
            return c.to(s["C"].dtype)
        ends = s["offsets"][1:].contiguous()
        row = torch.arange(s["M"], dtype=torch.int32, device=a.device)
        group = torch.searchsorted(ends, row, right=True)
        place, most = _place(group, G)
        padded = a.new_zeros(G, most, K)
        padded[group, place] = a
        c = torch.bmm(b, padded.transpose(1, 2).contiguous())[group, :, place]
        if s["bias"]:
            c = c + s["biases"][group]
        return c.to(s["C"].dtype)
    T, k, H, F = s["T"], s["topk"], s["H"], s["F"]
    reached, group = torch.unique(s["ids"].flatten().long(), return_inverse=True)
    place, most = _place(group, reached.numel())
    if s["weights"] == "mx4":
        w1 = _values(s["W1"][reached], s["scale1"][reached], H)
        w2 = _values(s["W2"][reached], s["scale2"][reached], F)
    else:
        w1, w2 = s["W1"][reached].float(), s["W2"][reached].float()
        if s["weights"] == "i8":
            w1 = w1 * s["scale1"][reached][:, :, None]
            w2 = w2 * s["scale2"][reached][:, :, None]
    x = w1.new_zeros(reached.numel(), most, H)
    x[group, place] = s["X"].float().repeat_interleave(k, 0)
    h = torch.bmm(w1, x.transpose(1, 2).contiguous())
    gate, up = h[:, :F], h[:, F:]
    y = torch.bmm(w2, gate / (1 + torch.exp(-gate)) * up)[group, :, place]
    return (y.view(T, k, H) * s["mix"][:, :, None]).sum(1).to(s["out"].dtype)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    """Each input read once, each output written once; of the experts' weights those that the
    tokens can reach (of a layer, as many as even choices reach on average)."""
    if case["op"] in ("norm", "train", "round"):
        M, K, size = case["M"], case["K"], DTYPES[case["type"]].itemsize
        if case["op"] == "norm":  # x, r, the sum and 8 bits
            return {"bytes": M * K * (3 * size + 1) + 4 * (M + K), "flops": 8 * M * K}
        if case["op"] == "train":  # x, r, h, y; dy, dh, h, dx
            return {"bytes": M * K * 8 * size + 8 * K, "flops": 16 * M * K}
        return {"bytes": M * K * 2 * size + 2 * M * (K // 2 + K // 32), "flops": 4 * M * K}
    if case["op"] == "product":
        M, N, K, G = case["M"], case["N"], case["K"], max(case["groups"], 1)
        reached = min(G, M)
        return {"bytes": (M + reached * N) * K * 17 / 32 + 4 * reached * N * case["bias"] +
                M * N * DTYPES[case["out"]].itemsize, "flops": 2 * M * N * K}
    T, k, E, H, F = (case[n] for n in ("T", "topk", "E", "H", "F"))
    size = DTYPES[case["type"]].itemsize
    reached = E * (1 - (1 - k / E) ** T)
    each = {"same": size, "i8": 1, "mx4": 17 / 32}[case["weights"]]
    return {"bytes": reached * 3 * H * F * each + 2 * T * H * size + 8 * T * k,
            "flops": 6 * T * k * H * F}


# --- 64-bit values -------------------------------------------------------------------------


def _exact_values(packed, scale, K):
    """One matrix's 4-bit values from sign, exponent and mantissa, in 64 bits."""
    rows = packed.shape[0]
    code = torch.empty(rows, 2 * packed.shape[1], dtype=torch.int64, device=DEVICE)
    code[:, 0::2] = packed.long() % 16
    code[:, 1::2] = packed.long() // 16
    code = code[:, :K]
    sign = 1.0 - 2.0 * (code // 8).double()
    power, last = code // 2 % 4, (code % 2).double()
    value = torch.where(power == 0, last / 2, (1 + last / 2) * torch.pow(2.0, (power - 1).double()))
    k = torch.arange(K, device=DEVICE)
    block = k // 32
    byte = scale[block // 4, :, block % 4].T.double()
    return sign * value * torch.pow(2.0, byte - 127)


def exact(case, seed):
    """The definitions in 64 bits, expert by expert."""
    s = prepare(case, seed)
    if case["op"] in ("norm", "train"):
        K = case["K"]
        h = (s["X"].double() + s["R"].double()).to(s["X"].dtype)
        x, w = h.double(), s["weight"].double()
        rstd = 1 / (x.square().sum(1) / K + EPS).sqrt()
        if case["op"] == "norm":
            # the products are 32-bit numbers and so is their step, and the integers go by those
            t = (x * w).float().double()
            step = (t.abs().max(1).values / 127).clamp(min=2.0 ** -126).float().double()
            return {"H": x, "Q": (t / step[:, None]).round().to(torch.int8), "scale": step * rstd}
        dy, xhat = s["dY"].double(), x * rstd[:, None]
        along = (dy * w * xhat).sum(1) / K
        return {"H": x, "Y": xhat * w, "dweight": (dy * xhat).sum(0),
                "dX": s["dH"].double() + rstd[:, None] * (dy * w - xhat * along[:, None])}
    if case["op"] == "round":
        x, K = s["X"].double(), case["K"]
        out = torch.empty_like(x)
        level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEVICE)
        for k in range(0, K, 32):
            part = x[:, k:k + 32]
            power = torch.pow(2.0, torch.floor(torch.log2(part.abs().max(1).values)) - 2)
            v = part.abs() / power[:, None]
            near = (v[:, :, None] - level).abs()
            # of two equally near levels the one with the even code
            near = near + 1e-9 * (torch.arange(8, device=DEVICE) % 2)
            out[:, k:k + 32] = level[near.argmin(2)] * power[:, None] * part.sign()
        return out
    if case["op"] == "product":
        G, K = case["groups"], case["K"]
        a = _exact_values(s["A"], s["sA"], K)
        out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=DEVICE)
        ends = s["offsets"].tolist() if G else [0, case["M"]]
        for e in range(max(G, 1)):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                out[lo:hi] = a[lo:hi] @ _exact_values(s["B"][e], s["sB"][e], K).T
                if case["bias"]:
                    out[lo:hi] += s["biases"][e].double()
        return out
    T, H, F = case["T"], case["H"], case["F"]
    x = s["X"].double()
    out = torch.zeros(T, H, dtype=torch.float64, device=DEVICE)
    for e in range(case["E"]):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        if case["weights"] == "mx4":
            w1 = _exact_values(s["W1"][e], s["scale1"][e], H)
            w2 = _exact_values(s["W2"][e], s["scale2"][e], F)
        else:
            w1, w2 = s["W1"][e].double(), s["W2"][e].double()
            if case["weights"] == "i8":
                w1 = w1 * s["scale1"][e].double()[:, None]
                w2 = w2 * s["scale2"][e].double()[:, None]
        h = x[t] @ w1.T
        hidden = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]
        out.index_add_(0, t, (hidden @ w2.T) * s["mix"][t, j].double()[:, None])
    return out
