"""The operators around the experts of a mixture layer and the 8-bit integer
product, as measured cases: each in a plain torch form and through the calls
of this package.

  product   C = (A B^T) * scaleA[row] * scaleB[channel] + bias, A and B in 8-bit
            integers (i8gemm), or with the rows of A sorted by expert and one B
            an expert (i8gemm_grouped)
  quantize  rows to 8-bit integers with one scale a row (i8_quantize_rows)
  route     tokens sorted by expert and back with weights (expert_sort,
            expert_gather, expert_combine)
  unroute   the gradients of the two (expert_combine_grad, and expert_combine
            without weights, the gradient of expert_gather)
  experts   fp32 products of rows sorted by expert (sgemm_grouped) and, for a
            training step, their two gradients (sgemm_grouped with the other
            transpose, sgemm_grouped_outer)

A routed token carries `topk` expert numbers; a number outside [0, experts) is
a slot without an expert (a padding token, or an expert held elsewhere).
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
DEVICE = "cuda"


def listed():
    return [
        # one token through a square projection: the weights' bytes and the latency of a call
        {"name": "product_token", "op": "product", "M": 1, "N": 4096, "K": 4096, "groups": 0,
         "out": "bf16", "bias": False},
        # a prompt of odd length through a wide projection
        {"name": "product_prompt", "op": "product", "M": 4001, "N": 8192, "K": 4096, "groups": 0,
         "out": "fp16", "bias": True},
        # 64 tokens with 4 of 64 experts each: every expert's weights for a few rows
        {"name": "product_experts_decode", "op": "product", "M": 256, "N": 2048, "K": 2048,
         "groups": 64, "out": "bf16", "bias": False},
        # a batch of prompts over 32 experts, unevenly loaded
        {"name": "product_experts_prompt", "op": "product", "M": 16384, "N": 4096, "K": 2048,
         "groups": 32, "out": "fp32", "bias": False},
        # the activations of a few decoded tokens
        {"name": "quantize_decode", "op": "quantize", "M": 4, "K": 4096, "in": "bf16"},
        # a batch of prompts in fp32, rows of an odd length
        {"name": "quantize_prompt", "op": "quantize", "M": 16384, "K": 4092, "in": "fp32"},
        # a decode step of 32 sequences, 8 of 128 experts
        {"name": "route_decode", "op": "route", "T": 32, "topk": 8, "E": 128, "H": 2048,
         "type": "bf16", "absent": 0.0},
        # prompts, 4 of 64 experts, with padding tokens at the end
        {"name": "route_prompt", "op": "route", "T": 16384, "topk": 4, "E": 64, "H": 2048,
         "type": "bf16", "absent": 0.03},
        # a small training batch in fp32 with a width of 1000, 2 of 8 experts
        {"name": "unroute_small", "op": "unroute", "T": 500, "topk": 2, "E": 8, "H": 1000,
         "type": "fp32", "absent": 0.0},
        # a training batch, 8 of 64 experts
        {"name": "unroute_batch", "op": "unroute", "T": 8192, "topk": 8, "E": 64, "H": 2048,
         "type": "bf16", "absent": 0.03},
        # the forward products of a handful of rows in fp32
        {"name": "experts_few_rows", "op": "experts", "M": 100, "N": 1024, "K": 1024, "groups": 16,
         "backward": False},
        # both gradients of the experts' products in a training step
        {"name": "experts_backward", "op": "experts", "M": 8192, "N": 2048, "K": 1024,
         "groups": 16, "backward": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "product", "quantize", "route", "unroute", "experts"])
    if op == "product":
        groups = rng.choice([0, 0, _log(rng, 2, 128)])
        case = {"op": op, "M": _log(rng, 1, 16384), "N": _log(rng, 16, 8192),
                "K": _log(rng, 16, 8192), "groups": groups,
                "out": rng.choice(["fp32", "fp16", "bf16"]), "bias": rng.random() < 0.3}
        if rng.random() < 0.7:  # most models' widths are multiples of 64
            case["N"] = -(-case["N"] // 64) * 64
            case["K"] = -(-case["K"] // 64) * 64
        while case["M"] * case["N"] * case["K"] > 1 << 37:
            case["M"] = (case["M"] + 1) // 2
        while max(groups, 1) * case["N"] * case["K"] > 1 << 28:
            case["groups"] = groups = max(groups // 2, 1)
        return case
    if op == "quantize":
        case = {"op": op, "M": _log(rng, 1, 32768), "K": _log(rng, 1, 16384),
                "in": rng.choice(["fp32", "fp16", "bf16"])}
        while case["M"] * case["K"] > 1 << 26:
            case["M"] = (case["M"] + 1) // 2
        return case
    if op in ("route", "unroute"):
        E = _log(rng, 2, 256)
        case = {"op": op, "T": _log(rng, 1, 32768), "topk": rng.randint(1, min(8, E)), "E": E,
                "H": _log(rng, 16, 8192), "type": rng.choice(["fp32", "fp16", "bf16"]),
                "absent": rng.choice([0.0, 0.0, 0.05, 0.5])}
        while case["T"] * case["topk"] * case["H"] > 1 << 27:
            case["T"] = (case["T"] + 1) // 2
        return case
    case = {"op": op, "M": _log(rng, 1, 16384), "N": _log(rng, 16, 4096), "K": _log(rng, 16, 4096),
            "groups": _log(rng, 1, 64), "backward": rng.random() < 0.5}
    while case["M"] * case["N"] * case["K"] > 1 << 34:
        case["M"] = (case["M"] + 1) // 2
    while case["groups"] * case["N"] * case["K"] > 1 << 26:
        case["groups"] = (case["groups"] + 1) // 2
    return case


# --- inputs --------------------------------------------------------------------------------


def _counts(rows, groups, g):
    """Rows of each group: a router's uneven load, some groups without any."""
    share = torch.exp(0.7 * torch.randn(groups, generator=g, device=DEVICE))
    which = torch.multinomial(share, rows, replacement=True, generator=g)
    return torch.bincount(which, minlength=groups)


def _offsets(counts):
    off = torch.zeros(counts.numel() + 1, dtype=torch.int32, device=DEVICE)
    off[1:] = torch.cumsum(counts, 0)
    return off


def _int8(shape, g):
    """Bell-shaped 8-bit values, as weights and activations give."""
    out = torch.empty(shape, dtype=torch.int8, device=DEVICE)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i:i + (1 << 26)]
        part.copy_((40.0 * torch.randn(part.numel(), generator=g, device=DEVICE)).round_()
                   .clamp_(-127, 127))
    return out


def _padded(counts):
    """For the plain grouped products: the group and the place in it of every row, and the
    rows of the largest group."""
    group = torch.repeat_interleave(torch.arange(counts.numel(), device=DEVICE), counts)
    first = torch.cumsum(counts, 0) - counts
    place = torch.arange(group.numel(), device=DEVICE) - first[group]
    return group, place, max(1, int(counts.max()))


def _ids(case, g):
    """topk different experts of every token, uneven over the experts; a share of the tokens,
    the last ones, has none."""
    T, k, E = case["T"], case["topk"], case["E"]
    liking = 0.7 * torch.randn(E, generator=g, device=DEVICE)
    score = liking + torch.randn(T, E, generator=g, device=DEVICE)
    ids = torch.topk(score, k, dim=1).indices.to(torch.int32)
    ids[T - int(case["absent"] * T):] = -1
    weights = torch.softmax(torch.randn(T, k, generator=g, device=DEVICE), 1)
    return ids.contiguous(), weights


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    s = dict(case)
    randn = lambda *shape: torch.randn(shape, generator=g, device=DEVICE)  # noqa: E731
    if case["op"] == "product":
        M, N, K, G = case["M"], case["N"], case["K"], case["groups"]
        s["A"] = _int8((M, K), g)
        s["sA"] = (0.5 + torch.rand(M, generator=g, device=DEVICE)) / 40
        s["B"] = _int8((max(G, 1), N, K), g)
        s["sB"] = (0.5 + torch.rand(max(G, 1), N, generator=g, device=DEVICE)) / 40 / math.sqrt(K)
        s["biases"] = randn(max(G, 1), N) if case["bias"] else None
        s["C"] = torch.zeros(M, N, dtype=DTYPES[case["out"]], device=DEVICE)
        if G:
            counts = _counts(M, G, g)
            s["offsets"] = _offsets(counts)
            s["padded"] = _padded(counts)
    elif case["op"] == "quantize":
        M, K = case["M"], case["K"]
        # a few channels of a model's activations are much larger than the others
        large = 1 + 20 * (torch.rand(K, generator=g, device=DEVICE) < 0.01)
        s["X"] = (randn(M, K) * large).to(DTYPES[case["in"]])
        s["Q"] = torch.zeros(M, K, dtype=torch.int8, device=DEVICE)
        s["scale"] = torch.zeros(M, device=DEVICE)
    elif case["op"] in ("route", "unroute"):
        T, k, E, H, dt = case["T"], case["topk"], case["E"], case["H"], DTYPES[case["type"]]
        s["ids"], s["weights"] = _ids(case, g)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=DEVICE)
        s["row_of_slot"] = torch.zeros(T, k, dtype=torch.int32, device=DEVICE)
        s["Y"] = randn(T * k, H).to(dt)
        if case["op"] == "route":
            s["X"] = randn(T, H).to(dt)
            s["sorted"] = torch.zeros(T * k, H, dtype=dt, device=DEVICE)
            s["out"] = torch.zeros(T, H, dtype=dt, device=DEVICE)
            # more than the sort asks for at any of these sizes
            s["workspace"] = torch.empty(4 << 20, dtype=torch.uint8, device=DEVICE)
        else:
            s["dout"] = randn(T, H).to(dt)
            s["dsorted"] = randn(T * k, H).to(dt)
            s["dY"] = torch.zeros(T * k, H, dtype=dt, device=DEVICE)
            s["dweights"] = torch.zeros(T, k, device=DEVICE)
            s["dX"] = torch.zeros(T, H, dtype=dt, device=DEVICE)
            # the forward pass's order, which a training program holds
            key = torch.where((s["ids"] >= 0) & (s["ids"] < E), s["ids"], E).flatten().long()
            order = torch.sort(key, stable=True).indices
            row = torch.empty_like(order)
            row[order] = torch.arange(T * k, device=DEVICE)
            s["row_of_slot"] = torch.where(key < E, row, -1).to(torch.int32).view(T, k)
    else:
        M, N, K, G = case["M"], case["N"], case["K"], case["groups"]
        counts = _counts(M, G, g)
        s["offsets"] = _offsets(counts)
        s["padded"] = _padded(counts)
        s["A"] = randn(M, K)
        s["B"] = randn(G, K, N) / math.sqrt(K)
        if case["backward"]:
            s["dC"] = randn(M, N)
            s["dA"] = torch.zeros(M, K, device=DEVICE)
            s["dB"] = torch.zeros(G, K, N, device=DEVICE)
        else:
            s["C"] = torch.zeros(M, N, device=DEVICE)
    return s


# --- the calls of this package -------------------------------------------------------------


def _run_own(s):
    import precision_gemm_amd as pg
    if s["op"] == "product":
        M, N, K, G = s["M"], s["N"], s["K"], s["groups"]
        if G:
            pg.i8gemm_grouped(M, N, K, G, s["offsets"], s["A"], K, s["sA"], s["B"], K, N * K,
                              s["sB"], s["biases"], s["C"], N)
        else:
            pg.i8gemm(M, N, K, s["A"], K, s["sA"], s["B"], K, s["sB"], s["biases"], s["C"], N)
        return s["C"]
    if s["op"] == "quantize":
        M, K = s["M"], s["K"]
        pg.i8_quantize_rows(M, K, s["X"], K, s["Q"], K, s["scale"])
        return {"Q": s["Q"], "scale": s["scale"]}
    if s["op"] == "route":
        T, k, E, H = s["T"], s["topk"], s["E"], s["H"]
        pg.expert_sort(T, k, E, s["ids"], s["offsets"], s["row_of_slot"], s["workspace"])
        pg.expert_gather(T, k, H, s["X"], H, s["row_of_slot"], s["sorted"], H)
        pg.expert_combine(T, k, H, s["Y"], H, s["row_of_slot"], s["weights"], s["out"], H)
        return {"offsets": s["offsets"], "row_of_slot": s["row_of_slot"], "sorted": s["sorted"],
                "out": s["out"]}
    if s["op"] == "unroute":
        T, k, H = s["T"], s["topk"], s["H"]
        pg.expert_combine_grad(T, k, H, s["dout"], H, s["Y"], H, s["row_of_slot"], s["weights"],
                               s["dY"], H, s["dweights"])
        pg.expert_combine(T, k, H, s["dsorted"], H, s["row_of_slot"], None, s["dX"], H)
        return {"dY": s["dY"], "dweights": s["dweights"], "dX": s["dX"]}
    M, N, K, G = s["M"], s["N"], s["K"], s["groups"]
    if not s["backward"]:
        pg.sgemm_grouped(0, M, N, K, G, s["offsets"], 1.0, s["A"], K, s["B"], N, K * N, 0.0,
                         s["C"], N)
        return s["C"]
    pg.sgemm_grouped(1, M, K, N, G, s["offsets"], 1.0, s["dC"], N, s["B"], N, K * N, 0.0,
                     s["dA"], K)
    pg.sgemm_grouped_outer(K, N, M, G, s["offsets"], 1.0, s["A"], K, s["dC"], N, 0.0, s["dB"], N,
                           K * N)
    return {"dA": s["dA"], "dB": s["dB"]}


# --- the plain forms -----------------------------------------------------------------------


def _pad(rows, padded, groups):
    """Rows sorted by group as [groups, most rows, width], zeros behind each group's last."""
    group, place, most = padded
    out = rows.new_zeros(groups, most, rows.shape[1])
    out[group, place] = rows
    return out


def _run_plain(s):
    if s["op"] == "product":
        # sums of 8-bit products pass 2^24, the whole numbers that 32 bits hold exactly
        G, dt = s["groups"], s["C"].dtype
        if G:
            group, place, _ = s["padded"]
            a = _pad(s["A"].double(), s["padded"], G)
            acc = torch.bmm(s["B"].double(), a.transpose(1, 2).contiguous())[group, :, place]
            c = acc.float() * s["sA"][:, None] * s["sB"][group]
            if s["bias"]:
                c = c + s["biases"][group]
        else:
            acc = torch.mm(s["A"].double(), s["B"][0].double().t())
            c = acc.float() * s["sA"][:, None] * s["sB"]
            if s["bias"]:
                c = c + s["biases"]
        return c.to(dt)
    if s["op"] == "quantize":
        x = s["X"].float()
        # both quotients in 64 bits: in 32 they round onto the border between two integers
        scale = (x.abs().amax(1).double() / 127).float().clamp_min(torch.finfo(torch.float32).tiny)
        q = torch.round(x.double() / scale.double()[:, None])
        return {"Q": q.to(torch.int8), "scale": scale}
    if s["op"] == "route":
        T, k, E, H = s["T"], s["topk"], s["E"], s["H"]
        ids = s["ids"].flatten().long()
        held = (ids >= 0) & (ids < E)
        key = torch.where(held, ids, E)
        order = torch.sort(key, stable=True).indices
        row = torch.empty_like(order)
        row[order] = torch.arange(T * k, device=ids.device)
        offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=ids.device))
        gathered = torch.where(held[order][:, None], s["X"][order // k], s["sorted"])
        y = torch.where(held[:, None], s["Y"][row].float(), 0.0).view(T, k, H)
        out = (y * s["weights"][:, :, None]).sum(1)
        return {"offsets": offsets.to(torch.int32),
                "row_of_slot": torch.where(held, row, -1).to(torch.int32).view(T, k),
                "sorted": gathered, "out": out.to(s["X"].dtype)}
    if s["op"] == "unroute":
        T, k, H, dt = s["T"], s["topk"], s["H"], s["Y"].dtype
        rows = s["row_of_slot"].flatten().long()
        held = (rows >= 0)[:, None]
        dout = s["dout"].float()
        per_slot = (dout[:, None, :] * s["weights"][:, :, None]).view(T * k, H).to(dt)
        # slots without an expert write behind the last row, which is then cut off
        dY = torch.cat([s["dY"], s["dY"].new_zeros(1, H)])
        dY[torch.where(held[:, 0], rows, T * k)] = per_slot
        y = torch.where(held, s["Y"][rows.clamp_min(0)].float(), 0.0).view(T, k, H)
        dweights = (y * dout[:, None, :]).sum(2)
        dX = torch.where(held, s["dsorted"][rows.clamp_min(0)].float(), 0.0).view(T, k, H).sum(1)
        return {"dY": dY[:T * k], "dweights": dweights, "dX": dX.to(dt)}
    G = s["groups"]
    group, place, _ = s["padded"]
    a = _pad(s["A"], s["padded"], G)
    if not s["backward"]:
        return torch.bmm(a, s["B"])[group, place]
    dc = _pad(s["dC"], s["padded"], G)
    return {"dA": torch.bmm(dc, s["B"].transpose(1, 2).contiguous())[group, place],
            "dB": torch.bmm(a.transpose(1, 2).contiguous(), dc)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    """Each input read once, each output written once; of the experts' weights those that the
    rows can reach."""
    if case["op"] == "product":
        M, N, K, G = case["M"], case["N"], case["K"], max(case["groups"], 1)
        size = DTYPES[case["out"]].itemsize
        reached = min(G, M)
        return {"bytes": M * K + 4 * M + reached * (N * K + 4 * N * (1 + case["bias"])) + M * N * size,
                "flops": 2 * M * N * K}
    if case["op"] == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (DTYPES[case["in"]].itemsize + 1) + 4 * M, "flops": 3 * M * K}
    if case["op"] in ("route", "unroute"):
        T, k, H = case["T"], case["topk"], case["H"]
        size = DTYPES[case["type"]].itemsize
        held = (T - int(case["absent"] * T)) * k
        if case["op"] == "route":
            # X once and its sorted rows; the experts' rows and the sum
            values = (T - int(case["absent"] * T)) * H + held * H + held * H + T * H
            return {"bytes": values * size + 4 * (2 * T * k + held + case["E"] + 1),
                    "flops": 2 * held * H}
        values = (T - int(case["absent"] * T)) * H + 3 * held * H + T * H
        return {"bytes": values * size + 4 * (2 * T * k + 2 * held), "flops": 4 * held * H}
    M, N, K, G = case["M"], case["N"], case["K"], case["groups"]
    reached = min(G, M)
    if not case["backward"]:
        return {"bytes": 4 * (M * K + reached * K * N + M * N), "flops": 2 * M * N * K}
    return {"bytes": 4 * (2 * M * K + M * N + (reached + G) * K * N), "flops": 4 * M * N * K}


# --- 64-bit values -------------------------------------------------------------------------


def exact(case, seed):
    """The definitions in 64 bits, expert by expert and slot by slot."""
    s = prepare(case, seed)
    if case["op"] == "product":
        G, B = case["groups"], s["B"]
        out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=DEVICE)
        ends = s["offsets"].tolist() if G else [0, case["M"]]
        for e in range(max(G, 1)):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                a = s["A"][lo:hi].to(torch.float64) * s["sA"][lo:hi, None].to(torch.float64)
                out[lo:hi] = (a @ B[e].to(torch.float64).T) * s["sB"][e].to(torch.float64)
                if case["bias"]:
                    out[lo:hi] += s["biases"][e].to(torch.float64)
        return out
    if case["op"] == "quantize":
        x = s["X"].to(torch.float64)
        # the scale is a 32-bit number, and the integers go by that number
        peak = x.abs().max(dim=1).values
        scale = torch.maximum(peak / 127, torch.full_like(peak, 2.0 ** -126)).to(torch.float32)
        q = torch.empty(case["M"], case["K"], dtype=torch.int8, device=DEVICE)
        for lo in range(0, case["M"], 4096):
            q[lo:lo + 4096] = (x[lo:lo + 4096] / scale[lo:lo + 4096, None].to(torch.float64)) \
                .round().to(torch.int8)
        return {"Q": q, "scale": scale.to(torch.float64)}
    if case["op"] == "route":
        T, k, E, H = case["T"], case["topk"], case["E"], case["H"]
        flat = s["ids"].cpu().flatten().tolist()
        held = [i for i, e in enumerate(flat) if 0 <= e < E]
        sequence = sorted(held, key=lambda i: flat[i])  # stable
        row_of = [-1] * (T * k)
        for r, i in enumerate(sequence):
            row_of[i] = r
        offsets = [0] * (E + 1)
        for i in held:
            offsets[flat[i] + 1] += 1
        for e in range(E):
            offsets[e + 1] += offsets[e]
        rows = torch.tensor(row_of, device=DEVICE).view(T, k)
        src = torch.tensor(sequence, dtype=torch.int64, device=DEVICE)
        gathered = s["sorted"].to(torch.float64)
        gathered[:len(sequence)] = s["X"].to(torch.float64)[src // k]
        out = torch.zeros(T, H, dtype=torch.float64, device=DEVICE)
        for j in range(k):
            has = rows[:, j] >= 0
            out[has] += s["weights"][has, j, None].to(torch.float64) * \
                s["Y"][rows[has, j]].to(torch.float64)
        return {"offsets": torch.tensor(offsets, dtype=torch.int32, device=DEVICE),
                "row_of_slot": rows.to(torch.int32), "sorted": gathered, "out": out}
    if case["op"] == "unroute":
        T, k, H = case["T"], case["topk"], case["H"]
        rows = s["row_of_slot"].long()
        dout = s["dout"].to(torch.float64)
        dY = s["dY"].to(torch.float64)
        dw = torch.zeros(T, k, dtype=torch.float64, device=DEVICE)
        dX = torch.zeros(T, H, dtype=torch.float64, device=DEVICE)
        for j in range(k):
            has = rows[:, j] >= 0
            r = rows[has, j]
            dY[r] = s["weights"][has, j, None].to(torch.float64) * dout[has]
            dw[has, j] = (dout[has] * s["Y"][r].to(torch.float64)).sum(1)
            dX[has] += s["dsorted"][r].to(torch.float64)
        return {"dY": dY, "dweights": dw, "dX": dX}
    ends = s["offsets"].tolist()
    A, B = s["A"].to(torch.float64), s["B"].to(torch.float64)
    if not case["backward"]:
        out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=DEVICE)
        for e in range(case["groups"]):
            out[ends[e]:ends[e + 1]] = A[ends[e]:ends[e + 1]] @ B[e]
        return out
    dC = s["dC"].to(torch.float64)
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for e in range(case["groups"]):
        lo, hi = ends[e], ends[e + 1]
        dA[lo:hi] = dC[lo:hi] @ B[e].T
        dB[e] = A[lo:hi].T @ dC[lo:hi]
    return {"dA": dA, "dB": dB}
