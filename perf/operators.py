"""Cases of the serving operators of a quantized feed-forward block: one-token products with packed 4-bit
weights, tokens sorted by expert and back (with the gradients), and the experts' products.

``run`` computes a case in plain torch operations (``own`` false) or through the framework's operators (``own``
true), on what ``prepare`` made; ``exact`` gives the same outputs from the definitions in 64 bits.

Formulas. A packed weight row o holds codes q in 0..15 (eight per 32-bit word, in-feature k at bits
4 (k % 8) of word k / 8), and per group g = k / 128 a step and a zero point: w[o, k] = (q - z[o, g]) step[o, g].

* gemv:     Y = X w^T (+ bias); gated: rows 0..O/2-1 give a, rows O/2..O-1 give b, Y = silu(a) b.
* sort:     slots s = t k + j of ids [T, k]; rows r = 0.. in order of (expert, slot) of the slots with an id in
            0..E-1; offsets[e] = first row of expert e, order[r] = slot (-1 behind the last row), pos[t, j] = row
            (-1 where the id names no expert).
* gather:   Xs[r] = X[order[r] / k], divided by the expert's scale vector where one is given.
* combine:  Y[t] = sum_j weight[t, j] Ys[pos[t, j]]; its gradients dYs[r] = weight dY[t], dweight = <dY[t], Ys[r]>;
            the gather's gradient dX[t] = sum_j dXs[pos[t, j]] / scales[e].
* experts:  Y[r] = Xs[r] w_e^T for the rows r of expert e; gated as above.
"""
import torch

own = False

GROUP = 128


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's projection at 4096 features: the smallest call, latency counts
        {"name": "gemv 1x4096-4096", "op": "gemv", "M": 1, "K": 4096, "O": 4096, "gated": False, "bias": True},
        # a decode step of the largest down projection
        {"name": "gemv 1x28672-8192", "op": "gemv", "M": 1, "K": 28672, "O": 8192, "gated": False, "bias": False},
        # a few sequences decoded together through a gate and up projection, an odd number of groups
        {"name": "gemv gated 5x4224-21512", "op": "gemv", "M": 5, "K": 4224, "O": 21512, "gated": True, "bias": False},
        # one decode step's tokens to their experts
        {"name": "dispatch 8 tokens", "op": "dispatch", "T": 8, "k": 2, "E": 8, "K": 4096, "scaled": False,
         "pad": 0, "ids": 64},
        # a prefill's tokens to many experts, with padded tokens and a scale vector per expert
        {"name": "dispatch 8192 tokens", "op": "dispatch", "T": 8192, "k": 8, "E": 128, "K": 4096, "scaled": True,
         "pad": 500, "ids": 32},
        # back from the experts: a decode batch, and a prefill of odd length
        {"name": "combine 33 tokens", "op": "combine", "T": 33, "k": 4, "E": 16, "K": 4096, "pad": 3},
        {"name": "combine 6001 tokens", "op": "combine", "T": 6001, "k": 8, "E": 64, "K": 4096, "pad": 0},
        # both gradients, of a short batch and of a long one
        {"name": "gradients 250 tokens", "op": "grad", "T": 250, "k": 2, "E": 8, "K": 4096, "scaled": True, "pad": 6},
        {"name": "gradients 8192 tokens", "op": "grad", "T": 8192, "k": 4, "E": 32, "K": 4096, "scaled": False,
         "pad": 0},
        # the experts' products of a decode batch: every expert has a row or two, gate and up
        {"name": "experts 8 tokens", "op": "experts", "T": 8, "k": 2, "E": 8, "K": 4096, "O": 28672, "gated": True},
        # a middling batch through the down projections, tens of rows for each expert
        {"name": "experts 300 tokens", "op": "experts", "T": 300, "k": 2, "E": 8, "K": 14336, "O": 4096,
         "gated": False},
        # a prefill through the gate and up projections of many small experts
        {"name": "experts 4096 tokens", "op": "experts", "T": 4096, "k": 4, "E": 32, "K": 4096, "O": 4096,
         "gated": True},
    ]


def _spread(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "dispatch", "combine", "grad", "experts", "experts"])
    if op == "gemv":
        gated = rng.random() < 0.4
        K = GROUP * _spread(rng, 1, 224)
        O = 2 * _spread(rng, 32, max(64, min(14336, 110_000_000 // K)))
        return {"op": op, "M": rng.randint(1, 8), "K": K, "O": O, "gated": gated,
                "bias": not gated and rng.random() < 0.5}
    if op == "experts":
        gated = rng.random() < 0.5
        T, k = _spread(rng, 1, 2048), rng.choice([1, 2, 4, 8])
        E = max(k, _spread(rng, 4, 64))
        K = GROUP * _spread(rng, 4, 64)
        most = min(28672, 250_000_000 // (E * K), 270_000_000_000 // (T * k * K), 200_000 // E)
        O = 8 * _spread(rng, 32, max(64, most // 8))
        return {"op": op, "T": T, "k": k, "E": E, "K": K, "O": O, "gated": gated}
    T, k = _spread(rng, 1, 6000), rng.choice([1, 2, 3, 4, 6, 8])
    case = {"op": op, "T": T, "k": k, "E": max(k, _spread(rng, 4, 256)), "K": 8 * _spread(rng, 64, 896),
            "pad": rng.randint(0, T // 4)}
    if op != "combine":
        case["scaled"] = rng.random() < 0.5
    if op == "dispatch":
        case["ids"] = rng.choice([32, 64])
    return case


# ------------------------------------------------------------------------------------------------ inputs
def _quantized(rows, K, gen):
    """Codes, steps and zero points of normal weights, rounded to nearest in groups of 128."""
    codes = torch.empty(rows, K // 8, dtype=torch.int32, device="cuda")
    steps = torch.empty(rows, K // GROUP, device="cuda")
    zeros = torch.empty(rows, K // GROUP, device="cuda")
    shifts = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    chunk = max(1, (1 << 27) // K)
    for a in range(0, rows, chunk):
        n = min(chunk, rows - a)
        w = torch.randn(n, K // GROUP, GROUP, device="cuda", generator=gen).mul_(K ** -0.5)
        low, high = torch.aminmax(w, dim=2, keepdim=True)
        step = ((high - low) / 15).clamp(min=1e-5)
        zero = torch.round(-low / step)
        q = (torch.round(w.div_(step)).add_(zero)).clamp_(0, 15).to(torch.int32)
        codes[a:a + n] = (q.view(n, K // 8, 8) << shifts).sum(2, dtype=torch.int32)
        steps[a:a + n], zeros[a:a + n] = step[..., 0], zero[..., 0]
    return codes, steps, zeros


def _routed(case, gen):
    """A router's picks and weights: every token's k likeliest of E experts, some experts liked more than others;
    the last `pad` tokens of the batch are padding and name no expert."""
    T, k, E = case["T"], case["k"], case["E"]
    logits = torch.randn(T, E, device="cuda", generator=gen)
    logits += 0.7 * torch.randn(E, device="cuda", generator=gen)
    value, ids = torch.topk(logits, k, dim=1)
    ids[T - case.get("pad", 0):] = -1
    return ids, torch.softmax(value, 1)


def _sorted(ids, E):
    """offsets, order, pos of the ids, for preparing inputs and for the plain form."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    ranked, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ranked, torch.arange(E + 1, device=ids.device))
    rows = torch.arange(flat.numel(), device=ids.device)
    pos = torch.empty_like(rows)
    pos[order] = torch.where(rows < offsets[E], rows, -1)
    order = torch.where(rows < offsets[E], order, -1)
    return offsets.int(), order.int(), pos.int().view(ids.shape)


def _like_activations(gen, *shape):
    """bf16 activations with a few channels of large magnitude."""
    x = torch.randn(*shape, device="cuda", generator=gen)
    x[..., torch.randperm(shape[-1], device="cuda", generator=gen)[:max(1, shape[-1] // 200)]] *= 20
    return x.bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, K = case["op"], case["K"]
    s = {"case": case}
    if op == "gemv":
        s["X"] = _like_activations(gen, case["M"], K)
        s["codes"], s["steps"], s["zeros"] = _quantized(case["O"], K, gen)
        s["bias"] = torch.randn(case["O"], device="cuda", generator=gen).bfloat16() if case["bias"] else None
        return s
    T, k, E = case["T"], case["k"], case["E"]
    ids, weights = _routed(case, gen)
    s["weights"] = weights
    n = T * k
    if op == "experts":
        s["offsets"], _, _ = _sorted(ids, E)
        s["X"] = _like_activations(gen, n, K)
        codes, steps, zeros = _quantized(E * case["O"], K, gen)
        s["codes"], s["steps"], s["zeros"] = (t.view(E, case["O"], -1) for t in (codes, steps, zeros))
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())  # the plain form's padding
        return s
    s["scales"] = torch.rand(E, K, device="cuda", generator=gen).add_(0.5) if case.get("scaled") else None
    if op == "dispatch":
        s["ids"] = ids.int() if case["ids"] == 32 else ids
        s["X"] = _like_activations(gen, T, K)
        s["Xs"] = torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")  # rows behind the last stay as they are
        return s
    s["ids"] = ids.int()
    s["offsets"], s["order"], s["pos"] = _sorted(ids, E)
    s["Ys"] = torch.randn(n, K, device="cuda", generator=gen).bfloat16()
    if op == "grad":
        s["dY"] = torch.randn(T, K, device="cuda", generator=gen).bfloat16()
        s["dXs"] = torch.randn(n, K, device="cuda", generator=gen).bfloat16()
        s["dYs"] = torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from weight_only_quantization_act_b200 import awq

    case = s["case"]
    op = case["op"]
    if op == "gemv":
        return awq.w4a16_gemv(s["X"], s["codes"], s["steps"], s["zeros"], bias=s["bias"], gated=case["gated"])
    if op == "experts":
        if "workspace" not in s:  # kept from pass to pass, as a serving loop keeps it
            s["workspace"] = awq.w4a16_experts_workspace(s["codes"], s["X"].shape[0])
        return awq.w4a16_experts(s["X"], s["offsets"], s["codes"], s["steps"], s["zeros"], gated=case["gated"],
                                 workspace=s["workspace"])
    if op == "dispatch":
        sort = awq.expert_sort(s["ids"], case["E"])
        Xs = awq.expert_gather(s["X"], sort, scales=s["scales"], out=s["Xs"])
        return {"offsets": sort.offsets, "order": sort.order, "pos": sort.pos, "Xs": Xs}
    sort = awq.ExpertSort(s["offsets"], s["order"], s["pos"])
    if op == "combine":
        return awq.expert_combine(s["Ys"], sort, weights=s["weights"])
    dYs, dweights = awq.expert_combine_backward(s["dY"], s["Ys"], sort, s["weights"], out=s["dYs"])
    return {"dYs": dYs, "dweights": dweights, "dX": awq.expert_gather_backward(s["dXs"], sort, scales=s["scales"])}


def _plain_weights(codes, steps, zeros):
    shifts = torch.arange(0, 32, 4, device=codes.device, dtype=torch.int32)
    q = ((codes[..., None] >> shifts) & 15).float().view(*steps.shape, GROUP)
    return ((q - zeros[..., None]) * steps[..., None]).view(*steps.shape[:-1], -1)


def _plain_gate(P, gated):
    if not gated:
        return P
    a, b = P.chunk(2, dim=-1)
    return a / (1 + torch.exp(-a)) * b


def _plain_rows(s, source):
    """source[pos] in 32 bits as [T, k, K], zeros where a slot has no row."""
    pos = s["pos"].long()
    return torch.where((pos >= 0)[..., None], source[pos.clamp(min=0)].float(), 0.0)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "gemv":
        P = s["X"].float() @ _plain_weights(s["codes"], s["steps"], s["zeros"]).T
        if s["bias"] is not None:
            P = P + s["bias"].float()
        return _plain_gate(P, case["gated"]).bfloat16()
    if op == "experts":
        offsets = s["offsets"].long()
        rows = torch.arange(s["X"].shape[0], device=s["X"].device)
        expert = torch.searchsorted(offsets, rows, right=True) - 1
        at = expert * s["most"] + rows - offsets[expert]
        padded = torch.zeros(case["E"] * s["most"], case["K"], device=s["X"].device)
        padded[at] = s["X"].float()
        W = _plain_weights(s["codes"], s["steps"], s["zeros"])
        P = torch.bmm(padded.view(case["E"], s["most"], -1), W.transpose(1, 2))
        return _plain_gate(P.view(case["E"] * s["most"], -1)[at], case["gated"]).bfloat16()
    if op == "dispatch":
        offsets, order, pos = _sorted(s["ids"], case["E"])
        slot = order.clamp(min=0).long()
        x = s["X"].float()[slot // case["k"]]
        if s["scales"] is not None:
            x = x / s["scales"][s["ids"].reshape(-1)[slot].long().clamp(min=0)]
        return {"offsets": offsets, "order": order, "pos": pos,
                "Xs": torch.where((order >= 0)[:, None], x, 0.0).bfloat16()}
    if op == "combine":
        return (s["weights"][..., None] * _plain_rows(s, s["Ys"])).sum(1).bfloat16()
    order = s["order"].long()
    slot = order.clamp(min=0)
    dYs = s["weights"].reshape(-1)[slot, None] * s["dY"].float()[slot // case["k"]]
    dweights = (s["dY"].float()[:, None] * _plain_rows(s, s["Ys"])).sum(2)
    dx = _plain_rows(s, s["dXs"])
    if s["scales"] is not None:
        dx = dx / s["scales"][s["ids"].long().clamp(min=0)]
    return {"dYs": torch.where((order >= 0)[:, None], dYs, 0.0).bfloat16(), "dweights": dweights,
            "dX": dx.sum(1).bfloat16()}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    """Bytes that have to be read once or written once, and operations. The rows of a routed batch: those of its
    real tokens; of the experts' weights, those of the experts that can have a row."""
    op, K = case["op"], case["K"]
    if op == "gemv":
        M, O = case["M"], case["O"]
        weights = O * K // 2 + 8 * O * (K // GROUP)
        out = O // 2 if case["gated"] else O
        return {"bytes": weights + 2 * M * K + 2 * M * out + (2 * O if case["bias"] else 0), "flops": 2 * M * K * O}
    T, k, E = case["T"], case["k"], case["E"]
    n, real = T * k, T - case.get("pad", 0)
    if op == "experts":
        O = case["O"]
        out = O // 2 if case["gated"] else O
        return {"bytes": min(E, n) * (O * K // 2 + 8 * O * (K // GROUP)) + 2 * n * (K + out) + 4 * (E + 1),
                "flops": 2 * n * K * O}
    scales = 4 * min(E, real * k) * K if case.get("scaled") else 0
    if op == "dispatch":
        return {"bytes": n * (case["ids"] // 8) + 8 * n + 4 * (E + 1) + 2 * real * K + 2 * real * k * K + scales,
                "flops": real * k * K if case["scaled"] else 0}
    if op == "combine":
        return {"bytes": 8 * n + 2 * real * k * K + 2 * T * K, "flops": 2 * real * k * K}
    return {"bytes": (8 * n + 2 * real * K + 4 * real * k * K + 4 * n) + (8 * n + 2 * real * k * K + 2 * T * K) + scales,
            "flops": (5 if case["scaled"] else 4) * real * k * K}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_product(x, codes, steps, zeros, bias, gated):
    """x w^T of one weight in 64 bits, nibble by nibble."""
    x = x.double()
    K = x.shape[1]
    total = torch.zeros(x.shape[0], codes.shape[0], dtype=torch.float64, device=x.device)
    half = 4096 if K > 4096 else K
    for k0 in range(0, K, half):
        k1 = min(K, k0 + half)
        words = codes[:, k0 // 8:k1 // 8].long() & 0xFFFFFFFF
        w = torch.empty(codes.shape[0], k1 - k0, dtype=torch.float64, device=x.device)
        for i in range(8):
            w[:, i::8] = ((words >> (4 * i)) % 16).double()
        g = slice(k0 // GROUP, k1 // GROUP)
        w -= zeros[:, g].double().repeat_interleave(GROUP, 1)
        w *= steps[:, g].double().repeat_interleave(GROUP, 1)
        total += x[:, k0:k1] @ w.T
    if bias is not None:
        total += bias.double()
    if gated:
        half = total.shape[1] // 2
        total = total[:, :half] * torch.sigmoid(total[:, :half]) * total[:, half:]
    return total


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemv":
        return _exact_product(s["X"], s["codes"], s["steps"], s["zeros"], s["bias"], case["gated"])
    if op == "experts":
        edges = s["offsets"].tolist()
        parts = [_exact_product(s["X"][a:b], s["codes"][e], s["steps"][e], s["zeros"][e], None, case["gated"])
                 for e, (a, b) in enumerate(zip(edges, edges[1:]))]
        return torch.cat(parts)
    T, k, E, K = case["T"], case["k"], case["E"], case["K"]
    ids = s["ids"].tolist()
    by_expert = [[] for _ in range(E)]
    for t, picks in enumerate(ids):
        for j, e in enumerate(picks):
            if 0 <= e < E:
                by_expert[e].append((t, j))
    slots = [slot for one in by_expert for slot in one]
    token = torch.tensor([t for t, _ in slots], dtype=torch.long, device="cuda")
    pick = torch.tensor([j for _, j in slots], dtype=torch.long, device="cuda")
    expert = s["ids"].long()[token, pick]
    R = len(slots)
    if op == "dispatch":
        Xs = torch.zeros(T * k, K, dtype=torch.float64, device="cuda")
        Xs[:R] = s["X"].double()[token]
        if s["scales"] is not None:
            Xs[:R] /= s["scales"].double()[expert]
        return {"offsets": None, "order": None, "pos": None, "Xs": Xs}
    weight = s["weights"].double()[token, pick]
    rows = s["Ys"][:R].double()
    if op == "combine":
        Y = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        return Y.index_add_(0, token, rows * weight[:, None])
    dY = s["dY"].double()[token]
    dYs = torch.zeros(T * k, K, dtype=torch.float64, device="cuda")
    dYs[:R] = dY * weight[:, None]
    dweights = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    dweights[token, pick] = (dY * rows).sum(1)
    dxs = s["dXs"][:R].double()
    if s["scales"] is not None:
        dxs /= s["scales"].double()[expert]
    dX = torch.zeros(T, K, dtype=torch.float64, device="cuda").index_add_(0, token, dxs)
    return {"dYs": dYs, "dweights": dweights, "dX": dX}
