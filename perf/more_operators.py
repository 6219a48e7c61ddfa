"""Measured cases of the 8-bit floating-point linear and the mixture of experts built on it: activations quantised to e4m3 with
a scale for each 128 elements, alone or behind the gated product; the product with weights that have a scale for each
128 x 128 block; the router's selection; the products grouped by expert; the weighted sum of the experts' rows.

`run` computes an operator in its plain form (elementary torch operations in fp32) or, where `own` is set, by the calls a
user makes of the library.  Both take the same state: the tensors that a model has in hand."""
import torch

own = False

DEV = "cuda"
BLOCK = 128   # elements of a row, and of a weight's column too, that share a scale
TOP = 448.0   # the largest e4m3 value
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token's hidden state before a projection: the smallest call of a decode step
        {"name": "quant decode 1x4096", "op": "quant", "M": 1, "K": 4096, "gate": ""},
        # the gated product of a long prefill's MLP
        {"name": "quant gated prefill 8192x12288", "op": "quant", "M": 8192, "K": 12288, "gate": "silu"},
        # gate and up packed, eight drafted tokens: a weight stream
        {"name": "linear verify 8x4096x24576", "op": "linear", "M": 8, "K": 4096, "N": 24576},
        # ragged everything, too small to fill the GPU
        {"name": "linear ragged 37x5136x1000", "op": "linear", "M": 37, "K": 5136, "N": 1000},
        # a prefill's up projection: tensor cores
        {"name": "linear prefill 2048x4096x12288", "op": "linear", "M": 2048, "K": 4096, "N": 12288},
        # the router of a verify pass: a launch's latency
        {"name": "route verify 5x64", "op": "route", "M": 5, "E": 64, "k": 6, "score": "softmax", "renorm": True, "half": False, "pad": 0},
        # the router of a long prefill, bf16 logits as a linear gives them
        {"name": "route prefill 8192x128", "op": "route", "M": 8192, "E": 128, "k": 8, "score": "softmax", "renorm": True, "half": True,
         "pad": 0},
        # experts' gate and up projections for eight tokens: about half of the experts' weights are streamed, a row or two each
        {"name": "grouped decode 8x4 of 64", "op": "grouped", "M": 8, "E": 64, "k": 4, "K": 4096, "N": 2816, "gather": True, "pad": 0},
        # experts' down projections of a verify pass over many sequences, sorted rows, a width of eleven blocks
        {"name": "grouped verify 185x8 of 48", "op": "grouped", "M": 185, "E": 48, "k": 8, "K": 1408, "N": 2048, "gather": False, "pad": 0},
        # a prefill through unevenly loaded experts, rows fetched in the experts' order
        {"name": "grouped prefill 4096x4 of 32", "op": "grouped", "M": 4096, "E": 32, "k": 4, "K": 2048, "N": 2560, "gather": True, "pad": 0},
        # the sum of two experts' rows for three tokens, odd width
        {"name": "combine verify 3x2x1001", "op": "combine", "M": 3, "k": 2, "N": 1001, "base": True},
        # the sum of eight experts' rows for a prefill
        {"name": "combine prefill 4096x8x4096", "op": "combine", "M": 4096, "k": 8, "N": 4096, "base": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "route", "grouped", "grouped", "combine"])
    if op == "quant":
        K = 16 * _log(rng, 4, 768)
        return {"op": op, "M": _log(rng, 1, 8192), "K": K, "gate": rng.choice(["", "relu", "silu"])}
    if op == "linear":
        K, N = 16 * _log(rng, 8, 768), _log(rng, 16, 24576)
        return {"op": op, "M": _log(rng, 1, max(1, min(2048, 2048 * 12288 * 4096 // (K * N)))), "K": K, "N": N}
    if op == "route":
        E = _log(rng, 4, 256)
        M = _log(rng, 1, 8192)
        return {"op": op, "M": M, "E": E, "k": rng.randrange(1, min(8, E) + 1), "score": rng.choice(["softmax", "sigmoid"]),
                "renorm": rng.random() < 0.6, "half": rng.random() < 0.5, "pad": rng.choice([0, 0, M // 3])}
    if op == "grouped":
        E = _log(rng, 2, 64)
        k = rng.randrange(1, min(8, E) + 1)
        K, N = 16 * _log(rng, 8, 256), _log(rng, 64, 4096)
        M = _log(rng, 1, max(1, min(4096, 4096 * 4 * 2048 * 2560 // (k * K * N))))
        return {"op": op, "M": M, "E": E, "k": k, "K": K, "N": N, "gather": rng.random() < 0.5, "pad": rng.choice([0, 0, M // 3])}
    N = _log(rng, 64, 8192)
    k = rng.randrange(1, 9)
    return {"op": op, "M": _log(rng, 1, max(1, min(8192, 4096 * 8 * 4096 // (k * N)))), "k": k, "N": N, "base": rng.random() < 0.5}


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    c = case
    if c["op"] == "quant":
        n = c["M"] * c["K"]
        return {"bytes": n * (5 if c["gate"] else 3) + 4 * c["M"] * _blocks(c["K"]), "flops": n * (12 if c["gate"] else 4)}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K + N * K + 2 * M * N + 4 * _blocks(K) * (M + _blocks(N)), "flops": 2 * M * N * K}
    if c["op"] == "route":
        slots = c["M"] * c["k"]
        return {"bytes": c["M"] * c["E"] * (2 if c["half"] else 4) + 16 * slots + 4 * c["E"], "flops": 4 * c["M"] * c["E"]}
    if c["op"] == "grouped":
        rows, N, K = (c["M"] - c["pad"]) * c["k"], c["N"], c["K"]
        seen = min(c["E"], rows)                           # experts whose weights are read, at most
        a = (c["M"] - c["pad"]) if c["gather"] else rows
        return {"bytes": a * K + seen * N * K + 2 * rows * N + 4 * _blocks(K) * (a + seen * _blocks(N)), "flops": 2 * rows * N * K}
    n = c["M"] * c["N"]
    return {"bytes": 2 * n * (c["k"] + 1 + c["base"]) + 8 * c["M"] * c["k"], "flops": 2 * n * (c["k"] + c["base"])}


# ------------------------------------------------------------------------------------------------ the format

def _pad(x, rows):
    """x with its last dimension, and the one before where `rows` is set, filled up with zeros to whole blocks."""
    n, k = x.shape[-2:]
    out = x.new_zeros(x.shape[:-2] + (_blocks(n) * BLOCK if rows else n, _blocks(k) * BLOCK))
    out[..., :n, :k] = x
    return out


def _scale(amax):
    s = amax / torch.full((), TOP, device=DEV)
    return torch.where(s == 0, 1.0, s)


def _quantised(x):
    """fp32 [M, K] -> (codes [M, K] e4m3, scales [M, blocks of 128])."""
    b = _pad(x, False).unflatten(-1, (-1, BLOCK))
    s = _scale(b.abs().amax(-1))
    code = (b / s[..., None]).clamp(-TOP, TOP).flatten(-2)[..., :x.shape[-1]]
    return code.to(F8), s


def _quantised_weight(w):
    """fp32 [N, K] -> (codes [N, K] e4m3, scales [blocks of N, blocks of K])."""
    n, k = w.shape
    b = _pad(w, True).unflatten(-1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))    # block, row, block, column
    s = _scale(b.abs().amax((1, 3)))
    code = (b / s[:, None, :, None]).clamp(-TOP, TOP).flatten(2, 3).flatten(0, 1)[:n, :k]
    return code.to(F8).contiguous(), s


def _values(q, s):
    """Codes [..., K] and scales [..., blocks] as the fp32 values they stand for."""
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _weight_values(q, s):
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]].repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :]


# ------------------------------------------------------------------------------------------------ inputs

def _selected(x, k):
    """The k largest logits of each row, the lowest id first among equals; -1 where no logit is above -inf."""
    top, at = torch.sort(x, dim=1, descending=True, stable=True)
    top, at = top[:, :k], at[:, :k]
    return torch.where(top > float("-inf"), at, -1), top


def _sorted_rows(ids, E):
    """Rows in their experts' order: offsets [E + 1], the row of each slot [M, k] (-1: none), the token of each row."""
    M, k = ids.shape
    flat = torch.where(ids < 0, E, ids).flatten()
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), counts[:E].cumsum(0)))
    order = torch.argsort(flat, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(M * k, device=DEV)
    src = torch.where(torch.arange(M * k, device=DEV) < offsets[E], order // k, -1)
    pos = torch.where(flat < E, row, -1).view(M, k)
    return offsets.to(torch.int32), src.to(torch.int32), pos.to(torch.int32)


def _logits(c, normal):
    """Router logits: some experts are liked more than others; padding tokens allow none."""
    x = normal(c["M"], c["E"]) + 0.7 * normal(c["E"])
    if c["pad"]:
        x[c["M"] - c["pad"]:] = float("-inf")
    return x


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def hidden(m, k):
        return normal(m, k) * torch.exp(0.7 * normal(k))  # some channels are larger than others

    if c["op"] == "quant":
        M, K = c["M"], c["K"]
        x = hidden(M, 2 * K if c["gate"] else K).bfloat16()
        return {"case": c, "x": x, "q": torch.empty((M, K), dtype=F8, device=DEV), "s_a": torch.empty((M, _blocks(K)), device=DEV)}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        q, s_a = _quantised(hidden(M, K))
        w, s_w = _quantised_weight(normal(N, K) * K ** -0.5)
        return {"case": c, "q": q, "s_a": s_a, "w": w, "s_w": s_w, "y": torch.empty((M, N), dtype=torch.bfloat16, device=DEV)}
    if c["op"] == "route":
        M, E, k = c["M"], c["E"], c["k"]
        x = _logits(c, normal)

        def ints(*shape):
            return torch.empty(shape, dtype=torch.int32, device=DEV)

        return {"case": c, "logits": x.bfloat16() if c["half"] else x, "ids": ints(M, k), "weights": torch.empty((M, k), device=DEV),
                "offsets": ints(E + 1), "src": ints(M * k), "pos": ints(M, k)}
    if c["op"] == "grouped":
        M, E, k, K, N = c["M"], c["E"], c["k"], c["K"], c["N"]
        offsets, src, _ = _sorted_rows(_selected(_logits(c, normal), k)[0], E)
        q, s_a = _quantised(hidden(M if c["gather"] else M * k, K))
        w, s_w = torch.empty((E, N, K), dtype=F8, device=DEV), torch.empty((E, _blocks(N), _blocks(K)), device=DEV)
        for e in range(E):
            w[e], s_w[e] = _quantised_weight(normal(N, K) * K ** -0.5)
        n = (offsets[1:] - offsets[:-1])
        busy = torch.nonzero(n)[:, 0]
        return {"case": c, "q": q, "s_a": s_a, "src": src if c["gather"] else None, "offsets": offsets, "w": w, "s_w": s_w,
                "busy": busy, "most": int(n.max()), "y": torch.zeros((M * k, N), dtype=torch.bfloat16, device=DEV)}
    M, k, N = c["M"], c["k"], c["N"]
    pos = torch.randperm(M * k, generator=g, device=DEV).view(M, k).to(torch.int32)
    pos[torch.rand((M, k), generator=g, device=DEV) < 0.02] = -1          # slots that no expert took
    return {"case": c, "rows": normal(M * k, N).bfloat16(), "pos": pos, "weights": torch.rand((M, k), generator=g, device=DEV),
            "base": normal(M, N).bfloat16() if c["base"] else None, "y": torch.empty((M, N), dtype=torch.bfloat16, device=DEV)}


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _gated(x, gate):
    """bf16 gate|up [M, 2K] -> fp32 products [M, K]."""
    g, u = x.float().chunk(2, -1)
    g = torch.where(g > 0, g, 0.0) if gate == "relu" else g / (1.0 + torch.exp(-g))
    return g * u


def _plain_quant(s):
    gate = s["case"]["gate"]
    q, scale = _quantised(_gated(s["x"], gate) if gate else s["x"].float())
    return {"q": q, "s_a": scale}


def _plain_linear(s):
    return torch.matmul(_values(s["q"], s["s_a"]), _weight_values(s["w"], s["s_w"]).t()).bfloat16()


def _plain_route(s):
    c = s["case"]
    x = s["logits"].float()
    ids, top = _selected(x, c["k"])
    taken = ids >= 0
    if c["score"] == "softmax":
        high = x.amax(1, keepdim=True)
        high = torch.where(high > float("-inf"), high, 0.0)
        w = torch.exp(top - high)
        whole = torch.exp(x - high).sum(1, keepdim=True)
    else:
        w, whole = 1.0 / (1.0 + torch.exp(-top)), torch.ones((), device=DEV)
    if c["renorm"]:
        whole = w.sum(1, keepdim=True)
    offsets, src, pos = _sorted_rows(ids, c["E"])
    return {"ids": ids.to(torch.int32), "weights": torch.where(taken, w / torch.where(whole > 0, whole, 1.0), 0.0), "offsets": offsets,
            "src": src, "pos": pos}


def _plain_grouped(s):
    busy, first = s["busy"], s["offsets"][:-1].long()[s["busy"]]
    n = s["offsets"][1:].long()[busy] - first
    i = torch.arange(s["most"], device=DEV)
    there = i < n[:, None]                                            # [experts, rows of the busiest]
    row = torch.where(there, first[:, None] + i, 0)
    token = row if s["src"] is None else s["src"].long()[row]
    x = _values(s["q"], s["s_a"])[token]
    y = torch.matmul(x, _weight_values(s["w"][busy], s["s_w"][busy]).transpose(1, 2)).bfloat16()
    out = torch.zeros_like(s["y"])
    out[row[there]] = y[there]
    return out


def _plain_combine(s):
    pos, w = s["pos"].long(), s["weights"]
    rows = s["rows"][pos.clamp(min=0)].float()                        # [M, k, N]
    y = (rows * torch.where(pos < 0, 0.0, w)[..., None]).sum(1)
    return (y if s["base"] is None else s["base"].float() + y).bfloat16()


_plain = {"quant": _plain_quant, "linear": _plain_linear, "route": _plain_route, "grouped": _plain_grouped, "combine": _plain_combine}


def _library(s):
    """The library and the workspace that a program makes once."""
    if "bi" not in s:
        import invariant_quantized_linear_gb300 as bi
        s["bi"] = bi
        op = s["case"]["op"]
        if op == "route":
            s["ws"] = bi.new_moe_route_workspace(s["case"]["M"], s["case"]["E"])
        elif op in ("linear", "grouped"):
            s["ws"] = bi.new_f8_workspace()
    return s["bi"]


def _own_quant(s):
    bi, c = _library(s), s["case"]
    if c["gate"]:
        bi.bi_gated_quantize_f8(s["x"], bi.BI_GATE_SILU if c["gate"] == "silu" else bi.BI_GATE_RELU, s["q"], s["s_a"])
    else:
        bi.bi_quantize_act_f8(s["x"], s["q"], s["s_a"])
    return {"q": s["q"], "s_a": s["s_a"]}


def _own_linear(s):
    _library(s).bi_linear_f8(s["q"], s["s_a"], s["w"], s["s_w"], s["y"], s["ws"])
    return s["y"]


def _own_route(s):
    bi, c = _library(s), s["case"]
    bi.bi_moe_route(s["logits"], bi.BI_ROUTE_SOFTMAX if c["score"] == "softmax" else bi.BI_ROUTE_SIGMOID, c["renorm"], 1.0, s["ids"],
                    s["weights"], s["offsets"], s["src"], s["pos"], s["ws"])
    return {k: s[k] for k in ("ids", "weights", "offsets", "src", "pos")}


def _own_grouped(s):
    _library(s).bi_linear_f8_grouped(s["q"], s["s_a"], s["src"], s["offsets"], s["w"], s["s_w"], s["y"], s["ws"])
    return s["y"]


def _own_combine(s):
    _library(s).bi_moe_combine(s["rows"], s["pos"], s["weights"], s["base"], s["y"])
    return s["y"]


_own = {"quant": _own_quant, "linear": _own_linear, "route": _own_route, "grouped": _own_grouped, "combine": _own_combine}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    return {"quant": _exact_quant, "linear": _exact_linear, "route": _exact_route, "grouped": _exact_grouped,
            "combine": _exact_combine}[case["op"]](prepare(case, seed))


def _exact_quant(s):
    c, x = s["case"], s["x"]
    K = c["K"]
    q = torch.empty((c["M"], K), dtype=torch.float64, device=DEV)         # the quotients before they are rounded to e4m3
    scale = torch.empty(s["s_a"].shape, dtype=torch.float64, device=DEV)
    for b in range(_blocks(K)):
        cols = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        v = x[:, cols].double()
        if c["gate"]:
            up = x[:, K + cols.start:K + cols.stop].double()
            v = (v.clamp(min=0) if c["gate"] == "relu" else v * torch.sigmoid(v)) * up
        top = v.abs().max(1).values
        step = torch.where(top > 0, top / TOP, torch.ones_like(top))
        scale[:, b] = step
        q[:, cols] = torch.clamp(v / step.float().double()[:, None], -TOP, TOP)
    return {"q": q, "s_a": scale}


def _exact_product(q, s_a, w, s_w):
    """Row by column sums of code products, each block of 128 with its two scales, in fp64."""
    y = torch.zeros((q.shape[0], w.shape[0]), dtype=torch.float64, device=DEV)
    n = torch.arange(w.shape[0], device=DEV) // BLOCK
    for b in range(s_a.shape[1]):
        cols = slice(b * BLOCK, (b + 1) * BLOCK)
        y += (q[:, cols].double() @ w[:, cols].double().t()) * s_a[:, b].double()[:, None] * s_w[n, b].double()
    return y


def _exact_linear(s):
    return _exact_product(s["q"], s["s_a"], s["w"], s["s_w"])


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double()
    w = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    w = torch.where(x > float("-inf"), w, torch.zeros_like(w))
    w = w.gather(1, torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["k"]])
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    return {"ids": None, "weights": w, "offsets": None, "src": None, "pos": None}


def _exact_grouped(s):
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    at = s["offsets"].tolist()
    for e, (a, z) in enumerate(zip(at, at[1:])):
        if z > a:
            rows = torch.arange(a, z, device=DEV) if s["src"] is None else s["src"][a:z].long()
            y[a:z] = _exact_product(s["q"][rows], s["s_a"][rows], s["w"][e], s["s_w"][e])
    return y


def _exact_combine(s):
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV) if s["base"] is None else s["base"].double()
    for j in range(s["case"]["k"]):
        p = s["pos"][:, j].long()
        m = torch.nonzero(p >= 0)[:, 0]
        y[m] += s["weights"][m, j].double()[:, None] * s["rows"][p[m]].double()
    return y
