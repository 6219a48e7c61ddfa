"""Measured cases of the decoder-step operators around the W8A8 linears: RMS norm with int8 output, rotary positions with
the append to a 4-bit paged cache, attention over that cache, and the rules applied to logits before the argmax.

`run` computes an operator in its plain form (elementary torch operations in fp32) or, where `own` is set, by the calls a
user makes of the library.  Both take the same state: the tensors that a decode loop has in hand."""
import torch

own = False

DEV = "cuda"
BLOCK = 64  # cache elements that share a scale and a minimum


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a 4096-wide decoder layer: the smallest call between two linears
        {"name": "norm decode 1x4096", "op": "norm", "M": 1, "K": 4096, "add": True},
        # a verify pass of five tokens for 37 sequences over an MLP width that no power of two divides evenly
        {"name": "norm verify 185x5136", "op": "norm", "M": 185, "K": 5136, "add": True},
        # a long prefill's rows
        {"name": "norm prefill 8192x4096", "op": "norm", "M": 8192, "K": 4096, "add": True},
        # one new token of one sequence, heads normed before the rotation, split-half layout
        {"name": "append decode b1", "op": "append", "B": 1, "q": 1, "ctx": 1000, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "interleaved": False, "norm": True, "page": 16},
        # prefill of three ragged prompts
        {"name": "append prefill b3", "op": "append", "B": 3, "q": 2731, "ctx": 0, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "interleaved": False, "norm": True, "page": 64},
        # small heads, a quarter of each rotated, interleaved pairs, ragged verify of up to 7 tokens for 40 sequences
        {"name": "append verify b40 d64", "op": "append", "B": 40, "q": 7, "ctx": 5000, "Hq": 15, "Hkv": 5, "D": 64, "rot": 16,
         "interleaved": True, "norm": False, "page": 32},
        # one token over a short cache: latency
        {"name": "attn decode b1 s517", "op": "attn", "B": 1, "q": 1, "ctx": 517, "Hq": 32, "Hkv": 8, "D": 128, "page": 16},
        # the verify pass of 8 drafted tokens after 4096 positions
        {"name": "attn verify b1 q8 s4104", "op": "attn", "B": 1, "q": 8, "ctx": 4104, "Hq": 32, "Hkv": 8, "D": 128, "page": 64},
        # batched decode of ragged sequences, the serving case
        {"name": "attn decode b96 s8191", "op": "attn", "B": 96, "q": 1, "ctx": 8191, "Hq": 32, "Hkv": 8, "D": 128, "page": 64},
        # ragged verify over long contexts, groups of 7 heads of 64
        {"name": "attn verify b6 q5 s40000", "op": "attn", "B": 6, "q": 5, "ctx": 40000, "Hq": 28, "Hkv": 4, "D": 64, "page": 128},
        # penalties, biases and a grammar mask on the five rows of one verify pass
        {"name": "logits verify 5x151936", "op": "logits", "B": 1, "q": 5, "V": 151936, "hist": 1500, "bias": 50, "mask": True,
         "out": True},
        # the same rules over a batch of 400 rows, odd vocabulary
        {"name": "logits batch 400x128259", "op": "logits", "B": 100, "q": 4, "V": 128259, "hist": 3000, "bias": 10, "mask": True,
         "out": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "append", "attn", "logits", "attn"])
    if op == "norm":
        K = 16 * _log(rng, 4, 800)
        return {"op": op, "M": _log(rng, 1, max(1, min(8192, 8192 * 4096 // K))), "K": K, "add": rng.random() < 0.8}
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _log(rng, 1, 64)
        q = _log(rng, 1, max(1, 8192 // B))
        return {"op": op, "B": B, "q": q, "ctx": rng.randrange(0, 9000), "Hq": min(32, Hkv * G) // Hkv * Hkv, "Hkv": Hkv, "D": D,
                "rot": rng.choice([D // 4, D // 2, D]), "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.5, "page": page}
    if op == "attn":
        B = _log(rng, 1, 96)
        q = _log(rng, 1, 16)
        ctx = q + _log(rng, 1, max(2, 700000 // B // 2))
        ctx = max(q, min(ctx, 131072, 15000000 // (B * q * Hkv * G)))
        return {"op": op, "B": B, "q": q, "ctx": ctx, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page}
    B = _log(rng, 1, 100)
    return {"op": op, "B": B, "q": rng.randrange(1, 5), "V": _log(rng, 1000, 128000), "hist": _log(rng, 1, 3000),
            "bias": rng.randrange(0, 64), "mask": rng.random() < 0.7, "out": rng.random() < 0.7}


def _q_lens(c):
    """New tokens of each sequence: the most for the first, fewer for the others of a ragged batch."""
    return [max(1, c["q"] - (b * 5) % max(1, (c["q"] + 1) // 2)) for b in range(c["B"])]


def _kv_lens(c):
    """Positions of each sequence, its new tokens included, between a quarter of the longest and all of it."""
    if c["op"] == "append":
        return [n + (c["ctx"] * (4 - b % 4)) // 4 for b, n in enumerate(_q_lens(c))]
    return [max(n, c["ctx"] - int(0.75 * c["ctx"] * ((b * 0.6180339887) % 1.0))) for b, n in enumerate(_q_lens(c))]


def _hists(c):
    """History of each sequence before the rows of this pass."""
    return [max(1, c["hist"] - (b * 37) % max(1, c["hist"] // 2)) for b in range(c["B"])]


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["M"] * c["K"]
        return {"bytes": n * (7 if c["add"] else 3) + 2 * c["K"] + 4 * c["M"], "flops": 8 * n}
    if c["op"] == "logits":
        rows = c["B"] * c["q"]
        ids = sum(_hists(c)) + c["B"] * c["q"] + 2 * c["bias"] * rows
        return {"bytes": rows * c["V"] * (2 + (4 if c["out"] else 0) + (0.125 if c["mask"] else 0)) + 4 * ids + 4 * rows,
                "flops": 6 * rows * c["V"]}
    T, D = sum(_q_lens(c)), c["D"]
    per = D / 2 + 4 * (D // BLOCK)  # bytes of one head's k (or v) at one position
    if c["op"] == "append":
        kv = 2 * T * c["Hkv"]
        return {"bytes": 4 * T * c["Hq"] * D + kv * (2 * D + per) + 4 * c["rot"] * T + 2 * kv * D,
                "flops": T * (c["Hq"] + 2 * c["Hkv"]) * D * 8}
    lens = _kv_lens(c)
    seen = sum(n * s - n * (n - 1) // 2 for n, s in zip(_q_lens(c), lens))
    return {"bytes": sum(lens) * c["Hkv"] * 2 * per + 4 * T * c["Hq"] * D, "flops": 4 * seen * c["Hq"] * D}


# ------------------------------------------------------------------------------------------------ the cache's layout
#
# A page holds `page` positions; a block is one kv head of one page: k codes, v codes, then 32-bit words (scale, minimum)
# in bf16 for k and v of every 64 elements.  Element d of k: segment (d % 64) / 16 of four, block d / 64 within it, word
# (d % 16) / 8, nibble (d % 8) / 2 + 4 (d % 2).  Element d of v at position p: pair p / 2, segment (d % 64) / 8 of eight, block d / 64,
# word (d % 8) / 4, half p % 2, nibble d % 4.

def _block_bytes(page, D):
    return page * (D + 8 * (D // BLOCK))


def _regions(pool, page, D):
    """Views of a pool [pages, Hkv, block bytes]: k codes, v codes (position pairs), parameters (bf16)."""
    n, h = pool.shape[:2]
    g, half = D // BLOCK, page * D // 2
    k = pool[:, :, :half].view(n, h, page, 4, g, 2, 4)
    v = pool[:, :, half:2 * half].view(n, h, page // 2, 8, g, 2, 2, 2)
    m = pool[:, :, 2 * half:].view(torch.bfloat16).view(n, h, page, 2, g, 2)
    return k, v, m


def _pack_k(code):
    """uint8 codes [..., D] -> bytes [..., 4, D / 64, 2, 4]."""
    x = code.unflatten(-1, (-1, 4, 2, 2, 2, 2))  # block, segment, word, byte of the half, nibble of the byte, half
    x = x[..., 0, :] | (x[..., 1, :] << 4)       # block, segment, word, byte of the half, half
    return x.swapaxes(-1, -2).flatten(-2).swapaxes(-4, -3)


def _pack_v(code):
    """uint8 codes [..., D] of one position -> bytes [..., 8, D / 64, 2, 2]."""
    x = code.unflatten(-1, (-1, 8, 2, 2, 2))  # block, segment, word, byte, nibble
    return (x[..., 0] | (x[..., 1] << 4)).swapaxes(-4, -3)


def _unpack_k(b):
    """bytes [..., 4, D / 64, 2, 4] -> codes [..., D]."""
    x = torch.stack((b & 15, b >> 4), -1).unflatten(-2, (2, 2))  # segment, block, word, half, byte, nibble
    return x.swapaxes(-6, -5).movedim(-3, -1).flatten(-6)


def _unpack_v(b):
    """bytes [..., pairs, 8, D / 64, 2, 2, 2] -> codes [..., 2 pairs, D]."""
    x = torch.stack((b & 15, b >> 4), -1)              # pair, segment, block, word, position, byte, nibble
    x = x.movedim(-3, -6).swapaxes(-5, -4)             # pair, position, block, segment, word, byte, nibble
    return x.flatten(-5).flatten(-3, -2)


def _quantise(x):
    """fp32 holding bf16 values [..., D] -> (uint8 codes, scales, minima [..., D / 64], both bf16)."""
    g = x.unflatten(-1, (-1, BLOCK))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi - lo) / torch.full((), 15.0, device=x.device)).bfloat16()
    f = s.float()
    ok = (f > 0)[..., None]
    code = torch.where(ok, ((g - lo[..., None]) / torch.where(ok, f[..., None], 1.0)).round().clamp(0, 15), 0.0)
    return code.to(torch.uint8).flatten(-2), s, lo.bfloat16()


def _values(code, s, z):
    return (z.float()[..., None] + s.float()[..., None] * code.unflatten(-1, (-1, BLOCK)).float()).flatten(-2)


# ------------------------------------------------------------------------------------------------ inputs

def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _batch(c, g, spare=3):
    """cu_q, kv_len and a shuffled page table; entries past a sequence's pages hold -1."""
    ql, kl, page = _q_lens(c), _kv_lens(c), c["page"]
    need = [-(-n // page) for n in kl]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    at, width = torch.tensor([0] + need).cumsum(0), max(need)
    col = torch.arange(width, device=DEV)[None]
    start, count = at[:-1].to(DEV)[:, None], torch.tensor(need, device=DEV)[:, None]
    table = torch.where(col < count, order[(start + col).clamp(max=total - 1)], -1).to(torch.int32)
    cu = [0]
    for n in ql:
        cu.append(cu[-1] + n)
    return {"cu_q": _ints(cu), "kv_len": _ints(kl), "table": table.contiguous(), "pages": total, "T": cu[-1], "max_q": max(ql),
            "max_kv": max(kl)}


def _fill(pool, page, D, g):
    """Codes and parameters of normally distributed keys and values."""
    k, v, m = _regions(pool, page, D)
    half = page * D // 2
    step = max(1, (1 << 26) // (pool.shape[1] * 2 * half))
    for a in range(0, pool.shape[0], step):
        part = pool[a:a + step, :, :2 * half]
        x = torch.randn((2,) + tuple(part.shape), generator=g, device=DEV).mul_(2.9).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        part.copy_(x[0] | (x[1] << 4))
    s = torch.exp(0.3 * torch.randn(m.shape[:-1], generator=g, device=DEV)) * torch.tensor([0.3, 0.2], device=DEV)[:, None]
    m[..., 0] = s.bfloat16()
    m[..., 1] = (-7.5 * s + 0.4 * s * torch.randn(s.shape, generator=g, device=DEV)).bfloat16()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        channel = torch.exp(0.7 * normal(K))
        return {"case": c, "h": (normal(M, K) * channel * 3).bfloat16(), "y": (normal(M, K) * channel).bfloat16() if c["add"] else None,
                "w": (1 + 0.3 * normal(K)).bfloat16(), "h_out": torch.empty((M, K), dtype=torch.bfloat16, device=DEV),
                "q": torch.empty((M, K), dtype=torch.int8, device=DEV), "s_a": torch.empty(M, device=DEV),
                "value": torch.empty((M, K), dtype=torch.bfloat16, device=DEV)}
    if c["op"] == "logits":
        B, q, V, hist = c["B"], c["q"], c["V"], _hists(c)
        rows = B * q
        begin, at = [], 0
        for n in hist:  # a sequence's ids, the tokens drafted in this pass behind them
            begin.append(at)
            at += n + q
        # few distinct tokens make up most of a text
        ids = (V * torch.rand(at, generator=g, device=DEV) ** 6).long().clamp(max=V - 1).to(torch.int32)
        s = {"case": c, "logits": (3 * normal(rows, V)).bfloat16(), "ids": ids,
             "begin": _ints([begin[b] for b in range(B) for _ in range(q)]),
             "mid": _ints([begin[b] + hist[b] // 3 for b in range(B) for _ in range(q)]),
             "end": _ints([begin[b] + hist[b] + i for b in range(B) for i in range(q)]),
             "repetition": 1 + 0.5 * torch.rand(rows, generator=g, device=DEV), "presence": torch.rand(rows, generator=g, device=DEV),
             "frequency": 0.3 * torch.rand(rows, generator=g, device=DEV),
             "bias_ids": ((torch.randint(0, V, (rows, 1), generator=g, device=DEV) + 7 * torch.arange(c["bias"], device=DEV)) % V).to(torch.int32),
             "bias": 4 * normal(rows, c["bias"]),
             "mask": None, "out": torch.empty((rows, V), device=DEV) if c["out"] else None,
             "argmax": torch.empty(rows, dtype=torch.int32, device=DEV)}
        if c["mask"]:
            words = torch.randint(-2 ** 31, 2 ** 31, (rows, -(-V // 32)), generator=g, device=DEV)
            words[torch.rand(words.shape, generator=g, device=DEV) < 0.5] = 0  # a grammar forbids whole stretches
            words[96::97] = 0                                      # and, in a dead end, everything
            s["mask"] = words.to(torch.int32)
        return s
    D, Hq, Hkv, page = c["D"], c["Hq"], c["Hkv"], c["page"]
    s = {"case": c, **_batch(c, g)}
    s["pool"] = torch.zeros((s["pages"], Hkv, _block_bytes(page, D)), dtype=torch.uint8, device=DEV)
    if c["op"] == "append":
        rows = normal(s["T"], Hq + 2 * Hkv, D) * torch.exp(0.5 * normal(Hq + 2 * Hkv, D))
        s["qkv"] = rows.bfloat16().flatten(1)  # a packed projection's output
        rot = c["rot"]
        inv = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        angle = torch.arange(s["max_kv"], dtype=torch.float64, device=DEV)[:, None] * inv
        s["rope"] = torch.stack((angle.cos(), angle.sin()), -1).float()  # [positions, rot / 2, 2]
        s["q_norm"] = (1 + 0.2 * normal(D)).bfloat16() if c["norm"] else None
        s["k_norm"] = (1 + 0.2 * normal(D)).bfloat16() if c["norm"] else None
        s["q_out"] = torch.empty((s["T"], Hq, D), dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty((s["T"], Hkv, D), dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty((s["T"], Hkv, D), dtype=torch.bfloat16, device=DEV)
        return s
    _fill(s["pool"], page, D, g)
    s["q"] = normal(s["T"], Hq, D).bfloat16()
    s["o"] = torch.empty_like(s["q"])
    s["scale"] = D ** -0.5
    return s


# ------------------------------------------------------------------------------------------------ one pass

EPS = 1e-6


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _plain_norm(s):
    h = s["h"].float()
    if s["y"] is not None:
        h = (h + s["y"].float()).bfloat16().float()
    t = h * s["w"].float()
    r = 1.0 / torch.sqrt((h * h).mean(-1) + EPS)
    a = t.abs().amax(-1)
    step = torch.where(a > 0, a / torch.full((), 127.0, device=DEV), 1.0)
    code = (t / step[:, None]).round().clamp(-127, 127)
    s_a = torch.where(a > 0, step * r, 1.0)
    return {"h": h.bfloat16(), "value": (code * s_a[:, None]).bfloat16(), "s_a": s_a}


def _head_norm(x, w):
    """RMS norm of each head, its squares added in halves, neighbours and halves again."""
    if w is None:
        return x
    q = x * x
    q = q[..., :q.shape[-1] // 2] + q[..., q.shape[-1] // 2:]
    q = q[..., 0::2] + q[..., 1::2]
    while q.shape[-1] > 1:
        q = q[..., :q.shape[-1] // 2] + q[..., q.shape[-1] // 2:]
    r = 1.0 / torch.sqrt(q / x.shape[-1] + EPS)
    return x * r * w.float()


def _rotate(x, cs, rot, interleaved):
    a, rest = x[..., :rot], x[..., rot:]
    co, si = cs[:, None, :, 0], cs[:, None, :, 1]
    if interleaved:
        p, q = a[..., 0::2], a[..., 1::2]
        a = torch.stack((p * co - q * si, q * co + p * si), -1).flatten(-2)
    else:
        p, q = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat((p * co - q * si, q * co + p * si), -1)
    return torch.cat((a, rest), -1)


def _tokens(s):
    """Sequence and position of every new token."""
    t = torch.arange(s["T"], dtype=torch.int32, device=DEV)
    b = torch.searchsorted(s["cu_q"][1:], t, right=True)
    return b, (s["kv_len"][b] - s["cu_q"][b + 1] + t).long()


def _plain_append(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    x = s["qkv"].view(s["T"], Hq + 2 * Hkv, D).float()
    b, pos = _tokens(s)
    cs = s["rope"][pos]
    q = _rotate(_head_norm(x[:, :Hq], s["q_norm"]), cs, c["rot"], c["interleaved"]).bfloat16()
    k = _rotate(_head_norm(x[:, Hq:Hq + Hkv], s["k_norm"]), cs, c["rot"], c["interleaved"]).bfloat16().float()
    block, slot = s["table"][b, pos // page].long(), pos % page
    pk, pv, pm = _regions(s["pool"], page, D)
    kc, ks, kz = _quantise(k)
    vc, vs, vz = _quantise(x[:, Hq + Hkv:])
    pk[block, :, slot] = _pack_k(kc)
    pv[block, :, slot // 2, :, :, :, slot % 2] = _pack_v(vc)
    pm[block, :, slot] = torch.stack((torch.stack((ks, kz), -1), torch.stack((vs, vz), -1)), 2)
    return {"q": q, "k": _values(kc, ks, kz).bfloat16(), "v": _values(vc, vs, vz).bfloat16()}


def _plain_attn(s):
    c = s["case"]
    Hq, Hkv, D, page, B, mq = c["Hq"], c["Hkv"], c["D"], c["page"], c["B"], s["max_q"]
    G = Hq // Hkv
    blocks = s["table"].clamp(min=0).long()                      # [B, n]
    pk, pv, pm = _regions(s["pool"][blocks.flatten()], page, D)
    S = blocks.shape[1] * page

    def spread(codes, which):                                    # [B n, Hkv, page, D] -> [B, Hkv, S, D]
        x = _values(codes, pm[:, :, :, which, :, 0], pm[:, :, :, which, :, 1])
        return x.view(B, -1, Hkv, page, D).transpose(1, 2).reshape(B, Hkv, S, D)

    at = s["cu_q"][:-1, None] + torch.arange(mq, device=DEV)      # [B, mq]
    n = s["cu_q"][1:] - s["cu_q"][:-1]
    real = torch.arange(mq, device=DEV) < n[:, None]
    q = s["q"][at.clamp(max=s["T"] - 1).long()].float()          # [B, mq, Hq, D]
    q = q.view(B, mq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, mq * G, D)
    score = torch.matmul(q, spread(_unpack_k(pk), 0).transpose(2, 3)) * s["scale"]
    last = s["kv_len"][:, None] - n[:, None] + torch.arange(mq, device=DEV)
    seen = (torch.arange(S, device=DEV) <= last[:, :, None]).repeat_interleave(G, 1)[:, None]
    score = score.masked_fill(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top.isinf(), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, spread(_unpack_v(pv), 1)) / torch.where(total > 0, total, 1.0)
    o = o.view(B, Hkv, mq, G, D).permute(0, 2, 1, 3, 4).reshape(B, mq, Hq, D)
    b, pos = _tokens(s)
    i = torch.arange(s["T"], device=DEV) - s["cu_q"][b]
    return o[b, i].bfloat16()


def _plain_logits(s):
    c = s["case"]
    V, rows = c["V"], c["B"] * c["q"]
    x = s["logits"].float()
    at = s["begin"][:, None] + torch.arange(c["hist"] + c["q"], device=DEV)
    inside = at < s["end"][:, None]
    ids = s["ids"][at.clamp(max=s["ids"].numel() - 1)].long()
    ids = torch.where(inside, ids, V)                            # column V takes what no row holds
    new = inside & (at >= s["mid"][:, None])
    count = torch.zeros((rows, V + 1), dtype=torch.int32, device=DEV).scatter_add_(1, ids, new.to(torch.int32))[:, :V]
    held = torch.zeros((rows, V + 1), dtype=torch.int32, device=DEV).scatter_add_(1, ids, inside.to(torch.int32))[:, :V] > 0
    rep = s["repetition"][:, None]
    x = torch.where(held, torch.where(x > 0, x / rep, x * rep), x)
    x = torch.where(count > 0, x - s["frequency"][:, None] * count.float() - s["presence"][:, None], x)
    if c["bias"]:
        x = x.scatter_add(1, s["bias_ids"].long(), s["bias"])
    if s["mask"] is not None:
        col = torch.arange(V, device=DEV)
        allowed = (s["mask"][:, col // 32] >> (col % 32)) & 1
        x = torch.where(allowed > 0, x, float("-inf"))
    top = x.amax(1, keepdim=True)
    first = torch.where(x == top, torch.arange(V, dtype=torch.int32, device=DEV), V).amin(1)
    first = torch.where(top[:, 0].isinf(), -1, first).to(torch.int32)
    return (x, first) if c["out"] else (first,)


_plain = {"norm": _plain_norm, "append": _plain_append, "attn": _plain_attn, "logits": _plain_logits}


def _handles(s):
    """What a user's program builds once for its cache and batch."""
    if "cache" not in s:
        import invariant_quantized_linear_gb300 as bi
        c = s["case"]
        s["bi"] = bi
        s["cache"] = bi.kv4_cache(s["pool"], c["page"], c["D"])
        s["batch"] = bi.kv4_batch(s["cu_q"], s["kv_len"], s["table"], s["T"], s["max_q"], s["max_kv"])
        if c["op"] == "attn":
            s["ws"] = bi.new_attention_kv4_workspace(c["Hq"], s["cache"], s["batch"])
        else:
            qkv = s["qkv"].view(s["T"], -1, c["D"])
            s["parts"] = qkv[:, :c["Hq"]], qkv[:, c["Hq"]:c["Hq"] + c["Hkv"]], qkv[:, c["Hq"] + c["Hkv"]:]
    return s["bi"]


def _own_norm(s):
    import invariant_quantized_linear_gb300 as bi
    bi.bi_rmsnorm_quantize(s["h"], s["y"], s["w"], EPS, s["h_out"] if s["y"] is not None else None, s["q"], s["s_a"])
    # the codes as the values they stand for
    torch.mul(s["q"], s["s_a"][:, None], out=s["value"])
    return {"h": s["h_out"] if s["y"] is not None else s["h"], "value": s["value"], "s_a": s["s_a"]}


def _own_append(s):
    bi, c = _handles(s), s["case"]
    q, k, v = s["parts"]
    bi.bi_rope_append_kv4(q, k, v, s["rope"], c["rot"], bi.BI_ROPE_INTERLEAVED if c["interleaved"] else bi.BI_ROPE_HALF, s["q_out"],
                          s["cache"], s["batch"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
    # the cache's new positions as the values they stand for
    bi.bi_kv4_gather(s["cache"], s["batch"], s["k_out"], s["v_out"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_attn(s):
    bi = _handles(s)
    bi.bi_attention_kv4(s["q"], s["cache"], s["batch"], s["scale"], s["o"], s["ws"])
    return s["o"]


def _own_logits(s):
    if "rules" not in s:
        import invariant_quantized_linear_gb300 as bi
        s["bi"] = bi
        s["rules"] = bi.logits_rules(ids=s["ids"], begin=s["begin"], mid=s["mid"], end=s["end"], repetition=s["repetition"],
                                     presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"],
                                     mask=s["mask"])
        s["ws"] = bi.new_logits_workspace(s["logits"].shape[0])
    s["bi"].bi_logits_process(s["logits"], s["rules"], s["out"], s["argmax"], s["ws"])
    return (s["out"], s["argmax"]) if s["out"] is not None else (s["argmax"],)


_own = {"norm": _own_norm, "append": _own_append, "attn": _own_attn, "logits": _own_logits}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    return {"norm": _exact_norm, "append": _exact_append, "attn": _exact_attn, "logits": _exact_logits}[case["op"]](prepare(case, seed))


def _exact_norm(s):
    h = s["h"].double() + (s["y"].double() if s["y"] is not None else 0.0)
    h = h.bfloat16().double()  # the sum is held in bf16, and the norm reads what is held
    w = s["w"].double()
    value, scale = torch.empty_like(h), torch.empty(h.shape[0], dtype=torch.float64, device=DEV)
    for a in range(0, h.shape[0], 1024):
        x = h[a:a + 1024]
        n = x / (x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS).sqrt() * w
        top = n.abs().max(1, keepdim=True).values
        step = torch.where(top > 0, top / 127, torch.ones_like(top))
        value[a:a + 1024] = torch.clamp(torch.round(n / step), -127, 127) * step
        scale[a:a + 1024] = step[:, 0]
    return {"h": h, "value": value, "s_a": scale}


def _exact_quantised(x):
    out = torch.empty_like(x)
    for d in range(0, x.shape[-1], BLOCK):
        part = x[..., d:d + BLOCK]
        lo, hi = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
        s = ((hi - lo) / 15).float().bfloat16().double()  # held in bf16
        code = torch.clamp(torch.round((part - lo) / torch.where(s > 0, s, torch.ones_like(s))), 0, 15)
        out[..., d:d + BLOCK] = lo + code * s
    return out


def _exact_append(s):
    c = s["case"]
    Hq, Hkv, D, rot = c["Hq"], c["Hkv"], c["D"], c["rot"]
    x = s["qkv"].double().view(s["T"], Hq + 2 * Hkv, D)
    first = s["cu_q"].tolist()
    at = torch.cat([torch.arange(n - (b - a), n, device=DEV) for a, b, n in zip(first, first[1:], s["kv_len"].tolist())])
    turn = torch.complex(s["rope"][at, :, 0].double(), s["rope"][at, :, 1].double())[:, None]

    def turned(v, w):
        if w is not None:
            v = v / (v.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        v = v.clone()
        one, two = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(v[..., one], v[..., two]) * turn
        v[..., one], v[..., two] = z.real, z.imag
        return v

    k = turned(x[:, Hq:Hq + Hkv], s["k_norm"]).float().bfloat16().double()  # rounded to bf16 before it is quantised
    return {"q": turned(x[:, :Hq], s["q_norm"]), "k": _exact_quantised(k), "v": _exact_quantised(x[:, Hq + Hkv:])}


def _exact_attn(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    G, blocks, half = Hq // Hkv, D // BLOCK, page * D // 2
    d = torch.arange(D, device=DEV)
    nib = d % 8 // 2 + 4 * (d % 2)
    k_byte, k_shift = ((d % 64 // 16) * blocks + d // 64) * 8 + d % 16 // 8 * 4 + nib // 2, 4 * (nib % 2)
    v_byte, v_shift = (((d % 64 // 8) * blocks + d // 64) * 2 + d % 8 // 4) * 4 + d % 4 // 2, 4 * (d % 2)
    first, out = s["cu_q"].tolist(), []
    for b, (a, e, n) in enumerate(zip(first, first[1:], s["kv_len"].tolist())):
        p = torch.arange(n, device=DEV)
        rows = s["table"][b].long()[p // page]
        slot = p % page
        heads = []
        for h in range(Hkv):
            raw = s["pool"][:, h][rows.unique_consecutive()]                       # [pages of the sequence, bytes]
            own_page = p // page
            k = raw[own_page[:, None], slot[:, None] * (D // 2) + k_byte].long() >> k_shift & 15
            v = raw[own_page[:, None], half + slot[:, None] // 2 * D + slot[:, None] % 2 * 2 + v_byte].long() >> v_shift & 15
            par = raw[:, 2 * half:].contiguous().view(torch.bfloat16).double().view(-1, page, 2, blocks, 2)[own_page, slot]
            k = par[:, 0, d // 64, 0] * k + par[:, 0, d // 64, 1]
            v = par[:, 1, d // 64, 0] * v + par[:, 1, d // 64, 1]
            q = s["q"][a:e, h * G:(h + 1) * G].double()
            w = torch.einsum("tgd,nd->tgn", q, k) * s["scale"]
            w[(p[None] > n - (e - a) + torch.arange(e - a, device=DEV)[:, None])[:, None].expand_as(w)] = float("-inf")
            heads.append(torch.einsum("tgn,nd->tgd", torch.softmax(w, -1), v))
        out.append(torch.cat(heads, 1))
    return torch.cat(out)


def _exact_logits(s):
    c = s["case"]
    if not c["out"]:
        return None
    rows, V = s["logits"].shape
    out = torch.empty((rows, V), dtype=torch.float64, device=DEV)
    begin, mid, end = (s[k].tolist() for k in ("begin", "mid", "end"))
    for r in range(rows):
        x = s["logits"][r].double()
        every, new = s["ids"][begin[r]:end[r]].long(), s["ids"][mid[r]:end[r]].long()
        rep = s["repetition"][r].double()
        seen = every.unique()
        x[seen] = torch.where(x[seen] > 0, x[seen] / rep, x[seen] * rep)
        tok, n = new.unique(return_counts=True)
        x[tok] -= s["frequency"][r].double() * n + s["presence"][r].double()
        x[s["bias_ids"][r].long()] += s["bias"][r].double()
        if s["mask"] is not None:
            bits = (s["mask"][r][:, None] >> torch.arange(32, device=DEV) & 1).flatten()[:V]
            x[bits == 0] = float("-inf")
        out[r] = x
    return out, None
