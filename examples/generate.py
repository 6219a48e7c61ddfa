"""Greedy generation from a quantised decoder, one token a step or speculatively.

A decoder with random weights serves a few sequences at once: RMS norm with the
residual update into int8 codes, W8A8 linears, rotation with the append to the
4-bit paged cache, attention over it, the gated MLP, and logits under penalties
and a token mask.  Drafts come from the sequence itself (what followed the last
occurrence of its last two tokens); a verify pass runs them all at once and
keeps the prefix that plain decoding would have chosen.  Every row of every call
has the same bits whatever shares the call, so both ways give the same tokens,
which main() checks.

    python examples/generate.py [--new 64] [--draft 4]
"""
import argparse
import os
import sys
import time
from dataclasses import dataclass

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import invariant_quantized_linear_gb300 as bi  # noqa: E402


@dataclass
class Config:
    layers: int = 4
    hidden: int = 1024
    heads: int = 8
    kv_heads: int = 2
    head_size: int = 128
    inner: int = 2816
    vocab: int = 32003
    page: int = 64
    max_len: int = 1024
    eps: float = 1e-6
    rope_base: float = 10000.0


class Decoder:
    """Random weights and a paged cache for `sequences` sequences."""

    def __init__(self, cfg: Config, sequences: int, seed: int = 0, device="cuda"):
        self.cfg, self.device, self.B = cfg, device, sequences
        gen = torch.Generator(device=device).manual_seed(seed)
        H, D, I = cfg.hidden, cfg.head_size, cfg.inner
        qkv = (cfg.heads + 2 * cfg.kv_heads) * D

        def linear(n, k):
            w = torch.randn((n, k), device=device, generator=gen) * k ** -0.5
            codes, scale = torch.empty((n, k), dtype=torch.int8, device=device), torch.empty(n, device=device)
            bi.bi_quantize_weight(w, codes, scale)
            bi.bi_requant_pow2(codes, scale, codes, scale)
            return codes, scale

        def norm(n):
            return (1 + 0.1 * torch.randn(n, device=device, generator=gen)).bfloat16()

        self.embed = torch.randn((cfg.vocab, H), device=device, generator=gen).bfloat16()
        self.layers = [dict(norm1=norm(H), qkv=linear(qkv, H), q_norm=norm(D), k_norm=norm(D), o=linear(H, cfg.heads * D),
                            norm2=norm(H), gu=linear(2 * I, H), down=linear(H, I)) for _ in range(cfg.layers)]
        self.norm, self.head = norm(H), linear(cfg.vocab, H)
        inv = cfg.rope_base ** (-torch.arange(0, D, 2, dtype=torch.float64, device=device) / D)
        self.rope = torch.empty((cfg.max_len, D // 2, 2), device=device)
        bi.bi_rope_table(inv, self.rope)
        # one pool, [page, layer, ...]: a layer's cache is a view of it; pages are dealt out of order
        n = -(-cfg.max_len // cfg.page)
        block = bi.bi_kv4_block_bytes(cfg.page, D)
        self.pool = torch.zeros((sequences * n, cfg.layers, cfg.kv_heads, block), dtype=torch.uint8, device=device)
        self.caches = [bi.kv4_cache(self.pool[:, i], cfg.page, D) for i in range(cfg.layers)]
        self.pages = torch.randperm(sequences * n, device=device, generator=gen).int().view(sequences, n)
        self.ws, self.tokens = None, 0

    def _room(self, T: int) -> None:
        """Buffers for passes of up to T tokens."""
        if T <= self.tokens:
            return
        c, dev = self.cfg, self.device
        D, QR = c.head_size, c.heads * c.head_size

        def buf(n, dtype=torch.bfloat16):
            return torch.empty((T, n), dtype=dtype, device=dev)
        self.tokens = T
        self.y = dict(qkv=buf(QR + 2 * c.kv_heads * D), o=buf(c.hidden), gu=buf(2 * c.inner), down=buf(c.hidden))
        self.codes = dict(h=buf(c.hidden, torch.int8), o=buf(QR, torch.int8), m=buf(c.inner, torch.int8))
        self.scales = torch.empty(T, device=dev)
        self.q, self.o = (torch.empty((T, c.heads, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
        shapes = [self.layers[0][n][0].shape for n in ("qkv", "o", "gu", "down")] + [self.head[0].shape]
        self.ws = torch.zeros(max(bi.bi_linear_workspace_size(t, *s) for s in shapes for t in (1, T)), dtype=torch.uint8,
                              device=dev)
        bound = bi.kv4_batch(torch.zeros(self.B + 1, dtype=torch.int32), torch.zeros(self.B, dtype=torch.int32), self.pages, T,
                             T, c.max_len)
        self.attn_ws = bi.new_attention_kv4_workspace(c.heads, self.caches[0], bound, dev)
        self.logits_ws = bi.new_logits_workspace(T, dev)

    def forward(self, ids: torch.Tensor, counts: list[int], lengths: list[int], rows: torch.Tensor) -> torch.Tensor:
        """Appends counts[b] new tokens (ids int32 [T], in order) of each sequence, whose length becomes lengths[b], and
        returns the logits, bf16 [len(rows), vocab], of the tokens in `rows`."""
        c, dev, T = self.cfg, self.device, sum(counts)
        D, QR, KV = c.head_size, c.heads * c.head_size, c.kv_heads * c.head_size
        self._room(T)
        cu_q = torch.tensor([0] + counts, device=dev).cumsum(0).int()
        kv_len = torch.tensor(lengths, dtype=torch.int32, device=dev)
        batch = bi.kv4_batch(cu_q, kv_len, self.pages, T, max(counts), max(lengths))
        y = {k: v[:T] for k, v in self.y.items()}
        codes, s = {k: v[:T] for k, v in self.codes.items()}, self.scales[:T]
        q, o = self.q[:T], self.o[:T]
        h, add = self.embed[ids.long()], None
        qkv = y["qkv"]
        q_in, k_in, v_in = (qkv[:, a:b].unflatten(1, (-1, D)) for a, b in ((0, QR), (QR, QR + KV), (QR + KV, QR + 2 * KV)))
        for w, cache in zip(self.layers, self.caches):
            bi.bi_rmsnorm_quantize(h, add, w["norm1"], c.eps, None if add is None else h, codes["h"], s)
            bi.bi_linear_w8a8(codes["h"], s, *w["qkv"], qkv, self.ws)
            bi.bi_rope_append_kv4(q_in, k_in, v_in, self.rope, D, bi.BI_ROPE_HALF, q, cache, batch, w["q_norm"], w["k_norm"],
                                  c.eps)
            bi.bi_attention_kv4(q, cache, batch, D ** -0.5, o, self.attn_ws)
            bi.bi_quantize_act(o.view(T, QR), codes["o"], s)
            bi.bi_linear_w8a8(codes["o"], s, *w["o"], y["o"], self.ws)
            bi.bi_rmsnorm_quantize(h, y["o"], w["norm2"], c.eps, h, codes["h"], s)
            bi.bi_linear_w8a8(codes["h"], s, *w["gu"], y["gu"], self.ws)
            bi.bi_relu_mul_quantize(y["gu"], c.inner, codes["m"], s)
            bi.bi_linear_w8a8(codes["m"], s, *w["down"], y["down"], self.ws)
            add = y["down"]
        bi.bi_rmsnorm_quantize(h, add, self.norm, c.eps, h, codes["h"], s)
        logits = torch.empty((len(rows), c.vocab), dtype=torch.bfloat16, device=dev)
        bi.bi_linear_w8a8(codes["h"][rows], s[rows], *self.head, logits, self.ws)
        return logits


def draft_of(text: list[int], n: int) -> list[int]:
    """Up to n tokens that followed the last earlier occurrence of the text's last two."""
    for i in range(len(text) - 3, -1, -1):
        if text[i:i + 2] == text[-2:]:
            return text[i + 2:i + 2 + n]
    return []


def generate(model: Decoder, prompts: list[list[int]], new: int, draft: int = 0, repetition: float = 1.0, presence: float = 0.0,
             frequency: float = 0.0, mask: torch.Tensor | None = None):
    """`new` greedy tokens for each prompt, with up to `draft` drafted tokens a pass; mask: int32 words [1, ceil(vocab / 32)]
    of allowed tokens.  Returns the token lists and the number of passes."""
    c, dev, B = model.cfg, model.device, len(prompts)
    assert B == model.B and all(2 <= len(p) <= c.max_len - new - draft for p in prompts)
    texts = [list(p) for p in prompts]
    history = torch.zeros((B, c.max_len), dtype=torch.int32, device=dev)   # what the penalties look at
    counts, passes = [len(p) for p in prompts], 0
    drafts: list[list[int]] = [[] for _ in prompts]
    while True:
        # a pass: of each sequence the tokens that are not in the cache yet, and its drafts
        feed = [t[len(t) - n:] + d for t, n, d in zip(texts, counts, drafts)]
        lengths = [len(t) + len(d) for t, d in zip(texts, drafts)]
        for b, (t, n, f) in enumerate(zip(texts, counts, feed)):
            history[b, len(t) - n:len(t) - n + len(f)] = torch.tensor(f, dtype=torch.int32, device=dev)
        # logits of the last token and of the drafts
        first, rows, seqs, ends = 0, [], [], []
        for b, (t, n, f) in enumerate(zip(texts, counts, feed)):
            for i in range(n - 1, len(f)):
                rows.append(first + i)
                seqs.append(b)
                ends.append(b * c.max_len + len(t) - n + i + 1)
            first += len(f)
        M = len(rows)
        logits = model.forward(torch.tensor(sum(feed, []), dtype=torch.int32, device=dev), [len(f) for f in feed], lengths,
                               torch.tensor(rows, device=dev))

        def column(x, dtype):
            return torch.tensor(x, dtype=dtype, device=dev)
        rules = dict(ids=history.view(-1), begin=column([b * c.max_len for b in seqs], torch.int32),
                     mid=column([b * c.max_len + len(prompts[b]) for b in seqs], torch.int32), end=column(ends, torch.int32),
                     repetition=column([repetition] * M, torch.float32), presence=column([presence] * M, torch.float32),
                     frequency=column([frequency] * M, torch.float32))
        if mask is not None:
            rules["mask"] = mask.expand(M, -1).contiguous()
        choice = torch.empty(M, dtype=torch.int32, device=dev)
        bi.bi_logits_process(logits, bi.logits_rules(**rules), None, choice, model.logits_ws)
        passes += 1
        accepted, at = torch.empty((B, 2), dtype=torch.int32, device=dev), 0
        for b, d in enumerate(drafts):
            bi.bi_greedy_verify(choice[at:at + len(d) + 1], column(d, torch.int32) if d else None, accepted[b])
            at += len(d) + 1
        for b, (n, token) in enumerate(accepted.tolist()):
            texts[b] += drafts[b][:n] + [token]
        done = [len(t) - len(p) >= new for t, p in zip(texts, prompts)]
        if all(done):
            return [t[:len(p) + new] for t, p in zip(texts, prompts)], passes
        # a sequence that has its tokens goes along, one token at a time, and its text is not extended
        for b, t in enumerate(texts):
            texts[b] = t[:len(prompts[b]) + new]
        counts = [1] * B
        drafts = [[] if e or not draft else draft_of(t, min(draft, len(p) + new - len(t))) for t, p, e in
                  zip(texts, prompts, done)]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--new", type=int, default=64, help="tokens to generate")
    ap.add_argument("--draft", type=int, default=4, help="drafted tokens a pass")
    args = ap.parse_args()
    cfg = Config()
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, cfg.vocab, (n,), generator=gen).tolist() for n in (17, 300, 64)]
    model = Decoder(cfg, len(prompts))
    # a grammar of few tokens: random weights then repeat themselves, and drafts have something to find
    words = torch.zeros((1, (cfg.vocab + 31) // 32), dtype=torch.int32)
    words[0, 100], words[0, 700] = 0x0F, 0x0F
    mask = words.cuda()
    generate(model, prompts, 2, mask=mask)                 # first calls load the kernels
    outs = []
    for draft in (0, args.draft):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        texts, passes = generate(model, prompts, args.new, draft, mask=mask)
        torch.cuda.synchronize()
        print("%-11s %3d passes, %.1f ms a token" % ("speculative" if draft else "plain", passes,
                                                     (time.perf_counter() - t0) * 1e3 / args.new))
        outs.append(texts)
    assert bi.bi_workspace_status(model.attn_ws) == bi.BI_OK and bi.bi_workspace_status(model.ws) == bi.BI_OK
    assert outs[0] == outs[1], "speculative decoding changed the output"
    print("the same %d tokens for each of %d sequences" % (args.new, len(prompts)))


if __name__ == "__main__":
    main()
