"""The decoder-step operators on the GPU against their plain references: bit
for bit where the definition fixes every rounding (norm codes, rotations, the
packed cache, logits), within derived tolerances of fp64 elsewhere (the norm's
scale, attention); batch invariance, other streams, captured graphs."""
import numpy as np
import pytest
import torch

from tests import step_ref as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bi():
    import invariant_quantized_linear_gb300 as m
    return m


def bits(rng, shape, sigma=1.0):
    return ref.bf16_bits((rng.normal(size=shape) * sigma).astype(np.float32))


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).to(DEV)


def host(t):
    a = t.cpu().numpy()
    return a.view(np.uint16) if a.dtype == np.int16 else a


def same(got, want, what=""):
    bad = np.argwhere(got != want)
    assert bad.size == 0, "%s: %d of %d differ, first at %s" % (what, len(bad), got.size, bad[:3].tolist())


# ------------------------------------------------------------------ norm

NORM = [(1, 16, 0), (1, 4096, 0), (3, 48, 16), (5, 5136, 8), (7, 2048, 0), (2, 8192, 64), (2, 16384, 0), (3, 20000, 8),
        (300, 1040, 0)]


@pytest.mark.parametrize("M,K,pad", NORM)
@pytest.mark.parametrize("mode", ["add", "in place", "plain"])
def test_norm(bi, M, K, pad, mode):
    rng = np.random.default_rng(M * K)
    h, y = bits(rng, (M, K + pad), 3.0), bits(rng, (M, K + pad))
    w = bits(rng, K)
    if M > 2:
        h[1, :K], y[1, :K] = 0, 0x8000                   # zero row
        h[2, :K], y[2, :K] = 0, 0
        h[2, 5] = 0x0001                                # one subnormal element
    add = mode != "plain"
    want_h, want_q, want_s = ref.rmsnorm_quantize(h[:, :K], y[:, :K] if add else None, w, np.float32(1e-6))
    hd, yd, wd = dev(h), dev(y), dev(w)
    out = hd if mode == "in place" else torch.full((M, K + pad), 7, dtype=torch.int16, device=DEV)
    q = torch.full((M, K), 99, dtype=torch.int8, device=DEV)
    s = torch.full((M,), -1.0, device=DEV)
    bi.bi_rmsnorm_quantize(hd, yd if add else None, wd, 1e-6, out if add else None, q, s,
                           flags=bi.BI_FLAG_PDL if M % 2 else 0)
    same(host(q), want_q, "codes")
    if add:
        same(host(out)[:, :K], want_h, "h'")
        same(host(out)[:, K:], (h if mode == "in place" else np.full((M, K + pad), 7, np.uint16))[:, K:], "row padding")
    # positive terms: at most one rounding a step of the sum (8 a thread and chunk, 13 to join), halved by the root,
    # and six more roundings (mean, eps, root, division, st, product)
    steps = 8 * -(-K // 2048) + 13
    assert (np.abs(host(s) - want_s) <= want_s * (steps / 2 + 6) * 2.0 ** -24).all()


def test_norm_rows_do_not_depend_on_the_batch(bi):
    rng = np.random.default_rng(5)
    M, K = 33, 4096
    h, y, w = dev(bits(rng, (M, K))), dev(bits(rng, (M, K))), dev(bits(rng, K))

    def go(a, b):
        n = b - a
        o, q, s = torch.empty((n, K), dtype=torch.int16, device=DEV), torch.empty((n, K), dtype=torch.int8, device=DEV), \
            torch.empty(n, device=DEV)
        bi.bi_rmsnorm_quantize(h[a:b], y[a:b], w, 1e-5, o, q, s)
        return o, q, s
    whole = go(0, M)
    for r in (0, 17, 32):
        for x, z in zip(go(r, r + 1), whole):
            assert torch.equal(x[0], z[r])


# ------------------------------------------------------------------ cache

class Batch:
    """Sequences (new tokens, positions) with a shuffled page table, on both sides."""

    def __init__(self, bi, seqs, Hkv, D, P, seed=0, spare=2, max_q=None, max_kv=None, layers=1):
        rng = np.random.default_rng(seed)
        self.seqs, self.Hkv, self.D, self.P = seqs, Hkv, D, P
        need = [max(1, -(-n // P)) for _, n in seqs]
        self.n = sum(need) + spare
        order = rng.permutation(self.n).astype(np.int32)
        self.pages = np.full((len(seqs), max(need)), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.pages[b, :m] = order[at:at + m]
            at += m
        self.cu = np.concatenate([[0], np.cumsum([q for q, _ in seqs])]).astype(np.int32)
        self.len = np.array([n for _, n in seqs], np.int32)
        self.T = max(1, int(self.cu[-1]))
        # any bytes may stand in unused places, parameters that are NaN among them
        self.pool = rng.integers(0, 256, (self.n, layers, Hkv, ref.block_bytes(P, D))).astype(np.uint8)
        self.pool[:, :, :, P * D:][rng.random((self.n, layers, Hkv, P * 8 * (D // 64))) < 0.3] = 0xFF
        self.max_q = max_q or max(1, max(q for q, _ in seqs))
        self.max_kv = max_kv or max(1, max(n for _, n in seqs))
        self.bi = bi

    def fill(self, layer, k, v):
        """k, v: lists of fp32 [n, Hkv, D] per sequence (bf16 values)."""
        for b, (_, n) in enumerate(self.seqs):
            for p in range(n):
                for h in range(self.Hkv):
                    ref.write_position(self.pool[self.pages[b, p // self.P], layer, h], self.P, self.D, p % self.P,
                                       k[b][p, h], v[b][p, h])

    def to_device(self, layer=0):
        self.d_pool = torch.from_numpy(self.pool).to(DEV)
        self.d = [torch.from_numpy(x).to(DEV) for x in (self.cu, self.len, self.pages)]
        self.cache = self.bi.kv4_cache(self.d_pool[:, layer], self.P, self.D)
        self.batch = self.bi.kv4_batch(*self.d, self.T, self.max_q, self.max_kv)
        return self


APPEND = [
    # sequences (new, total), Hq, Hkv, D, page, rot, interleaved, norm
    ([(1, 1)], 1, 1, 64, 16, 64, False, False),
    ([(1, 1001)], 32, 8, 128, 16, 128, False, True),
    ([(5, 5), (0, 40), (1, 17), (17, 48)], 6, 2, 128, 16, 64, False, True),
    ([(3, 130), (7, 7), (2, 64)], 5, 5, 64, 32, 16, True, False),
    ([(40, 90)], 3, 1, 128, 64, 128, True, True),
    ([(9, 200), (1, 128), (4, 129)], 15, 5, 64, 128, 32, False, True),
    ([(2, 30)] * 70, 2, 1, 64, 16, 4, True, False),
    ([(6, 20)], 4, 2, 128, 16, 0, False, False),
]


@pytest.mark.parametrize("seqs,Hq,Hkv,D,P,rot,inter,norm", APPEND)
def test_append_and_gather(bi, seqs, Hq, Hkv, D, P, rot, inter, norm):
    rng = np.random.default_rng(Hq * D + P)
    b = Batch(bi, seqs, Hkv, D, P, seed=rot, layers=2)
    qkv = bits(rng, (b.T, Hq + 2 * Hkv, D)) if D == 64 else bits(rng, (b.T, Hq + 2 * Hkv, D), 4.0)
    qkv[0, Hq, 3] = ref.bf16_bits(np.float32([60.0]))[0]      # an outlier channel
    qkv[-1, Hq + Hkv, :] = 0x3F80                            # a constant value head: scale 0
    n_pos = max(n for _, n in seqs)
    inv = 1e4 ** (-np.arange(0, rot, 2) / max(rot, 1))
    ang = np.arange(n_pos)[:, None] * inv
    rope = np.stack((np.cos(ang), np.sin(ang)), -1).astype(np.float32) if rot else np.zeros((n_pos, 1, 2), np.float32)
    qn, kn = (bits(rng, D), bits(rng, D)) if norm else (None, None)
    eps = np.float32(1e-5)
    pos = np.concatenate([np.arange(n - q, n) for q, n in seqs])
    x = ref.f32(qkv)
    cs = rope[pos][:, :rot // 2]
    q_ref = ref.rotate(ref.head_norm(x[:, :Hq], qn, eps), cs, rot, inter)
    k_ref = ref.bf16_round(ref.rotate(ref.head_norm(x[:, Hq:Hq + Hkv], kn, eps), cs, rot, inter))
    v_ref = x[:, Hq + Hkv:]
    want = b.pool.copy()
    t = 0
    for s, (q, n) in enumerate(seqs):
        for p in range(n - q, n):
            for h in range(Hkv):
                ref.write_position(want[b.pages[s, p // P], 1, h], P, D, p % P, k_ref[t, h], v_ref[t, h])
            t += 1
    b.to_device(layer=1)
    d_qkv = dev(qkv)
    q_out = torch.full((b.T, Hq, D), 7, dtype=torch.int16, device=DEV)
    bi.bi_rope_append_kv4(d_qkv[:, :Hq], d_qkv[:, Hq:Hq + Hkv], d_qkv[:, Hq + Hkv:], dev(rope), rot,
                          bi.BI_ROPE_INTERLEAVED if inter else bi.BI_ROPE_HALF, q_out, b.cache, b.batch,
                          q_norm=None if qn is None else dev(qn), k_norm=None if kn is None else dev(kn), eps=float(eps))
    same(host(q_out), ref.bf16_bits(q_ref), "q")
    same(host(b.d_pool), want, "cache bytes")
    # against fp64: one bf16 rounding of q, and fp32 roundings of the norm and of two products and their sum
    x64 = x[:, :Hq].astype(np.float64)
    if norm:
        x64 = x64 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + float(eps)) * ref.f32(qn)
    exact = ref.rotate(x64, cs.astype(np.float64), rot, inter)
    size = np.abs(x64).max(-1, keepdims=True) * 1.5
    assert (np.abs(ref.f32(host(q_out)) - exact) <= np.abs(exact) * 2.0 ** -8 + size * 16 * 2.0 ** -24).all()
    k_out = torch.full((b.T, Hkv, D), 7, dtype=torch.int16, device=DEV)
    v_out = torch.full((b.T, Hkv, D), 7, dtype=torch.int16, device=DEV)
    bi.bi_kv4_gather(b.cache, b.batch, k_out, v_out)
    t = 0
    for s, (q, n) in enumerate(seqs):
        if q == 0:
            continue
        k, v, ok = ref.read_sequence(want[:, 1], P, D, b.pages[s], n)
        assert ok.all()
        same(host(k_out)[t:t + q], ref.bf16_bits(k[n - q:].astype(np.float32)), "gathered k")
        same(host(v_out)[t:t + q], ref.bf16_bits(v[n - q:].astype(np.float32)), "gathered v")
        t += q


def test_append_leaves_out_what_has_no_place(bi):
    """Negative positions, positions past the table of rotations or of pages, pages outside the pool, tokens past max_q."""
    Hq, Hkv, D, P = 2, 1, 64, 16
    seqs = [(3, 1), (4, 18), (2, 40), (6, 6)]
    b = Batch(bi, seqs, Hkv, D, P, max_q=4)
    b.pages = b.pages[:, :2].copy()                     # positions 32 .. have no column
    b.pages[1, 1] = b.n                                 # one past the pool
    rng = np.random.default_rng(0)
    qkv = bits(rng, (b.T, Hq + 2 * Hkv, D))
    rope = np.stack((np.ones((39, 32)), np.zeros((39, 32))), -1).astype(np.float32)   # position 39 is past it
    pos = np.concatenate([np.arange(n - q, n) for q, n in seqs])
    first = np.concatenate([np.arange(q) for q, _ in seqs])
    x, want = ref.f32(qkv), b.pool.copy()
    seq = np.repeat(np.arange(4), [q for q, _ in seqs])
    keep = (pos >= 0) & (pos < 39) & (first < 4)
    for t in range(b.T):
        page = b.pages[seq[t], pos[t] // P] if 0 <= pos[t] < 32 else -1
        if keep[t] and 0 <= page < b.n:
            ref.write_position(want[page, 0, 0], P, D, pos[t] % P, x[t, Hq], x[t, Hq + 1])
    b.to_device()
    q_out = torch.full((b.T, Hq, D), 7, dtype=torch.int16, device=DEV)
    d = dev(qkv)
    bi.bi_rope_append_kv4(d[:, :2], d[:, 2:3], d[:, 3:], dev(rope), 64, bi.BI_ROPE_HALF, q_out, b.cache, b.batch)
    same(host(b.d_pool), want, "cache")
    got = host(q_out)
    for t in range(b.T):
        same(got[t], qkv[t, :Hq] if keep[t] else np.zeros((Hq, D), np.uint16), "q of token %d" % t)
    k = torch.full((b.T, Hkv, D), 7, dtype=torch.int16, device=DEV)
    v = k.clone()
    bi.bi_kv4_gather(b.cache, b.batch, k, v)
    for t in range(b.T):
        page = b.pages[seq[t], pos[t] // P] if 0 <= pos[t] < 32 else -1
        if not (0 <= page < b.n) or first[t] >= 4:
            assert not k[t].any() and not v[t].any()


def test_rope_table(bi):
    inv = 1e6 ** (-np.arange(0, 128, 2) / 128) / 4.0
    n, amp = 131072, 1.25
    rope = torch.empty((n, 64, 2), device=DEV)
    bi.bi_rope_table(torch.from_numpy(inv).to(DEV), rope, amp)
    ang = np.arange(n)[:, None] * inv
    got = rope.cpu().numpy()
    # one fp32 rounding of a value of at most amp; fp64's own error at angles of 3e4 is far below
    assert np.abs(got[..., 0] - np.cos(ang) * amp).max() <= amp * 2.0 ** -24
    assert np.abs(got[..., 1] - np.sin(ang) * amp).max() <= amp * 2.0 ** -24


# ------------------------------------------------------------------ attention

def kv(rng, seqs, Hkv, D, sigma_k=1.0, sigma_v=1.0):
    make = lambda n, s: ref.bf16_round((rng.normal(size=(n, Hkv, D)) * s).astype(np.float32))
    return [make(n, sigma_k) for _, n in seqs], [make(n, sigma_v) for _, n in seqs]


def attend(bi, b, q, scale, ws=None, flags=0):
    Hq = q.shape[1]
    o = torch.full((b.T, Hq, b.D), 7, dtype=torch.int16, device=DEV)
    if ws is None:
        ws = bi.new_attention_kv4_workspace(Hq, b.cache, b.batch)
    bi.bi_attention_kv4(dev(q) if isinstance(q, np.ndarray) else q, b.cache, b.batch, scale, o, ws, flags=flags)
    return o


def check_attention(b, q, o, scale, layer=0):
    got = ref.f32(host(o)).astype(np.float64)
    for s, (n_q, n) in enumerate(b.seqs):
        if n_q == 0:
            continue
        k, v, ok = ref.read_sequence(b.pool[:, layer], b.P, b.D, b.pages[s], max(n, 0))
        a = b.cu[s]
        x = ref.f32(q[a:a + n_q]).astype(np.float64)
        want, mag, big = ref.attention(x, k, v, ok, n - n_q, scale)
        # bf16 of the result (half a step, 2^-8); weights rounded to f16 (2^-11 each way, in the sum and in the product);
        # scores off by a rounding per term of fp32 sums, exp and the joins a few more
        tol = np.abs(want) * 2.0 ** -8 + mag * (2.0 ** -10 + 2 * (b.D + 16) * 2.0 ** -24 * (big + 1))
        err = np.abs(got[a:a + n_q] - want)
        assert (err <= tol).all(), "sequence %d: off by %.3g of the tolerance" % (s, (err / np.maximum(tol, 1e-300)).max())


ATTENTION = [
    # sequences (new, total), Hq, Hkv, D, page
    ([(1, 1)], 1, 1, 64, 16),
    ([(1, 1)], 8, 2, 128, 128),
    ([(1, 15), (1, 16), (1, 17), (2, 2)], 4, 4, 128, 16),
    ([(1, 63), (1, 64), (1, 65), (3, 66)], 6, 2, 64, 32),
    ([(1, 511), (1, 512), (1, 513), (2, 513)], 4, 1, 128, 64),
    ([(8, 1030)], 8, 2, 128, 64),
    ([(0, 40), (1, 300), (0, 0), (5, 5), (2, 129)], 7, 1, 64, 128),
    ([(1, 0), (3, 2), (4, 0)], 4, 2, 64, 16),            # rows that see nothing
    ([(16, 100)], 8, 1, 128, 16),                        # 128 rows of one kv head
    ([(37, 37), (1, 90)], 3, 1, 128, 32),
    ([(5, 2100)], 5, 1, 64, 128),
    ([(1, 700)] * 20, 3, 3, 64, 16),
    ([(2, 1600), (1, 70)], 24, 2, 128, 64),              # groups of 12
]


@pytest.mark.parametrize("seqs,Hq,Hkv,D,P", ATTENTION)
def test_attention(bi, seqs, Hq, Hkv, D, P):
    rng = np.random.default_rng(len(seqs) * Hq + D)
    b = Batch(bi, seqs, Hkv, D, P, seed=1)
    b.fill(0, *kv(rng, seqs, Hkv, D))
    b.to_device()
    q = bits(rng, (b.T, Hq, D), 1.5)
    o = attend(bi, b, q, D ** -0.5)
    if b.cu[-1] == b.T:
        check_attention(b, q, o, D ** -0.5)
    for s, (n_q, n) in enumerate(seqs):
        for i in range(n_q):
            if n - n_q + i < 0:
                assert not o[b.cu[s] + i].any()


@pytest.mark.parametrize("sigma_k,sigma_v,sigma_q", [(12.0, 1.0, 2.0), (0.01, 1e-20, 1.0), (1.0, 1e20, 1.0), (1e-3, 1.0, 1e4),
                                                     (1e6, 1.0, 1e-6)])
def test_attention_ranges(bi, sigma_k, sigma_v, sigma_q):
    """Peaked scores; keys, values and queries of other magnitudes."""
    rng = np.random.default_rng(2)
    seqs, Hq, Hkv, D, P = [(4, 800), (1, 90)], 4, 2, 128, 32
    b = Batch(bi, seqs, Hkv, D, P)
    k, v = kv(rng, seqs, Hkv, D, sigma_k, sigma_v)
    v[0][::7] *= np.float32(2.0 ** -12)                    # positions of very different value scales
    v[0][5] = np.float32(sigma_v)                        # a constant value: scale 0
    k[0][6] = 0
    b.fill(0, k, v)
    b.to_device()
    q = bits(rng, (b.T, Hq, D), sigma_q)
    check_attention(b, q, attend(bi, b, q, D ** -0.5), D ** -0.5)


def test_attention_skips_pages_outside_the_pool(bi):
    rng = np.random.default_rng(4)
    seqs, Hq, Hkv, D, P = [(3, 300), (2, 50)], 4, 2, 64, 16
    b = Batch(bi, seqs, Hkv, D, P)
    b.fill(0, *kv(rng, seqs, Hkv, D))
    b.pages[0, 3] = -1
    b.pages[0, 4] = b.n
    b.pages[0, 18] = 2 ** 31 - 1
    b.pages[1, :] = -5                                  # nothing left: zeros
    b.to_device()
    q = bits(rng, (b.T, Hq, D))
    o = attend(bi, b, q, 0.125)
    check_attention(b, q, o, 0.125)
    assert not o[3:].any()


def test_attention_rows_do_not_depend_on_the_batch(bi):
    """The same bits alone and in a batch, one query at a time and many, with other bounds and with a longer cache."""
    rng = np.random.default_rng(6)
    Hq, Hkv, D, P = 8, 2, 128, 16
    seqs = [(9, 2600), (1, 700), (4, 513), (2, 64)]
    b = Batch(bi, seqs, Hkv, D, P, seed=3)
    b.fill(0, *kv(rng, seqs, Hkv, D))
    b.to_device()
    q = bits(rng, (b.T, Hq, D), 2.0)
    whole = host(attend(bi, b, q, 0.09))
    d_q = dev(q)
    for s, (n_q, n) in enumerate(seqs):
        for i in range(n_q):
            t = b.cu[s] + i
            one = Batch.__new__(Batch)
            one.T, one.D = 1, D
            one.d = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1], [n - n_q + i + 1], [b.pages[s].tolist()])]
            one.cache = b.cache
            for max_kv in (n, 5000):
                one.batch = bi.kv4_batch(*one.d, 1, 1, max_kv)
                o = attend(bi, one, d_q[t:t + 1], 0.09)
                same(host(o)[0], whole[t], "token %d alone" % t)
    # many copies of the sequences: another split of the work over the GPU
    R = 40
    many = Batch.__new__(Batch)
    many.T, many.D = b.T * R, D
    cu = np.concatenate([[0], np.cumsum([n for n, _ in seqs] * R)]).astype(np.int32)
    many.d = [torch.from_numpy(x).to(DEV) for x in (cu, np.tile(b.len, R), np.tile(b.pages, (R, 1)))]
    many.cache = b.cache
    many.batch = bi.kv4_batch(*many.d, many.T, 9, 2600)
    o = host(attend(bi, many, np.tile(q, (R, 1, 1)), 0.09)).reshape(R, b.T, Hq, D)
    for r in range(R):
        same(o[r], whole, "copy %d" % r)


def test_attention_strided_queries_streams_and_one_workspace(bi):
    """q as a part of a packed row; a side stream; one workspace through calls of other shapes, large and small."""
    rng = np.random.default_rng(8)
    cases = []
    for seqs, Hq, Hkv, D, P in (([(3, 900), (1, 33)], 8, 2, 128, 32), ([(1, 40)], 4, 4, 64, 16), ([(12, 1500)], 6, 2, 64, 64)):
        b = Batch(bi, seqs, Hkv, D, P)
        b.fill(0, *kv(rng, seqs, Hkv, D))
        b.to_device()
        q = bits(rng, (b.T, Hq + 3, D))
        cases.append((b, q, dev(q), dev(q[:, 2:2 + Hq].copy())))
    ws = torch.zeros(max(bi.bi_attention_kv4_workspace_size(c[3].shape[1], c[0].cache, c[0].batch) for c in cases),
                     dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        for b, q, packed, alone in cases:
            plain = attend(bi, b, alone, 0.1)
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                o = attend(bi, b, packed[:, 2:2 + alone.shape[1]], 0.1, ws=ws, flags=bi.BI_FLAG_PDL)
            torch.cuda.synchronize()
            assert torch.equal(o, plain)


def test_step_in_a_graph_with_other_lengths(bi):
    """Append and attention captured once, replayed as the sequences grow: the lengths and pages are read on the device."""
    rng = np.random.default_rng(9)
    Hq, Hkv, D, P, cap = 4, 2, 64, 16, 200
    b = Batch(bi, [(2, cap), (1, cap)], Hkv, D, P)
    b.pool[:] = 0
    b.to_device()
    qkv = dev(bits(rng, (3, Hq + 2 * Hkv, D)))
    ang = np.arange(cap)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)
    rope = dev(np.stack((np.cos(ang), np.sin(ang)), -1).astype(np.float32))
    q_out = torch.empty((3, Hq, D), dtype=torch.int16, device=DEV)
    o = torch.empty_like(q_out)
    ws = bi.new_attention_kv4_workspace(Hq, b.cache, b.batch)

    def step():
        bi.bi_rope_append_kv4(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], rope, D, bi.BI_ROPE_HALF, q_out, b.cache,
                              b.batch)
        bi.bi_attention_kv4(q_out, b.cache, b.batch, 0.125, o, ws, flags=bi.BI_FLAG_PDL)
    b.d[1].copy_(torch.tensor([2, 1]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for n in (2, 40, 41, 150):
        x = dev(bits(rng, (3, Hq + 2 * Hkv, D)))
        qkv.copy_(x)
        b.d[1].copy_(torch.tensor([n, n + 1]))
        graph.replay()
        got = o.clone()
        o.fill_(7)
        step()
        assert torch.equal(got, o)
        b.pool = b.d_pool.cpu().numpy()
        b.seqs = [(2, n), (1, n + 1)]
        check_attention(b, host(q_out), o, 0.125)


# ------------------------------------------------------------------ logits

def rules_case(rng, M, V, kind):
    r = {}
    if "hist" in kind:
        n = rng.integers(0, 60, M)
        begin = np.concatenate([[0], np.cumsum(n)[:-1]])
        ids = rng.integers(0, max(2, V // 3), int(n.sum()) + 1)
        ids[::9] = [-1, V, 2 ** 31 - 1, -2 ** 31][M % 4]          # no token
        r.update(ids=ids.astype(np.int32), begin=begin.astype(np.int32), end=(begin + n).astype(np.int32),
                 mid=(begin + n // 2).astype(np.int32))
        if "pen" in kind:
            r.update(repetition=(1 + rng.random(M)).astype(np.float32), presence=rng.normal(size=M).astype(np.float32),
                     frequency=rng.normal(size=M).astype(np.float32))
    if "bias" in kind:
        r["bias_ids"] = rng.integers(-2, V + 2, (M, 17)).astype(np.int32)     # some equal, some outside
        r["bias"] = (5 * rng.normal(size=(M, 17))).astype(np.float32)
    if "mask" in kind:
        m = rng.integers(0, 2 ** 32, (M, (V + 31) // 32 + 2), dtype=np.uint64).astype(np.uint32)
        m[rng.random(m.shape) < 0.5] = 0
        if M > 2:
            m[2] = 0
        r["mask"] = m.view(np.int32)
    return r


@pytest.mark.parametrize("M,V,ldl,ldo", [(1, 1, 1, 1), (3, 31, 31, 31), (4, 4095, 4097, 4096), (2, 4096, 4096, 4096),
                                        (5, 32003, 32003, 32005), (7, 9000, 9008, 9000), (40, 12289, 12296, 12292)])
@pytest.mark.parametrize("kind", ["none", "hist", "hist pen", "bias", "mask", "hist pen bias mask"])
def test_logits(bi, M, V, ldl, ldo, kind):
    rng = np.random.default_rng(V + M)
    x = bits(rng, (M, ldl), 3.0)
    x[:, ::5] = ref.bf16_bits(np.float32([2.5]))[0]                  # ties
    if M > 3:
        x[1, V // 2] = 0x7FC0                                       # NaN
        x[3, :V:2], x[3, 1:V:2] = 0x8000, 0xFF80                    # -0 and -inf
    r = rules_case(rng, M, V, kind)
    want, best = ref.logits_process(x, V, **{k: v for k, v in r.items()})
    d = {k: dev(v) for k, v in r.items()}
    rules = bi.logits_rules(**d)
    dx = dev(x)[:, :V]
    ws = bi.new_logits_workspace(M)
    full = torch.full((M, ldo), 7.0, device=DEV)
    out, am = full[:, :V], torch.full((M,), -7, dtype=torch.int32, device=DEV)
    for want_out, want_am in ((True, True), (True, False), (False, True)):
        full.fill_(7.0)
        am.fill_(-7)
        bi.bi_logits_process(dx, rules, out if want_out else None, am if want_am else None, ws,
                             flags=bi.BI_FLAG_PDL if want_am else 0)
        if want_out:
            g = host(full)
            nan = np.isnan(want)
            assert np.array_equal(np.isnan(g[:, :V]), nan)
            same(np.where(nan, 0, g[:, :V]), np.where(nan, 0, want), "logits")
            assert (g[:, V:] == 7).all()
        if want_am:
            same(host(am), best, "argmax")
    assert not ws.any()


def test_logits_many_rows(bi):
    """Enough rows for the long slices: a few random rows of them against the reference, all of them against the same rows
    a few at a time (short slices)."""
    rng = np.random.default_rng(21)
    M, V = 170, 16389                                           # three slices of 8192
    x = bits(rng, (M, V + 2), 3.0)
    r = rules_case(rng, M, V, "hist pen bias mask")
    d = {k: dev(v) for k, v in r.items()}
    dx = dev(x)[:, :V]
    ws = bi.new_logits_workspace(M)
    out, am = torch.empty((M, V), device=DEV), torch.empty(M, dtype=torch.int32, device=DEV)
    bi.bi_logits_process(dx, bi.logits_rules(**d), out, am, ws)
    for a in range(0, M, 17):
        part = {k: v if k == "ids" else v[a:a + 17] for k, v in r.items()}
        if a % 51 == 0:
            want, best = ref.logits_process(x[a:a + 17], V, **part)
            same(host(out)[a:a + 17], want, "logits")
            same(host(am)[a:a + 17], best, "argmax")
        o2, a2 = torch.empty((17, V), device=DEV), torch.empty(17, dtype=torch.int32, device=DEV)
        bi.bi_logits_process(dx[a:a + 17], bi.logits_rules(**{k: dev(v) for k, v in part.items()}), o2, a2, ws)
        assert torch.equal(o2, out[a:a + 17]) and torch.equal(a2, am[a:a + 17])
    assert not ws.any()


def test_logits_more_marked_elements_than_are_done_at_once(bi):
    """A history that meets nearly every element of its row, in rows of long and of short slices."""
    rng = np.random.default_rng(22)
    V = 16500
    for M in (1, 320):
        x = bits(rng, (M, V), 3.0)
        n = 40000
        ids = rng.integers(0, V, n).astype(np.int32)
        begin = np.full(M, 3, np.int32)
        r = dict(ids=ids, begin=begin, mid=begin + 12345, end=np.full(M, n - 1, np.int32),
                 repetition=np.full(M, 1.25, np.float32), presence=rng.normal(size=M).astype(np.float32),
                 frequency=rng.normal(size=M).astype(np.float32), bias_ids=rng.integers(0, V, (M, 300)).astype(np.int32),
                 bias=rng.normal(size=(M, 300)).astype(np.float32))
        out, am = torch.empty((M, V), device=DEV), torch.empty(M, dtype=torch.int32, device=DEV)
        ws = bi.new_logits_workspace(M)
        bi.bi_logits_process(dev(x), bi.logits_rules(**{k: dev(v) for k, v in r.items()}), out, am, ws)
        some = slice(0, 2)
        want, best = ref.logits_process(x[some], V, **{k: v if k == "ids" else v[some] for k, v in r.items()})
        same(host(out)[some], want, "logits")
        same(host(am)[some], best, "argmax")


def test_attention_leaves_out_tokens_past_the_bound(bi):
    """Tokens past max_q have zeros, those before it their result, also where T does not show that there are any."""
    rng = np.random.default_rng(12)
    seqs, Hq, Hkv, D, P = [(6, 1500), (0, 9), (1, 40)], 4, 2, 64, 32
    b = Batch(bi, seqs, Hkv, D, P)
    b.fill(0, *kv(rng, seqs, Hkv, D))
    b.to_device()
    q = bits(rng, (b.T, Hq, D))
    whole = attend(bi, b, q, 0.1)
    b.batch = bi.kv4_batch(*b.d, b.T, 3, b.max_kv)
    o = attend(bi, b, q, 0.1)
    assert torch.equal(o[:3], whole[:3]) and torch.equal(o[6], whole[6]) and not o[3:6].any()
    b.batch = bi.kv4_batch(*b.d, 5, 6, b.max_kv)              # rows from T on are not touched
    o = attend(bi, b, q, 0.1)
    assert torch.equal(o[:5], whole[:5]) and (o[5:] == 7).all()


def test_attention_status(bi):
    """A call leaves the status at BI_OK; what a timeout would leave (set here) is reported once."""
    rng = np.random.default_rng(13)
    seqs = [(1, 70)]
    b = Batch(bi, seqs, 1, 64, 16)
    b.fill(0, *kv(rng, seqs, 1, 64))
    b.to_device()
    ws = bi.new_attention_kv4_workspace(2, b.cache, b.batch)
    o = torch.empty((1, 2, 64), dtype=torch.int16, device=DEV)
    bi.bi_attention_kv4(dev(bits(rng, (1, 2, 64))), b.cache, b.batch, 0.1, o, ws)
    assert bi.bi_workspace_status(ws) == bi.BI_OK
    ws.view(torch.int32)[0] = 1
    assert bi.bi_workspace_status(ws) == bi.BI_ERR_TIMEOUT
    assert bi.bi_workspace_status(ws) == bi.BI_OK


@pytest.mark.parametrize("M,V,most", [(160, 70000, 3000), (70, 150001, 9000), (620, 9001, 5000), (330, 20000, 2500)])
def test_logits_long_slices(bi, M, V, most):
    """Enough rows for long slices, one to ten a row: histories of no token, of ids that are none, of more in a slice than
    is kept between the passes; against the reference, and against the same rows a few at a time."""
    rng = np.random.default_rng(M)
    x = bits(rng, (M, V), 3.0)
    n = rng.integers(0, most, M)
    n[:4] = 0, 1, most, min(2 * most, 5000)
    begin = np.concatenate([[0], np.cumsum(n)])[:-1].astype(np.int32) + 1
    ids = rng.integers(-5, V + 5, int(n.sum()) + 2).astype(np.int32)
    ids[begin[2]:begin[2] + most // 2] = V - 1                  # one slice has most of them
    r = dict(ids=ids, begin=begin, mid=(begin + n // 3).astype(np.int32), end=(begin + n).astype(np.int32),
             repetition=np.full(M, 1.25, np.float32), presence=rng.normal(size=M).astype(np.float32),
             frequency=rng.normal(size=M).astype(np.float32), bias_ids=rng.integers(0, V, (M, 20)).astype(np.int32),
             bias=rng.normal(size=(M, 20)).astype(np.float32))
    d, dx = {k: dev(v) for k, v in r.items()}, dev(x)
    ws = bi.new_logits_workspace(M)
    out, am = torch.empty((M, V), device=DEV), torch.empty(M, dtype=torch.int32, device=DEV)
    bi.bi_logits_process(dx, bi.logits_rules(**d), out, am, ws)
    want, best = ref.logits_process(x[:5], V, **{k: v if k == "ids" else v[:5] for k, v in r.items()})
    same(host(out)[:5], want, "logits")
    same(host(am)[:5], best, "argmax")
    for a in range(0, M, 10):
        part = {k: v if k == "ids" else v[a:a + 10].contiguous() for k, v in d.items()}
        m = part["begin"].shape[0]
        o2, a2 = torch.empty((m, V), device=DEV), torch.empty(m, dtype=torch.int32, device=DEV)
        bi.bi_logits_process(dx[a:a + 10], bi.logits_rules(**part), o2, a2, ws)
        assert torch.equal(o2, out[a:a + 10]) and torch.equal(a2, am[a:a + 10])
    assert not ws.any()


@pytest.mark.parametrize("seqs,Hq,Hkv,D,P,norm", [
    ([(300, 300), (220, 500)], 64, 8, 128, 16, True),          # several batches of q heads a warp, the last one short
    ([(1300, 1300)], 13, 3, 64, 32, True),
    ([(2500, 2500)], 7, 1, 64, 64, True),                       # a warp a token
    ([(130, 130)], 9, 9, 128, 128, False),
    ([(1, 77), (2, 5)], 1, 1, 128, 16, True)])
def test_append_whole_heads(bi, seqs, Hq, Hkv, D, P, norm):
    """All of a head rotated in the half layout: heads of many and of few tokens, odd counts, one kv head."""
    test_append_and_gather(bi, seqs, Hq, Hkv, D, P, D, False, norm)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rot", [16, "D"])
def test_append_scales(bi, D, rot):
    """Groups of every kind at position 0, where a rotation changes nothing but a zero's sign: zeros of both signs,
    constants, scales that are subnormal, tiny and huge, one element apart from the rest."""
    rng = np.random.default_rng(D)
    Hkv, P = 24, 16
    x = rng.normal(size=(2, Hkv, D)).astype(np.float32) * 2.0 ** np.linspace(-126, 100, Hkv)[:, None].astype(np.float32)
    x[:, 0], x[:, 1], x[:, 2] = 0.0, -0.0, -3.5
    x[:, 3], x[:, 3, D // 2 + 1] = 1.0, 1.0078125
    x[:, 4, ::2], x[:, 4, 1::2] = 0.0, 1e-40
    x[:, 5, 1:], x[:, 5, 0] = 2.0 ** -9, 300.0
    x[:, 6, :D // 2], x[:, 6, D // 2:] = 2.0 ** -120, 2.0 ** 90
    rot = D if rot == "D" else rot
    b = Batch(bi, [(1, 1)], Hkv, D, P)
    k, v = ref.bf16_bits(x)
    want = b.pool.copy()
    rope = np.stack((np.ones((1, rot // 2)), np.zeros((1, rot // 2))), -1).astype(np.float32)
    k_ref = ref.bf16_round(ref.rotate(ref.f32(k)[None], rope, rot, False))[0]
    for h in range(Hkv):
        ref.write_position(want[b.pages[0, 0], 0, h], P, D, 0, k_ref[h], ref.f32(v[h]))
    b.to_device()
    q_out = torch.empty((1, 1, D), dtype=torch.int16, device=DEV)
    bi.bi_rope_append_kv4(dev(k[None, :1]), dev(k[None]), dev(v[None]), dev(rope), rot, bi.BI_ROPE_HALF, q_out, b.cache, b.batch)
    same(host(b.d_pool), want, "cache bytes")


@pytest.mark.parametrize("K", [1024, 2064, 4096, 5136, 8192, 10256, 16384])
def test_norm_forms_give_the_same_bits(bi, K):
    """Rows of a call large enough for one form against the same rows alone, which take another."""
    rng = np.random.default_rng(K)
    M = 700
    h, y, w = dev(bits(rng, (M, K), 2.0)), dev(bits(rng, (M, K))), dev(bits(rng, K))

    def go(a, b):
        n = b - a
        o, q, s = torch.empty((n, K), dtype=torch.int16, device=DEV), torch.empty((n, K), dtype=torch.int8, device=DEV), \
            torch.empty(n, device=DEV)
        bi.bi_rmsnorm_quantize(h[a:b], y[a:b], w, 1e-5, o, q, s)
        return o, q, s
    whole = go(0, M)
    for a, b in ((0, 1), (1, 300), (300, 500), (699, 700)):
        for x, z in zip(go(a, b), whole):
            assert torch.equal(x, z[a:b])


LONG = [
    # sequences (new, total), Hq, Hkv, D, page, bound on the positions
    ([(1, 4104)], 32, 8, 128, 64, 4104),                   # three spans of clusters, joined rank by rank
    ([(8, 4104)], 32, 8, 128, 16, 9000),                   # 32 rows, a bound past the sequence
    ([(1, 33000), (2, 32768), (1, 32769)], 2, 1, 64, 128, 33000),   # 17 spans: joined by a launch of its own
    ([(5, 40000), (3, 70)], 7, 1, 64, 128, 40000),         # 35 rows: two blocks of 16 and one of 3
    ([(1, 5000 - 7 * i) for i in range(40)], 8, 4, 128, 16, 5000),  # a span a CTA, joined by counters
    ([(3, 2500 + i) for i in range(30)], 12, 2, 128, 32, 4000),     # 18 rows: a block of 16 and one of 2
    ([(2, 2049 + 300 * i) for i in range(24)], 10, 2, 64, 16, 9000),
    ([(130, 2200), (64, 64)], 4, 2, 128, 64, 2200),        # a prefill: hundreds of rows
]


@pytest.mark.parametrize("seqs,Hq,Hkv,D,P,bound", LONG)
def test_attention_long(bi, seqs, Hq, Hkv, D, P, bound):
    """Contexts of several spans, filled by the append, in every split of the work; each sequence alone has the same bits."""
    rng = np.random.default_rng(Hq * D + bound)
    gen = torch.Generator(device=DEV).manual_seed(bound)
    total = [n for _, n in seqs]
    b = Batch(bi, [(n, n) for n in total], Hkv, D, P, seed=2)
    b.to_device()
    kv_in = torch.randn((2, b.T, Hkv, D), device=DEV, generator=gen).bfloat16()
    none = torch.zeros((b.T, 1, D), dtype=torch.bfloat16, device=DEV)
    bi.bi_rope_append_kv4(none, kv_in[0], kv_in[1], torch.zeros((max(total), 1, 2), device=DEV), 0, bi.BI_ROPE_HALF,
                          torch.empty_like(none), b.cache, b.batch)
    b.pool = b.d_pool.cpu().numpy()
    b.seqs = seqs
    b.cu = np.concatenate([[0], np.cumsum([q for q, _ in seqs])]).astype(np.int32)
    b.T = int(b.cu[-1])
    b.d[0] = torch.from_numpy(b.cu).to(DEV)
    most = max(q for q, _ in seqs)
    b.batch = bi.kv4_batch(*b.d, b.T, most, bound)
    q = bits(rng, (b.T, Hq, D), 1.5)
    o = attend(bi, b, q, D ** -0.5)
    got = torch.from_numpy(ref.f32(host(o))).to(DEV).double()
    for s in sorted({0, 1 % len(seqs), len(seqs) - 1}):
        n_q, n = seqs[s]
        k, v, ok = ref.read_sequence(b.pool[:, 0], P, D, b.pages[s], n)
        assert ok.all()
        k, v = (torch.from_numpy(x).to(DEV).double().repeat_interleave(Hq // Hkv, 1) for x in (k, v))
        x = torch.from_numpy(ref.f32(q[b.cu[s]:b.cu[s] + n_q])).to(DEV).double()
        scores = torch.einsum("qhd,nhd->qhn", x, k) * D ** -0.5
        hidden = torch.arange(n, device=DEV)[None] > n - n_q + torch.arange(n_q, device=DEV)[:, None]
        scores.masked_fill_(hidden[:, None], float("-inf"))
        p = scores.softmax(-1)
        want, mag = torch.einsum("qhn,nhd->qhd", p, v), torch.einsum("qhn,nhd->qhd", p, v.abs())
        big = (torch.einsum("qhd,nhd->qhn", x.abs(), k.abs()) * D ** -0.5).amax(-1, keepdim=True)
        tol = want.abs() * 2.0 ** -8 + mag * (2.0 ** -10 + 2 * (D + 16) * 2.0 ** -24 * (big + 1))
        assert ((got[b.cu[s]:b.cu[s] + n_q] - want).abs() <= tol).all(), "sequence %d" % s
        alone = Batch.__new__(Batch)
        alone.T, alone.D, alone.cache = n_q, D, b.cache
        alone.d = [torch.tensor(y, dtype=torch.int32, device=DEV) for y in ([0, n_q], [n], [b.pages[s].tolist()])]
        alone.batch = bi.kv4_batch(*alone.d, n_q, n_q, n)
        same(host(attend(bi, alone, q[b.cu[s]:b.cu[s] + n_q], D ** -0.5)), host(o)[b.cu[s]:b.cu[s] + n_q], "alone")


def test_cache_past_32_bits(bi):
    """Pages beyond the first 4 GiB of a pool: the same bytes, gathered values and attention as in a small pool."""
    Hq, Hkv, D, P, n = 16, 8, 128, 128, 700
    far = 2 ** 32 // (Hkv * bi.bi_kv4_block_bytes(P, D)) + 20
    gen = torch.Generator(device=DEV).manual_seed(0)
    qkv = torch.randn((n, Hq + 2 * Hkv, D), device=DEV, generator=gen).bfloat16()
    rope = torch.zeros((n, D // 2, 2), device=DEV)
    bi.bi_rope_table(1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=DEV) / D), rope)
    outs = []
    for pages, where in ((10, range(6)), (far, range(far - 6, far))):
        pool = torch.empty((pages, Hkv, bi.bi_kv4_block_bytes(P, D)), dtype=torch.uint8, device=DEV)
        pool[list(where)] = 0
        table = torch.tensor([list(where)], dtype=torch.int32, device=DEV)
        cu, length = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, n], [n]))
        c, batch = bi.kv4_cache(pool, P, D), bi.kv4_batch(cu, length, table, n, n, n)
        q, k, v = (torch.empty((n, h, D), dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
        o = torch.empty_like(q)
        bi.bi_rope_append_kv4(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], rope, D, bi.BI_ROPE_HALF, q, c, batch)
        bi.bi_kv4_gather(c, batch, k, v)
        bi.bi_attention_kv4(q, c, batch, D ** -0.5, o, bi.new_attention_kv4_workspace(Hq, c, batch))
        outs.append([pool[list(where)], q, k, v, o])
    for x, y in zip(*outs):
        assert torch.equal(x, y)
