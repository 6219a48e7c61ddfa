"""What a row of the attention and the append may depend on: its own query, positions and values, whatever form of
the kernel the call takes, whatever other rows see, and the bounds of the batch."""
import numpy as np
import pytest
import torch

from tests import step_ref as ref
from tests import test_gpu_step as step
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bi():
    import invariant_quantized_linear_gb300 as m
    return m


class Shared:
    """One cached sequence of k.shape[0] positions and one kv head, for any number of sequences that read it."""

    def __init__(self, bi, k, v, P=64):
        n, D = k.shape
        self.bi, self.n, self.D = bi, n, D
        self.pool = bi.new_kv4_pool(-(-n // P), 1, P, D)
        self.cache = bi.kv4_cache(self.pool, P, D)
        self.table = torch.arange(self.pool.shape[0], dtype=torch.int32, device=DEV)[None]
        x = [torch.from_numpy(y).to(DEV).bfloat16()[:, None] for y in (k, v)]
        cu, length = (torch.tensor(y, dtype=torch.int32, device=DEV) for y in ([0, n], [n]))
        none = torch.zeros((n, 1, D), dtype=torch.bfloat16, device=DEV)
        bi.bi_rope_append_kv4(none, *x, torch.zeros((n, 1, 2), device=DEV), 0, bi.BI_ROPE_HALF, torch.empty_like(none),
                              self.cache, bi.kv4_batch(cu, length, self.table, n, n, n))

    def attend(self, q, each, scale=0.125):
        """q bf16 [N, H, D], a token a sequence, `each` sequences a call."""
        o = torch.full_like(q, 7.0)
        for a in range(0, q.shape[0], each):
            x = q[a:a + each].contiguous()
            N = x.shape[0]
            d = (torch.arange(N + 1, dtype=torch.int32, device=DEV), torch.full((N,), self.n, dtype=torch.int32, device=DEV),
                 self.table.expand(N, -1).contiguous())     # a batch holds addresses: these live as long as it does
            batch = self.bi.kv4_batch(*d, N, 1, self.n)
            y = torch.empty_like(x)
            self.bi.bi_attention_kv4(x, self.cache, batch, scale, y,
                                     self.bi.new_attention_kv4_workspace(x.shape[1], self.cache, batch))
            o[a:a + each] = y
        return o


def differ(a, b):
    return int((a.view(torch.int16) != b.view(torch.int16)).sum())


def lane_sums(x, E):
    """fp32 sums of groups of 64, E elements one after the other, then halves of the lanes from the farthest: an order
    that depends on how many elements a lane holds."""
    lanes = np.zeros(x.shape[:-1] + (64 // E,), np.float32)
    y = x.reshape(*x.shape[:-1], 64 // E, E)
    for e in range(E):
        lanes = lanes + y[..., e]
    while lanes.shape[-1] > 1:
        h = lanes.shape[-1] // 2
        lanes = lanes[..., :h] + lanes[..., h:]
    return lanes[..., 0]


@pytest.mark.parametrize("D", [64, 128])
def test_queries_of_many_binades_in_every_form(bi, D):
    """Queries whose sums are not exact in fp32, over keys with minima: the same bits with 8 and with 16 rows a CTA, in a
    last block of 8, a span a CTA and a span a cluster."""
    rng = np.random.default_rng(D)
    n, N, H = 700, 300, 24
    s = Shared(bi, *(rng.normal(size=(2, n, D)) + np.float32([[[0.5]], [[0.0]]])).astype(np.float32))
    x = rng.normal(size=(N, H, D)) * np.exp(1.5 * rng.normal(size=(H, D))) * 2.0 ** -rng.integers(0, 12, (N, H, D))
    x = ref.bf16_round((x * 64 / np.linalg.norm(x, axis=-1, keepdims=True)).astype(np.float32))
    up = 2.0 ** (14 - np.floor(np.log2(np.abs(x).max(-1, keepdims=True))))
    g = (x * up).astype(np.float32).reshape(N, H, D // 64, 64)
    assert (lane_sums(g, D // 16) != lane_sums(g, D // 8)).mean() > 0.05      # the inputs can tell the orders apart
    q = torch.from_numpy(x).to(DEV).bfloat16()
    want = torch.cat([s.attend(q[:, h:h + 8], N) for h in (0, 8, 16)], 1)
    for what, heads, each in (("16 rows, a span a CTA", 16, N), ("16 rows, clusters", 16, 40), ("8 rows of 16, clusters", 16, 10),
                              ("16 and 8 rows, a span a CTA", 24, N), ("16 and 8 rows, clusters", 24, 20),
                              ("8 rows, clusters", 8, 60)):
        bad = differ(s.attend(q[:, :heads], each), want[:, :heads].contiguous())
        assert bad == 0, "%s: %d elements of %d differ" % (what, bad, want[:, :heads].numel())


# ------------------------------------------------------------------ values that are not finite

def verify_pass(bi, seqs, Hkv, D, P, copies=1, seed=5):
    """A batch of `copies` times the sequences, each on pages of its own, filled by the append."""
    rng = np.random.default_rng(seed)
    b = step.Batch(bi, [(n, n) for _, n in seqs] * copies, Hkv, D, P, seed=seed)
    b.pool[:] = 0
    b.to_device()
    x = torch.from_numpy(rng.normal(size=(2, b.T, Hkv, D)).astype(np.float32)).to(DEV).bfloat16()
    append(bi, b, *x)
    b.seqs = seqs * copies
    b.kv_x, b.first = x, b.cu
    b.cu = np.concatenate([[0], np.cumsum([q for q, _ in b.seqs])]).astype(np.int32)
    b.T = int(b.cu[-1])
    b.d[0] = torch.from_numpy(b.cu).to(DEV)
    b.batch = bi.kv4_batch(*b.d, b.T, max(q for q, _ in seqs), b.max_kv)
    return b


def append(bi, b, k, v):
    """k and v, not rotated, to the cache at the batch's positions."""
    none = torch.zeros((b.T, 1, b.D), dtype=torch.bfloat16, device=DEV)
    bi.bi_rope_append_kv4(none, k, v, torch.zeros((b.max_kv, 1, 2), device=DEV), 0, bi.BI_ROPE_HALF, torch.empty_like(none),
                          b.cache, b.batch)


@pytest.mark.parametrize("copies", [1, 40])
@pytest.mark.parametrize("D,P", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("kind", ["inf", "-inf", "nan scale", "inf minimum", "key"])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(bi, kind, D, P, copies):
    """A drafted token whose value (or key) has an element that is not finite: tokens before it have the bits that they have
    without it, those that see it NaN in the elements of its group and finite ones elsewhere."""
    Hq, Hkv = 4, 2
    seqs = [(5, 70), (3, 64), (4, 130), (9, 9)]
    at = [2, 1, 0, 7]                                          # the token that has it
    b = verify_pass(bi, seqs, Hkv, D, P, copies)
    rng = np.random.default_rng(1)
    q = torch.from_numpy(np.tile(rng.normal(size=(sum(n for n, _ in seqs), Hq, D)), (copies, 1, 1)).astype(np.float32)).to(DEV).bfloat16()
    clean = step.attend(bi, b, q, D ** -0.5)
    x = b.kv_x.clone()
    table, G = b.pages, D // 64
    for s, ((n_q, n), i) in enumerate(zip(b.seqs, at * copies)):
        pos = n - n_q + i
        if kind in ("inf", "-inf", "key"):
            x[0 if kind == "key" else 1, b.first[s] + pos, 1, 3] = float("-inf" if kind == "-inf" else "inf")
        else:                                                  # parameters of the first group of kv head 1's value
            words = b.d_pool[table[s, pos // P], 0, 1, P * D:].view(torch.int16).view(P, 2, G, 2)
            if kind == "nan scale":
                words[pos % P, 1, 0, 0] = 0x7FC0
            else:
                words[pos % P, 1, 0, 1] = 0x7F80
    if kind in ("inf", "-inf", "key"):
        whole, now = b.batch, b.T
        b.T = x.shape[1]
        cu = torch.from_numpy(b.first).to(DEV)
        b.batch = bi.kv4_batch(cu, b.d[1], b.d[2], b.T, max(n for _, n in seqs), b.max_kv)
        append(bi, b, *x)
        b.batch, b.T = whole, now
    o = step.attend(bi, b, q, D ** -0.5)
    value = lambda t: t.view(torch.bfloat16).float()
    for s, ((n_q, n), i) in enumerate(zip(b.seqs, at * copies)):
        a = b.cu[s]
        assert torch.equal(o[a:a + i], clean[a:a + i]), "sequence %d: a row before token %d" % (s, i)
        assert torch.equal(o[a:a + n_q, :2], clean[a:a + n_q, :2]), "sequence %d: the other kv head" % s
        if kind != "key":
            after = value(o[a + i:a + n_q, 2:])
            assert after[..., :64].isnan().all(), "sequence %d" % s
            # the other group: both results rounded to bf16, and their weights to f16, both ways; |v| < 6
            was = value(clean[a + i:a + n_q, 2:])[..., 64:]
            assert ((after[..., 64:] - was).abs() <= 2 * (was.abs() * 2.0 ** -8 + 6 * 2.0 ** -10)).all(), "sequence %d" % s


# ------------------------------------------------------------------ bounds of the batch

def test_positions_past_the_bound(bi):
    """Tokens at positions from max_kv on: zeros for q, not appended, gathered as zeros; the others as with a larger bound."""
    Hq, Hkv, D, P, bound = 2, 1, 64, 16, 37
    seqs = [(5, 40), (3, 20), (2, 31), (4, 60), (1, 37), (1, 38)]
    for rot, layout in ((64, "HALF"), (16, "HALF"), (32, "INTERLEAVED")):
        b = step.Batch(bi, seqs, Hkv, D, P, max_kv=bound)
        rng = np.random.default_rng(0)
        qkv = step.bits(rng, (b.T, Hq + 2 * Hkv, D))
        pos = np.concatenate([np.arange(n - q, n) for q, n in seqs])
        seq = np.repeat(np.arange(len(seqs)), [q for q, _ in seqs])
        rope = np.stack((np.ones((60, rot // 2)), np.zeros((60, rot // 2))), -1).astype(np.float32)
        x, want = ref.f32(qkv), b.pool.copy()
        for t in range(b.T):
            if pos[t] < bound:
                ref.write_position(want[b.pages[seq[t], pos[t] // P], 0, 0], P, D, pos[t] % P, x[t, Hq], x[t, Hq + 1])
        b.to_device()
        q_out = torch.full((b.T, Hq, D), 7, dtype=torch.int16, device=DEV)
        d = step.dev(qkv)
        bi.bi_rope_append_kv4(d[:, :2], d[:, 2:3], d[:, 3:], step.dev(rope), rot, getattr(bi, "BI_ROPE_" + layout), q_out,
                              b.cache, b.batch)
        step.same(step.host(b.d_pool), want, "cache")
        q_want = np.where((pos < bound)[:, None, None], qkv[:, :Hq], np.uint16(0))
        step.same(step.host(q_out), q_want, "q")
        k = torch.full((b.T, Hkv, D), 7, dtype=torch.int16, device=DEV)
        v = k.clone()
        bi.bi_kv4_gather(b.cache, b.batch, k, v)
        past = torch.from_numpy(pos >= bound).to(DEV)
        assert not k[past].any() and not v[past].any()
        b.batch = bi.kv4_batch(*b.d, b.T, b.max_q, 60)
        k2, v2 = torch.empty_like(k), torch.empty_like(v)
        bi.bi_kv4_gather(b.cache, b.batch, k2, v2)
        assert torch.equal(k[~past], k2[~past]) and torch.equal(v[~past], v2[~past])


BOUNDS = [
    # sequences (new, total), copies, Hq, Hkv, D, page, bound
    ([(5, 40), (3, 20), (2, 31), (4, 60), (1, 37), (1, 38)], 1, 4, 2, 64, 16, 37),
    ([(5, 40), (3, 20), (2, 31), (4, 60), (1, 37), (1, 38)], 40, 8, 2, 128, 32, 37),
    ([(20, 75), (20, 64)], 1, 4, 4, 128, 64, 64),
    ([(6, 4100), (2, 4099), (3, 2050)], 1, 8, 1, 64, 128, 4098),         # joined in the kernel
    ([(5, 32772), (2, 100)], 1, 2, 1, 64, 128, 32770),                   # and by a launch of its own
]


@pytest.mark.parametrize("seqs,copies,Hq,Hkv,D,P,bound", BOUNDS)
def test_attention_of_positions_past_the_bound(bi, seqs, copies, Hq, Hkv, D, P, bound):
    """Tokens at positions from max_kv on have zeros, the others what they have with a larger bound."""
    b = verify_pass(bi, seqs, Hkv, D, P, copies)
    gen = torch.Generator(device=DEV).manual_seed(bound)
    q = torch.randn((b.T, Hq, D), device=DEV, generator=gen).bfloat16()
    whole = step.attend(bi, b, q, D ** -0.5)
    most = max(n for n, _ in seqs)
    b.batch = bi.kv4_batch(*b.d, b.T, most, bound)
    o = step.attend(bi, b, q, D ** -0.5)
    pos = np.concatenate([np.arange(n - n_q, n) for n_q, n in b.seqs])
    past = torch.from_numpy(pos >= bound).to(DEV)
    assert past.any() and not past.all()
    assert not o[past].any(), "a token past the bound"
    assert torch.equal(o[~past], whole[~past]), "a token before the bound"


# ------------------------------------------------------------------ values that are zero, or nearly

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sigma", [0.0, 1e-27])
def test_blocks_of_small_values_far_below_the_maximum(bi, D, sigma):
    """Blocks whose values are zero or tiny and whose scores lie 11 to 20 binades below the row's largest: their part of
    the softmax sum is the same with a span a CTA as with a span a cluster."""
    rng = np.random.default_rng(7)
    n, N, H = 2048, 2000, 8
    k, v = np.zeros((n, D), np.float32), (rng.normal(size=(n, D)) * sigma).astype(np.float32)
    for p in (0, 64, 128, 192):                                # the first block of every chunk has one position that counts
        k[p, :4], v[p] = (15 / 15, 1 / 15, 2 / 15, 4 / 15), rng.normal(size=D)
    s = Shared(bi, k, v)
    q = rng.normal(size=(N, H, D)).astype(np.float32)
    q[..., 0] = rng.uniform(8, 14, (N, H)) / 0.125
    q[..., 1:4] *= 4                                           # scores of many different fractions
    q = torch.from_numpy(q).to(DEV).bfloat16()
    want = s.attend(q, N)
    bad = differ(s.attend(q, 60), want)
    assert bad == 0, "%d elements of %d differ" % (bad, want.numel())


# ------------------------------------------------------------------ append, several steps a warp

@pytest.mark.parametrize("seqs,Hq,Hkv,D,P,rot,inter,norm", [
    ([(1600, 1600)], 9, 5, 64, 16, 16, False, True),          # a warp a token: q, k and v heads one after the other
    ([(1600, 1700)], 9, 5, 64, 32, 64, True, False),
    ([(1700, 1700)], 7, 3, 128, 64, 32, False, True),
    ([(1600, 1600)], 7, 3, 128, 16, 64, True, True),
    ([(1600, 1650)], 13, 1, 128, 128, 64, False, False),      # more q heads than are in flight
    ([(700, 700), (300, 900)], 12, 4, 128, 64, 48, True, True),   # three warps a token: runs that end inside a kind
    ([(1000, 1000)], 12, 4, 128, 64, 64, False, True),
])
def test_append_of_prompts_in_every_layout(bi, seqs, Hq, Hkv, D, P, rot, inter, norm):
    """Heads rotated in part, or in pairs, in calls whose warps have several steps."""
    step.test_append_and_gather(bi, seqs, Hq, Hkv, D, P, rot, inter, norm)


@pytest.mark.parametrize("copies", [1, 60])
@pytest.mark.parametrize("D,P", [(64, 64), (128, 16)])
def test_a_seen_value_that_is_not_finite_spoils_its_group_alone(bi, D, P, copies):
    """An infinite value that every row of its block sees: NaN in its group, the head's other group and the other kv head
    as without it but for the weights' rounding."""
    b = verify_pass(bi, [(2, 300)], 2, D, P, copies)
    gen = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn((b.T, 8, D), device=DEV, generator=gen).bfloat16()
    value = lambda t: t.view(torch.bfloat16).float()
    clean = value(step.attend(bi, b, q, D ** -0.5))
    for s in range(copies):
        words = b.d_pool[int(b.pages[s, 70 // P]), 0, 1, P * D:].view(torch.int16).view(P, 2, D // 64, 2)
        words[70 % P, 1, 0, 0] = 0x7F80
    o = value(step.attend(bi, b, q, D ** -0.5))
    assert torch.equal(o[:, :4], clean[:, :4])
    assert o[:, 4:, :64].isnan().all()
    # both results rounded to bf16, and their weights to f16, both ways; |v| < 6
    was = clean[:, 4:, 64:]
    assert ((o[:, 4:, 64:] - was).abs() <= 2 * (was.abs() * 2.0 ** -8 + 6 * 2.0 ** -10)).all()
