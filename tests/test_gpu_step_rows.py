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
    for what, heads, each in (("16 rows, a span a CTA", 16, N), ("16 rows, clusters", 16, 60), ("8 rows of 16, clusters", 16, 10),
                              ("16 and 8 rows, a span a CTA", 24, N), ("16 and 8 rows, clusters", 24, 40),
                              ("8 rows, clusters", 8, 60)):
        bad = differ(s.attend(q[:, :heads], each), want[:, :heads].contiguous())
        assert bad == 0, "%s: %d elements of %d differ" % (what, bad, want[:, :heads].numel())
