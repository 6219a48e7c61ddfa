"""The e4m3 linears, the quantisers and the weighted sum on operands past 4 GiB and at the most rows: rows from both ends of
them have the bits that they have in a small call."""
import pytest
import torch

from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bi():
    import invariant_quantized_linear_gb300 as m
    return m


@pytest.fixture(scope="module")
def ws(bi):
    w = bi.new_f8_workspace()
    yield w
    assert bi.bi_workspace_status(w) == bi.BI_OK


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def codes(*shape):
    """Random codes, none of them NaN."""
    return torch.randint(0, 127, shape, dtype=torch.uint8, device=DEV)


def scales(*shape):
    return torch.rand(shape, device=DEV) + 0.5


def bits(t):
    return t.view(torch.int16)


def picked(M):
    return torch.tensor([0, 1, M // 2, M - 130, M - 2, M - 1], device=DEV)


@pytest.mark.parametrize("gate", [None, 0, 1])
def test_quantisers(bi, gate):
    M, K = 1 << 20, 2064                                       # x: 4.3 GB, behind a gate 8.7
    x = torch.randn((1, 2 * K), device=DEV).bfloat16().repeat(M, 1) if gate is not None else \
        torch.randn((1, K), device=DEV).bfloat16().repeat(M, 1)
    rows = picked(M)
    x[rows] = torch.randn((len(rows), x.shape[1]), device=DEV).bfloat16()

    def run(x):
        q, s = torch.empty((len(x), K), dtype=torch.uint8, device=DEV), torch.empty((len(x), 17), device=DEV)
        if gate is None:
            bi.bi_quantize_act_f8(x, q, s)
        else:
            bi.bi_gated_quantize_f8(x, gate, q, s)
        return q, s
    q, s = run(x)
    want_q, want_s = run(x[rows])
    assert torch.equal(q[rows], want_q) and torch.equal(s[rows], want_s)


def test_weight_quantiser(bi):
    N, K = (1 << 20) + 40, 1040                                # w: 4.4 GB; blocks of 128 rows
    w = torch.randn((1, K), device=DEV).repeat(N, 1)
    first = (N - 40) // 128 * 128
    w[first:] = torch.randn((N - first, K), device=DEV)

    def run(w):
        q = torch.empty(w.shape, dtype=torch.uint8, device=DEV)
        s = torch.empty((-(-len(w) // 128), 9), device=DEV)
        bi.bi_quantize_weight_f8(w, q, s)
        return q, s
    q, s = run(w)
    want_q, want_s = run(w[first:].contiguous())
    assert torch.equal(q[first:], want_q) and torch.equal(s[first // 128:], want_s)


@pytest.mark.parametrize("M, K, N", [(1 << 20, 4224, 16), (1 << 20, 16, 2200), (3, 16, 1 << 24), (200, 528, 1 << 23)])
def test_linear(bi, ws, M, K, N):
    """q, y and w past 4 GiB; the most rows and columns."""
    q, s_a, w, s_w = codes(M, K), scales(M, -(-K // 128)), codes(N, K), scales(-(-N // 128), -(-K // 128))
    y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    bi.bi_linear_f8(q, s_a, w, s_w, y, ws)
    rows = picked(M) if M > 200 else torch.arange(min(M, 6), device=DEV)
    n = (N - 1) // 128 * 128 if N > 5000 else 0                # the last columns alone, from a block of the weights on
    want = torch.empty((len(rows), N - n), dtype=torch.bfloat16, device=DEV)
    bi.bi_linear_f8(q[rows], s_a[rows], w[n:], s_w[n // 128:], want, ws)
    assert torch.equal(bits(y[rows, n:].contiguous()), bits(want))


@pytest.mark.parametrize("gather", [False, True])
def test_grouped(bi, ws, gather):
    """The last expert's weights lie past 4 GiB, so do the rows of q and of y."""
    E, N, K, R = 40, 2304, 48128, 1 << 20
    if gather:
        w = codes(E, N, K)                                     # 4.4 GB
        q, s_a = codes(90000, K), scales(90000, K // 128)      # 4.3 GB
        s_w = scales(E, N // 128, K // 128)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        offsets[1:], offsets[E] = 300, 700                     # the first and the last expert
        src = torch.randint(0, 90000, (700,), device=DEV).int()
        src[650:] = torch.arange(89950, 90000, device=DEV).int()
        y = torch.empty((700, N), dtype=torch.bfloat16, device=DEV)
        bi.bi_linear_f8_grouped(q, s_a, src, offsets, w, s_w, y, ws)
        for e, a, b in ((0, 0, 300), (E - 1, 300, 700)):
            want = torch.empty((b - a, N), dtype=torch.bfloat16, device=DEV)
            bi.bi_linear_f8(q[src[a:b].long()], s_a[src[a:b].long()], w[e], s_w[e], want, ws)
            assert torch.equal(bits(y[a:b]), bits(want)), e
        return
    w, s_w = codes(E, N, 16), scales(E, N // 128, 1)
    q, s_a = codes(R, 16), scales(R, 1)
    offsets = (torch.arange(E + 1, device=DEV) * R // E).int()
    y = torch.empty((R, N), dtype=torch.bfloat16, device=DEV)  # 4.8 GB
    bi.bi_linear_f8_grouped(q, s_a, None, offsets, w, s_w, y, ws)
    for e in (0, E - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        want = torch.empty((b - a, N), dtype=torch.bfloat16, device=DEV)
        bi.bi_linear_f8(q[a:b], s_a[a:b], w[e], s_w[e], want, ws)
        assert torch.equal(bits(y[a:b]), bits(want)), e


@pytest.mark.parametrize("M, k, R, N", [(65535, 2, 1 << 21, 1040), (65535, 1, 9, 33000)])
def test_combine(bi, M, k, R, N):
    rows, pos = torch.randn((1 << 12, N), device=DEV).bfloat16(), torch.randint(0, R, (M, k), device=DEV).int()
    rows = rows.repeat(-(-R // len(rows)), 1)[:R].contiguous()
    rows[-1] = 3.0
    pos[-1, 0] = R - 1
    weights, y = torch.rand((M, k), device=DEV), torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    bi.bi_moe_combine(rows, pos, weights, None, y)
    at = picked(M)
    want = torch.empty((len(at), N), dtype=torch.bfloat16, device=DEV)
    bi.bi_moe_combine(rows[pos[at].long().flatten()], torch.arange(len(at) * k, device=DEV).int().view(-1, k), weights[at], None,
                      want)
    assert torch.equal(bits(y[at]), bits(want))


def test_results_off_16_bytes(bi, ws):
    """y on 2 bytes, with a width that would allow wide stores."""
    q, s_a, w, s_w = codes(40, 272), scales(40, 3), codes(264, 272), scales(3, 3)
    buf = torch.full((40 * 264 + 2,), 7.0, dtype=torch.bfloat16, device=DEV)
    want = torch.empty((40, 264), dtype=torch.bfloat16, device=DEV)
    bi.bi_linear_f8(q, s_a, w, s_w, want, ws)
    bi.bi_linear_f8(q, s_a, w, s_w, buf[1:-1].view(40, 264), ws)
    assert torch.equal(bits(buf[1:-1].view(40, 264)), bits(want)) and buf[0] == 7 and buf[-1] == 7
