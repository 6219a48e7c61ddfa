"""The e4m3 linears and the mixture of experts on the GPU against their plain references: bit for bit where the
definition fixes every rounding (codes, scales, selection, order of rows), within derived tolerances of fp64 elsewhere;
a row's bits whatever shares its call; other streams, captured graphs, bad routing tables."""
import numpy as np
import pytest
import torch

from tests import f8_ref as ref
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def bf16(x):
    """fp32 array -> (device bf16 tensor, the fp32 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16()
    return t.to(DEV), t.float().numpy()


def same_codes(got, want):
    got = got.cpu().numpy()
    bad = (got != want) & ~(((got & 127) == 127) & ((want & 127) == 127))     # any NaN is a NaN
    assert not bad.any(), "%d codes differ, first at %s" % (bad.sum(), np.argwhere(bad)[:3].tolist())


def same_floats(got, want):
    np.testing.assert_array_equal(got.cpu().numpy(), want)


def empty_codes(M, K):
    return torch.empty((M, K), dtype=torch.uint8, device=DEV), torch.empty((M, ref.blocks(K)), device=DEV)


# ------------------------------------------------------------------ quantisers

@pytest.mark.parametrize("M, K, ld", [(1, 16, 16), (1, 4096, 4096), (3, 272, 288), (17, 1040, 1040), (700, 512, 520),
                                      (5, 12288, 12288), (3000, 1152, 1152)])
def test_quantize(bi, M, K, ld):
    rng = np.random.default_rng(M + K)
    xd, x = bf16(rng.normal(size=(M, ld)) * np.exp(rng.normal(size=(M, 1)) * 4))
    q, s = empty_codes(M, K)
    bi.bi_quantize_act_f8(xd, q, s)
    codes, scales = ref.quantize(x[:, :K])
    same_floats(s, scales)
    same_codes(q, codes)


def test_quantize_borders(bi):
    """Zeros, the smallest and largest values, infinities and NaN: a block that is not finite has codes of NaN where it
    matters and spoils no other."""
    x = np.zeros((9, 400), np.float32)
    x[1] = 1e-40
    x[2, 5] = 9.2e-41                                # the smallest bf16 value
    x[3] = 3.3e38
    x[4, 130] = np.inf
    x[5, 130] = -np.inf
    x[6, 399] = np.nan
    x[7] = np.linspace(-448, 448, 400)               # ties between codes
    x[8, :128] = np.repeat(ref.VALUES[:127], 2)[:128]
    xd, x = bf16(x)
    q, s = empty_codes(9, 400)
    bi.bi_quantize_act_f8(xd, q, s)
    codes, scales = ref.quantize(x)
    same_floats(s, scales)
    same_codes(q, codes)
    assert (s.cpu().numpy()[0] == 1).all() and not q.cpu().numpy()[0].any()


@pytest.mark.parametrize("M, K, ld", [(1, 16, 32), (3, 272, 560), (400, 1408, 2816), (3000, 400, 800)])
def test_gated_relu(bi, M, K, ld):
    rng = np.random.default_rng(M + K)
    xd, x = bf16(rng.normal(size=(M, ld)) * 3)
    q, s = empty_codes(M, K)
    bi.bi_gated_quantize_f8(xd, bi.BI_GATE_RELU, q, s)
    g, u = x[:, :K], x[:, K:2 * K]
    codes, scales = ref.quantize(np.where(g > 0, g, np.float32(0)) * u)
    same_floats(s, scales)
    same_codes(q, codes)


@pytest.mark.parametrize("M, K", [(1, 16), (5, 272), (900, 1408)])
def test_gated_silu(bi, M, K):
    """Against fp64: the product is off by (|g| + 8) 2^-23, the quotient and the scale by 2^-24 each, and a code by half a step
    (2^-4 of the value, 2^-10 below the smallest normal one)."""
    rng = np.random.default_rng(M + K)
    x = rng.normal(size=(M, 2 * K)) * 6
    x[0, :16] = np.linspace(-95, 95, 16)
    xd, x = bf16(x)
    q, s = empty_codes(M, K)
    bi.bi_gated_quantize_f8(xd, bi.BI_GATE_SILU, q, s)
    g, u = x[:, :K].astype(np.float64), x[:, K:].astype(np.float64)
    t = g / (1 + np.exp(-g)) * u
    off = (np.abs(g) + 8) * 2.0 ** -23
    got_s = s.cpu().numpy().astype(np.float64)
    for b in range(ref.blocks(K)):
        at = np.s_[:, b * 128:(b + 1) * 128]
        amax = np.abs(t[at]).max(1)
        want = np.where(amax > 0, amax / 448, 1)
        assert (np.abs(got_s[:, b] - want) <= want * (off[at].max(1) + 2.0 ** -23)).all()
        v = ref.decode(q.cpu().numpy())[at]
        exact = np.clip(t[at] / got_s[:, b:b + 1], -448, 448)
        assert (np.abs(v - exact) <= np.abs(exact) * (2.0 ** -4 + off[at] + 2.0 ** -22) + 2.0 ** -10).all()


@pytest.mark.parametrize("u_top", [1.0, 1e5, 1e38])
@pytest.mark.parametrize("g_lo, g_hi", [(-95, -85), (-84, -76), (-131, -95)])
def test_gated_silu_of_low_gates(bi, g_lo, g_hi, u_top):
    """Blocks whose gates are all so low that exp(-g), its reciprocal or the product leaves fp32's normal range.  The bounds
    of test_gated_silu, and half a subnormal step (2^-150) for each product, scale and quotient that is one."""
    rng = np.random.default_rng(-g_lo)
    K = 400
    x = np.concatenate((rng.uniform(g_lo, g_hi, (6, K)), rng.uniform(-1, 1, (6, K)) * u_top), 1)
    xd, x = bf16(x)
    q, s = empty_codes(6, K)
    bi.bi_gated_quantize_f8(xd, bi.BI_GATE_SILU, q, s)
    g, u = x[:, :K].astype(np.float64), x[:, K:].astype(np.float64)
    t = g / (1 + np.exp(-g)) * u
    off = (np.abs(g) + 8) * 2.0 ** -23
    got_s, got = s.cpu().numpy().astype(np.float64), ref.decode(q.cpu().numpy())
    for b in range(ref.blocks(K)):
        at = np.s_[:, b * 128:(b + 1) * 128]
        amax = np.abs(t[at]).max(1)
        want = amax / 448
        # where the largest product rounds to at least one subnormal step a scale has, else the scale is 1
        seen = amax / 448 > 2.0 ** -149
        assert (np.abs(got_s[:, b] - want) <= want * (off[at].max(1) + 2.0 ** -23) + 2.0 ** -149)[seen].all()
        assert (got_s[amax / 448 < 2.0 ** -151, b] == 1).all()
        exact = np.clip(t[at] / got_s[:, b:b + 1], -448, 448)
        bound = np.abs(exact) * (2.0 ** -4 + off[at] + 2.0 ** -22) + 2.0 ** -10 + 2.0 ** -149 / got_s[:, b:b + 1]
        assert (np.abs(got[at] - exact) <= bound)[seen].all()


def test_gated_silu_of_gates_below_all(bi):
    """Gates whose silu no fp32 product can see: zeros with a scale of 1."""
    x = np.concatenate((np.linspace(-3e38, -300, 256).reshape(2, 128), np.full((2, 128), 3e38)), 1)
    xd, _ = bf16(x)
    q, s = empty_codes(2, 128)
    bi.bi_gated_quantize_f8(xd, bi.BI_GATE_SILU, q, s)
    assert (s == 1).all() and not (q & 127).any()


@pytest.mark.parametrize("M, K", [(3, 1040), (3000, 1408)])
def test_low_gates_change_no_other_block(bi, M, K):
    """A gate below -80 sends its warp over all its blocks again: those without one keep their bits, in short calls and in
    those that read two blocks ahead."""
    rng = np.random.default_rng(M)
    x = rng.normal(size=(M, 2 * K)).astype(np.float32) * 5
    low = x.copy()
    block = rng.integers(0, K // 128, M)
    low[np.arange(M), block * 128 + rng.integers(0, 128, M)] = rng.uniform(-300, -81, M)
    low[M // 2:, :K] = x[M // 2:, :K]                # rows without any
    (q, s), (q2, s2) = empty_codes(M, K), empty_codes(M, K)
    bi.bi_gated_quantize_f8(bf16(x)[0], bi.BI_GATE_SILU, q, s)
    bi.bi_gated_quantize_f8(bf16(low)[0], bi.BI_GATE_SILU, q2, s2)
    same = np.ones((M, ref.blocks(K)), bool)
    same[np.arange(M // 2), block[:M // 2]] = False
    assert (s.cpu().numpy() == s2.cpu().numpy())[same].all()
    codes = (q.cpu().numpy() == q2.cpu().numpy())
    assert codes[np.repeat(same, 128, 1)[:, :K]].all()


@pytest.mark.parametrize("N, K, ld", [(1, 16, 16), (127, 128, 128), (300, 400, 404), (1024, 1040, 1040)])
def test_quantize_weight(bi, N, K, ld):
    rng = np.random.default_rng(N + K)
    w = (rng.normal(size=(N, ld)) * np.exp(rng.normal(size=(N, 1)))).astype(np.float32)
    w[0, :8] = 0
    q = torch.empty((N, K), dtype=torch.uint8, device=DEV)
    s = torch.empty((ref.blocks(N), ref.blocks(K)), device=DEV)
    bi.bi_quantize_weight_f8(dev(w), q, s)
    codes, scales = ref.quantize_weight(w[:, :K])
    same_floats(s, scales)
    same_codes(q, codes)


# ------------------------------------------------------------------ linears

def operand(rng, rows, K):
    """Random codes with scales that differ from block to block."""
    return rng.choice(np.r_[0:127, 128:255].astype(np.uint8), (rows, K)), \
        np.exp(rng.normal(size=(rows, ref.blocks(K)))).astype(np.float32)


def weight(rng, N, K, E=None):
    shape = (E or 1, N, K)
    w = rng.choice(np.r_[0:127, 128:255].astype(np.uint8), shape)
    s = np.exp(rng.normal(size=(E or 1, ref.blocks(N), ref.blocks(K)))).astype(np.float32) * K ** -0.5
    return (w, s) if E else (w[0], s[0])


def near(y, want, K):
    v, mag = want
    off = np.abs(y.float().cpu().numpy().astype(np.float64) - v)
    bound = ref.linear_bound(v, mag, K)
    assert (off <= bound).all(), "off by up to %.2f of the bound" % (off / bound).max()


SHAPES = [(1, 16, 16), (1, 4096, 200), (5, 272, 1), (8, 128, 24576), (16, 144, 1001), (17, 1024, 300), (32, 400, 129),
          (33, 5136, 72), (64, 1040, 640), (100, 272, 2050), (129, 256, 1000), (200, 128, 8192), (777, 528, 3300),
          (2048, 272, 1160), (3, 12288, 40)]


@pytest.mark.parametrize("M, K, N", SHAPES)
def test_linear(bi, ws, M, K, N):
    rng = np.random.default_rng(M + K + N)
    (q, s_a), (w, s_w) = operand(rng, M, K), weight(rng, N, K)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    bi.bi_linear_f8(dev(q), dev(s_a), dev(w), dev(s_w), y, ws)
    near(y, ref.linear(q, s_a, w, s_w), K)


@pytest.mark.parametrize("K, N", [(1040, 12300), (4096, 1000), (144, 20000)])
def test_rows_have_the_same_bits_in_every_call(bi, ws, K, N):
    """Token tiles of every width, on the weight stream and on the tensor cores, and rows at other places."""
    rng = np.random.default_rng(N)
    (q, s_a), (w, s_w) = operand(rng, 2100, K), weight(rng, N, K)
    q, s_a, w, s_w = dev(q), dev(s_a), dev(w), dev(s_w)

    def rows(a, b):
        y = torch.empty((b - a, N), dtype=torch.bfloat16, device=DEV)
        bi.bi_linear_f8(q[a:b].contiguous(), s_a[a:b].contiguous(), w, s_w, y, ws)
        return y.view(torch.int16)
    whole = rows(0, 2100)
    for a, b in ((0, 1), (2099, 2100), (3, 8), (0, 16), (5, 22), (100, 140), (7, 71), (0, 100), (1000, 1129), (0, 300), (11, 788),
                 (600, 2100)):
        assert torch.equal(rows(a, b), whole[a:b]), (a, b)


def test_nan_stays_with_its_row(bi, ws):
    rng = np.random.default_rng(1)
    (q, s_a), (w, s_w) = operand(rng, 40, 400), weight(rng, 300, 400)
    clean = torch.empty((40, 300), dtype=torch.bfloat16, device=DEV)
    bi.bi_linear_f8(dev(q), dev(s_a), dev(w), dev(s_w), clean, ws)
    q[7, 390] = 127
    s_a[20, 1] = np.inf
    y = torch.empty_like(clean)
    bi.bi_linear_f8(dev(q), dev(s_a), dev(w), dev(s_w), y, ws)
    assert y[7].isnan().all() and not y[20].isfinite().any()
    keep = [m for m in range(40) if m not in (7, 20)]
    assert torch.equal(y[keep].view(torch.int16), clean[keep].view(torch.int16))


def grouped(bi, ws, q, s_a, src, offsets, w, s_w, R, fill=7.0, **o):
    y = torch.full((R, w.shape[1]), fill, dtype=torch.bfloat16, device=DEV)
    bi.bi_linear_f8_grouped(dev(q), dev(s_a), None if src is None else dev(src), dev(np.asarray(offsets, np.int32)), dev(w), dev(s_w),
                            y, ws, **o)
    return y


CALLS = [([0, 1], 1, 16, 16), ([0, 0, 3, 3, 5], 5, 272, 130), ([2, 2, 9, 40, 41, 41], 64, 400, 1001),
         ([0, 100, 100, 300, 310], 320, 1040, 300), ([0, 700, 701, 1900], 2000, 528, 1160), ([0, 300, 800, 1400, 2500], 2500, 272, 4100),
         ([0] + [17 * i for i in range(1, 41)], 680, 144, 200)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("offsets, R, K, N", CALLS)
def test_grouped(bi, ws, offsets, R, K, N, gather):
    """Each expert's rows are the linear's, bit for bit; rows of no expert are left as they were."""
    rng = np.random.default_rng(R + K)
    E = len(offsets) - 1
    w, s_w = weight(rng, N, K, E)
    n = 90 if gather else R
    q, s_a = operand(rng, n, K)
    src = rng.integers(0, n, R).astype(np.int32) if gather else None
    y = grouped(bi, ws, q, s_a, src, offsets, w, s_w, R)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        row = src[a:b] if gather else np.arange(a, b)
        one = torch.empty((b - a, N), dtype=torch.bfloat16, device=DEV)
        bi.bi_linear_f8(dev(q[row]), dev(s_a[row]), dev(w[e]), dev(s_w[e]), one, ws)
        assert torch.equal(one.view(torch.int16), y[a:b].view(torch.int16)), e
        near(one, ref.linear(q[row], s_a[row], w[e], s_w[e]), K)
    assert (y[:offsets[0]] == 7).all() and (y[offsets[-1]:] == 7).all()


@pytest.mark.parametrize("R", [12, 900])
def test_grouped_tables_out_of_range(bi, ws, R):
    """src that names no row gives zeros, even beside NaN; offsets out of order or range leave experts empty."""
    rng = np.random.default_rng(R)
    w, s_w = weight(rng, 520, 272, 3)
    q, s_a = operand(rng, 20, 272)
    q[0, 3] = 127
    src = rng.integers(1, 20, R).astype(np.int32)
    bad = np.arange(R) % 4 == 1
    src[bad] = np.resize([-1, 20, 2 ** 31 - 1, -2 ** 31], bad.sum())
    y = grouped(bi, ws, q, s_a, src, [0, R // 3, R, R], w, s_w, R)
    assert (y[torch.from_numpy(bad)] == 0).all()
    good = grouped(bi, ws, q, s_a, np.where(bad, 1, src).astype(np.int32), [0, R // 3, R, R], w, s_w, R)
    assert torch.equal(y[torch.from_numpy(~bad)].view(torch.int16), good[torch.from_numpy(~bad)].view(torch.int16))
    a = R // 2
    for offsets, means in (([-5, a, a - 3, 2 * R], [0, a, a, R]), ([R + 9, -1, 5, R], [R, R, R, R])):
        assert torch.equal(grouped(bi, ws, q, s_a, src, offsets, w, s_w, R).view(torch.int16),
                           grouped(bi, ws, q, s_a, src, means, w, s_w, R).view(torch.int16))


def test_grouped_many_experts_and_no_rows(bi, ws):
    rng = np.random.default_rng(5)
    w, s_w = weight(rng, 16, 16, 1024)
    q, s_a = operand(rng, 3, 16)
    offsets = np.zeros(1025, np.int32)
    assert (grouped(bi, ws, q, s_a, None, offsets, w, s_w, 3) == 7).all()
    offsets[600:], offsets[1024:] = 2, 3
    y = grouped(bi, ws, q, s_a, None, offsets, w, s_w, 3)
    for r, e in ((0, 599), (1, 599), (2, 1023)):
        near(y[r:r + 1], ref.linear(q[r:r + 1], s_a[r:r + 1], w[e], s_w[e]), 16)


# ------------------------------------------------------------------ routing

def run_route(bi, x, k, score, renorm, scale=1.0, half=False, **o):
    M, E = x.shape
    xd = bf16(x)[0] if half else dev(x)

    def ints(*shape):
        return torch.full(shape, -9, dtype=torch.int32, device=DEV)
    out = ints(M, k), torch.full((M, k), -9.0, device=DEV), ints(E + 1), ints(M * k), ints(M, k)
    bi.bi_moe_route(xd, score, renorm, scale, *out, bi.new_moe_route_workspace(M, E), **o)
    return out


def check_route(bi, x, k, softmax, renorm, scale=1.0, half=False):
    if half:
        x = bf16(x)[1]
    out = run_route(bi, x, k, bi.BI_ROUTE_SOFTMAX if softmax else bi.BI_ROUTE_SIGMOID, renorm, scale, half)
    ids, weights, offsets, src, pos = (t.cpu().numpy() for t in out)
    for got, want in zip((ids, offsets, src, pos), ref.route(x, k)):
        np.testing.assert_array_equal(got, want)
    # expf: 2 ulp; the sum of up to E of them, the quotient and the factor: 2^-24 each and E / 32 + 6 additions
    want = ref.route_weights(x, ids, softmax, renorm, scale)
    bound = np.abs(want) * (x.shape[1] / 32 + 16) * 2.0 ** -23 + abs(scale) * 2.0 ** -126
    assert (np.abs(weights - want) <= bound).all()


@pytest.mark.parametrize("M, E, k", [(1, 1, 1), (1, 8, 2), (5, 64, 6), (64, 33, 4), (65, 128, 8), (300, 7, 7), (1000, 256, 8), (40, 1024, 32),
                                     (2500, 1000, 3), (11000, 48, 4)])
@pytest.mark.parametrize("softmax, renorm, half", [(True, True, False), (True, False, True), (False, True, True), (False, False, False)])
def test_route(bi, M, E, k, softmax, renorm, half):
    rng = np.random.default_rng(M + E)
    x = (rng.normal(size=(M, E)) * 2).astype(np.float32)
    x[rng.random(M) < 0.2] = -np.inf                             # padding
    x[rng.random((M, E)) < 0.1] = -np.inf                        # experts that are not allowed
    check_route(bi, x, k, softmax, renorm, 1.0 if renorm else 2.5, half)


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_borders(bi, softmax, renorm):
    """Ties, both zeros, masks of the lowest value, infinities, NaN, values whose exponentials leave fp32."""
    low = np.finfo(np.float32).min
    x = np.zeros((10, 40), np.float32)
    x[1, ::2] = -0.0
    x[2] = low
    x[3] = np.where(np.arange(40) % 3 == 0, low, 1)
    x[4] = -np.inf
    x[5, 7], x[5, 20:] = np.inf, -np.inf
    x[6, 3::5] = np.nan
    x[7] = np.nan
    x[8] = np.linspace(-300, 300, 40)
    x[9] = -120
    check_route(bi, x, 6, softmax, renorm)


def test_route_of_the_longest_calls(bi):
    """Chunks whose masks take more than 48 KB of shared memory."""
    M, E = 65535, 1024
    x = torch.rand((M, E), device=DEV)
    x[::7] = -float("inf")
    x.scatter_(1, torch.randint(0, E, (M, 1), device=DEV), 2.0)
    want = x.argmax(1).int()
    ints = [torch.empty(s, dtype=torch.int32, device=DEV) for s in ((M, 1), (E + 1,), (M,), (M, 1))]
    w = torch.empty((M, 1), device=DEV)
    bi.bi_moe_route(x, bi.BI_ROUTE_SOFTMAX, True, 1.0, ints[0], w, *ints[1:], bi.new_moe_route_workspace(M, E))
    assert torch.equal(ints[0][:, 0], want) and (w == 1).all()
    assert torch.equal(ints[2].long(), torch.sort(want, stable=True).indices)
    assert torch.equal(ints[1].long(), torch.cat((torch.zeros(1, device=DEV), torch.bincount(want, minlength=E).cumsum(0))).long())
    assert torch.equal(ints[2][ints[3][:, 0].long()].long(), torch.arange(M, device=DEV))


def test_route_rows_of_any_stride(bi):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(70, 30)).astype(np.float32)
    want = run_route(bi, np.ascontiguousarray(x[:, 3:20]), 3, bi.BI_ROUTE_SOFTMAX, True)
    big = dev(x)
    out = [torch.empty_like(t) for t in want]
    bi.bi_moe_route(big[:, 3:20], bi.BI_ROUTE_SOFTMAX, True, 1.0, *out, bi.new_moe_route_workspace(70, 17))
    for a, b in zip(out, want):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ weighted sum

@pytest.mark.parametrize("M, k, N, R", [(1, 1, 1, 1), (3, 2, 1001, 6), (5, 8, 64, 40), (17, 11, 4096, 100), (300, 4, 520, 1200)])
@pytest.mark.parametrize("base", [False, True, "in place"])
def test_combine(bi, M, k, N, R, base):
    """fp64 of the same fmas: each rounded to 2^-24, the result to half a step of bf16."""
    rng = np.random.default_rng(M + N)
    rd, rows = bf16(rng.normal(size=(R, N)))
    bd, b = bf16(rng.normal(size=(M, N)))
    pos = rng.integers(0, R, (M, k)).astype(np.int32)
    w = rng.normal(size=(M, k)).astype(np.float32)
    absent = rng.random((M, k)) < 0.3
    pos[absent] = np.resize([-1, R, -2 ** 31, 2 ** 31 - 1], absent.sum())
    w[absent] = np.resize([np.nan, np.inf, 1], absent.sum())     # left out whatever its weight
    y = bd if base == "in place" else torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    bi.bi_moe_combine(rd, dev(pos), dev(w), bd if base else None, y)
    t = np.where(absent, 0, w)[..., None].astype(np.float64) * rows.astype(np.float64)[np.where(absent, 0, pos)]
    want = t.sum(1) + (b if base else 0)
    bound = np.abs(want) * 2.0 ** -8 + (np.abs(t).sum(1) + np.abs(b)) * (k + 1) * 2.0 ** -24 + 2.0 ** -133
    assert (np.abs(y.float().cpu().numpy() - want) <= bound).all()


def test_combine_rows_off_16_bytes(bi):
    rng = np.random.default_rng(0)
    buf = torch.from_numpy(rng.normal(size=1 + 6 * 64).astype(np.float32)).bfloat16().to(DEV)
    pos, w = dev(np.arange(6, dtype=np.int32).reshape(3, 2)), dev(rng.normal(size=(3, 2)).astype(np.float32))
    a, b = (torch.empty((3, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    bi.bi_moe_combine(buf[1:].view(6, 64), pos, w, None, a)
    bi.bi_moe_combine(buf[1:].clone().view(6, 64), pos, w, None, b)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# ------------------------------------------------------------------ together

class Experts:
    """A layer of experts and its buffers for up to M tokens."""

    def __init__(self, bi, M, H, I, E, k, seed=0):
        rng = np.random.default_rng(seed)
        self.bi, self.k, self.E, self.H, self.I = bi, k, E, H, I
        self.up, self.down = weight(rng, 2 * I, H, E), weight(rng, H, I, E)
        self.w = [dev(a) for a in self.up + self.down]
        self.router = rng.normal(size=(E, H)).astype(np.float32) * H ** -0.5
        self.ws, self.route_ws = bi.new_f8_workspace(), bi.new_moe_route_workspace(M, E)

        def ints(*shape):
            return torch.empty(shape, dtype=torch.int32, device=DEV)
        self.q, self.m = empty_codes(M, H), empty_codes(M * k, I)
        self.ids, self.weights, self.offsets, self.src, self.pos = (ints(M, k), torch.empty((M, k), device=DEV), ints(E + 1),
                                                                    ints(M * k), ints(M, k))
        self.gu = torch.zeros((M * k, 2 * I), dtype=torch.bfloat16, device=DEV)
        self.rows = torch.zeros((M * k, H), dtype=torch.bfloat16, device=DEV)

    def __call__(self, x, logits, y, **o):
        bi, M = self.bi, x.shape[0]
        n = M * self.k
        q, m = [t[:M] for t in self.q], [t[:n] for t in self.m]
        bi.bi_moe_route(logits, bi.BI_ROUTE_SOFTMAX, True, 1.0, self.ids[:M], self.weights[:M], self.offsets, self.src[:n], self.pos[:M],
                        self.route_ws, **o)
        bi.bi_quantize_act_f8(x, *q, **o)
        bi.bi_linear_f8_grouped(*q, self.src[:n], self.offsets, self.w[0], self.w[1], self.gu[:n], self.ws, **o)
        bi.bi_gated_quantize_f8(self.gu[:n], bi.BI_GATE_SILU, *m, **o)
        bi.bi_linear_f8_grouped(*m, None, self.offsets, self.w[2], self.w[3], self.rows[:n], self.ws, **o)
        bi.bi_moe_combine(self.rows[:n], self.pos[:M], self.weights[:M], x, y, **o)
        return y


def layer_inputs(e, M, seed):
    rng = np.random.default_rng(seed)
    xd, x = bf16(rng.normal(size=(M, e.H)))
    return xd, dev((x @ e.router.T).astype(np.float32))


def test_a_layer_of_experts(bi):
    """Every step of the layer against its plain form on what the step was given."""
    e = Experts(bi, 50, 272, 400, 6, 2)
    x, logits = layer_inputs(e, 50, 1)
    y = e(x, logits, torch.empty_like(x))
    ids, offsets, src, pos = ref.route(logits.cpu().numpy(), 2)
    same_floats(e.ids, ids)
    same_floats(e.src, src)
    codes, scales = ref.quantize(x.float().cpu().numpy())
    same_codes(e.q[0], codes)
    m, s_m = (t.cpu().numpy() for t in e.m)
    for j in range(6):
        a, b = offsets[j], offsets[j + 1]
        near(e.gu[a:b], ref.linear(codes[src[a:b]], scales[src[a:b]], e.up[0][j], e.up[1][j]), 272)
        near(e.rows[a:b], ref.linear(m[a:b], s_m[a:b], e.down[0][j], e.down[1][j]), 400)
    rows, w = e.rows.float().cpu().numpy().astype(np.float64), e.weights.cpu().numpy().astype(np.float64)
    t = w[..., None] * rows[pos]
    want = x.float().cpu().numpy() + t.sum(1)
    bound = np.abs(want) * 2.0 ** -8 + (np.abs(t).sum(1) + np.abs(want)) * 2.0 ** -21
    assert (np.abs(y.float().cpu().numpy() - want) <= bound).all()


def test_a_layer_gives_a_token_the_same_bits_alone(bi):
    e = Experts(bi, 300, 400, 272, 9, 3)
    x, logits = layer_inputs(e, 300, 2)
    whole = e(x, logits, torch.empty_like(x)).clone()
    for a, b in ((0, 1), (299, 300), (3, 8), (10, 50), (0, 150)):
        y = e(x[a:b], logits[a:b], torch.empty((b - a, 400), dtype=torch.bfloat16, device=DEV))
        assert torch.equal(y.view(torch.int16), whole[a:b].view(torch.int16)), (a, b)


@pytest.mark.parametrize("flags", [0, 1])
def test_a_layer_captured_on_another_stream(bi, flags):
    """A captured layer is replayed on other inputs, whose routing differs; with and without programmatic launches."""
    e, plain = Experts(bi, 40, 272, 144, 5, 2), Experts(bi, 40, 272, 144, 5, 2)
    x, logits = layer_inputs(e, 40, 3)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e(x, logits, y, flags=flags)                 # kernels are loaded before the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            e(x, logits, y, flags=flags)
        for seed in (4, 5):
            x2, logits2 = layer_inputs(e, 40, seed)
            x.copy_(x2)
            logits.copy_(logits2)
            graph.replay()
            side.synchronize()
            want = plain(x2, logits2, torch.empty_like(x2))
            assert torch.equal(y.view(torch.int16), want.view(torch.int16))
    assert bi.bi_workspace_status(e.ws) == bi.BI_OK


def test_calls_at_once_share_a_workspace(bi, ws):
    """Two streams at a time, one workspace: it holds a status alone."""
    rng = np.random.default_rng(8)
    (q, s_a), (w, s_w) = operand(rng, 24, 2048), weight(rng, 5000, 2048)
    args = [dev(a) for a in (q, s_a, w, s_w)]
    want = torch.empty((24, 5000), dtype=torch.bfloat16, device=DEV)
    bi.bi_linear_f8(*args, want, ws)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(want) for _ in range(6)]
    for i, y in enumerate(outs):
        bi.bi_linear_f8(*args, y, ws, stream=streams[i % 2])
    torch.cuda.synchronize()
    for y in outs:
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))
