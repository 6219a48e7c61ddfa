"""Plain references of the e4m3 linears and the mixture of experts, in NumPy: quantisers and routing bit for bit as
include/bi.h defines them, products and sums in fp64."""
import numpy as np

BLOCK = 128
TOP = np.float32(448)


def _table():
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


VALUES = _table()                                # fp64 value of each code
_POS = VALUES[:127]                              # increasing; code = index


def decode(codes):
    return VALUES[codes]


def encode(x):
    """fp32 -> codes: round to nearest even, 448 at most, NaN -> 0x7F (with the sign that the value has)."""
    x = np.asarray(x, np.float32)
    a = np.minimum(np.abs(x.astype(np.float64)), 448.0)
    nan = np.isnan(x)
    a = np.where(nan, 0, a)
    hi = np.searchsorted(_POS, a)                # the first code with at least this value
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(nan, 127, c).astype(np.uint8)
    return c | (np.signbit(x) & ~nan).astype(np.uint8) << 7


def blocks(n):
    return -(-n // BLOCK)


def _scale(amax):
    with np.errstate(invalid="ignore"):
        s = (amax / TOP).astype(np.float32)
    return np.where(s == 0, np.float32(1), s)


def _amax(x, axis):
    with np.errstate(invalid="ignore"):
        return np.abs(x).max(axis)               # NaN wins, as in the kernel


def quantize(x):
    """fp32 [M, K] -> codes uint8 [M, K], scales fp32 [M, blocks]."""
    M, K = x.shape
    codes, scales = np.empty((M, K), np.uint8), np.empty((M, blocks(K)), np.float32)
    for b in range(blocks(K)):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        s = _scale(_amax(v, 1))
        scales[:, b] = s
        with np.errstate(invalid="ignore", over="ignore"):
            codes[:, b * BLOCK:(b + 1) * BLOCK] = encode(v / s[:, None])
    return codes, scales


def quantize_weight(w):
    N, K = w.shape
    codes, scales = np.empty((N, K), np.uint8), np.empty((blocks(N), blocks(K)), np.float32)
    for i in range(blocks(N)):
        for b in range(blocks(K)):
            at = np.s_[i * BLOCK:(i + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK]
            scales[i, b] = _scale(_amax(w[at], None))
            codes[at] = encode(w[at] / scales[i, b])
    return codes, scales


def linear(q, s_a, w, s_w):
    """(y, sum of magnitudes), fp64 [M, N], from codes and scales."""
    a = decode(q) * np.repeat(s_a.astype(np.float64), BLOCK, 1)[:, :q.shape[1]]
    b = decode(w) * np.repeat(np.repeat(s_w.astype(np.float64), BLOCK, 0)[:w.shape[0]], BLOCK, 1)[:, :w.shape[1]]
    return a @ b.T, np.abs(a) @ np.abs(b).T


def linear_bound(y, mag, K):
    """How far a result may be from fp64.  The tensor cores' sum of a block: four slices of 32 products and the sum so far,
    each of the 33 held to fp32's 2^-24 of the largest, whose magnitude is at most the magnitudes' sum: 132 2^-24 < 2^-16.
    RN(s_a s_w) and the fma of each block: 2^-24 each, over at most blocks + 1 of them.  The result: half a step of bf16."""
    return np.abs(y) * 2.0 ** -8 + mag * (2.0 ** -16 + (blocks(K) + 2) * 2.0 ** -24) + 2.0 ** -130


def route(x, k):
    """Selection and order: ids [M, k], offsets [E + 1], src [M k], pos [M, k] of fp32 logits."""
    M, E = x.shape
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.float32(3.4028234663852886e38)))
    x = np.where(x == 0, np.float32(0), x)
    order = np.argsort(-x, 1, kind="stable")[:, :k]
    ids = np.where(np.take_along_axis(x, order, 1) > -np.inf, order, -1).astype(np.int32)
    flat = ids.ravel()
    rows = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    counts = np.bincount(flat[flat >= 0], minlength=E)
    offsets = np.concatenate(([0], counts.cumsum())).astype(np.int32)
    n = offsets[-1]
    src, pos = np.full(M * k, -1, np.int32), np.full(M * k, -1, np.int32)
    src[:n] = rows[:n] // k
    pos[rows[:n]] = np.arange(n)
    return ids, offsets, src, pos.reshape(M, k)


def route_weights(x, ids, softmax, renorm, scale):
    x = np.minimum(np.where(np.isnan(x), -np.inf, x), np.float32(3.4028234663852886e38)).astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if softmax:
            m = x.max(1, keepdims=True)
            p = np.where(x > -np.inf, np.exp(x - np.where(m > -np.inf, m, 0)), 0)
            whole = p.sum(1, keepdims=True)
        elif not renorm:
            p, whole = 1 / (1 + np.exp(-x)), np.ones((len(x), 1))
        else:                                    # quotients of sigmoids that fp64 does not hold either, by their logarithms
            log = -np.logaddexp(0, -x)
            taken = np.where(ids >= 0, np.take_along_axis(log, np.maximum(ids, 0), 1), -np.inf)
            m = taken.max(1, keepdims=True)
            p = np.where(x > -np.inf, np.exp(log - np.where(m > -np.inf, m, 0)), 0)
    w = np.where(ids >= 0, np.take_along_axis(p, np.maximum(ids, 0), 1), 0)
    if renorm:
        whole = w.sum(1, keepdims=True)
    return w / np.where(whole > 0, whole, 1) * scale
