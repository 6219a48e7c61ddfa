"""Plain numpy references of the decoder-step operators, written from their
definitions in include/bi.h: bit-exact fp32 mirrors where the definition fixes
every rounding, fp64 where it does not."""
import numpy as np

import gen

F = np.float32
GROUP = 64


def f32(b):
    return gen.bf16_bits_to_f32(np.ascontiguousarray(b))


def bf16_bits(x):
    """fp32 -> bf16 bits, round to nearest even (finite values)."""
    u = np.ascontiguousarray(x, dtype=F).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_round(x):
    return f32(bf16_bits(x))


# ---------------------------------------------------------------- norm

def rmsnorm_quantize(h, y, w, eps):
    """bf16 bits -> (h' bits, codes int8, s_a fp64)."""
    x = f32(h)
    if y is not None:
        x = bf16_round(x + f32(y))
    t = x * f32(w)                                     # exact in fp32
    a = np.abs(t).max(1)
    st = np.where(a == 0, F(1), a / F(127)).astype(F)
    q = np.clip(np.rint(t / st[:, None]), -127, 127).astype(np.int8)
    rms = np.sqrt((x.astype(np.float64) ** 2).mean(1) + eps)
    s = np.where(a == 0, 1.0, st.astype(np.float64) / rms)
    return bf16_bits(x), q, s


# ---------------------------------------------------------------- 4-bit cache

def block_bytes(P, D):
    return P * (D + 8 * (D // GROUP))


def quantise(x):
    """fp32 holding bf16 values [..., D] -> codes uint8 [..., D], s and z bits [..., D / 64]."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.min(-1), g.max(-1)
    sb = bf16_bits((hi - lo) / F(15))
    s = f32(sb)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[..., None] > 0, (g - lo[..., None]) / s[..., None], F(0))
    return np.clip(np.rint(c), 0, 15).astype(np.uint8).reshape(x.shape), sb, bf16_bits(lo)


def k_place(D):
    """(byte, shift) of key element d within its position's codes."""
    d = np.arange(D)
    nib = d % 8 // 2 + 4 * (d % 2)
    return ((d % 64 // 16) * (D // 64) + d // 64) * 8 + d % 16 // 8 * 4 + nib // 2, 4 * (nib % 2)


def v_place(D):
    """(byte, shift) of value element d of an even position within its pair's codes (+ 2 bytes for the odd one)."""
    d = np.arange(D)
    return ((d % 64 // 8) * (D // 64) + d // 64) * 8 + d % 8 // 4 * 4 + d % 4 // 2, 4 * (d % 2)


def write_position(block, P, D, slot, k, v):
    """Quantises and stores one position's key and value (fp32 [D]) into a block (uint8 view)."""
    G = D // GROUP
    for which, (x, (byte, shift)) in enumerate(((k, k_place(D)), (v, v_place(D)))):
        code, s, z = quantise(x)
        base = slot * (D // 2) if which == 0 else P * (D // 2) + slot // 2 * D + slot % 2 * 2
        for d in range(D):
            b = base + byte[d]
            block[b] = (int(block[b]) & ~(15 << int(shift[d])) & 0xFF) | (int(code[d]) << int(shift[d]))
        p = P * D + slot * 8 * G + which * 4 * G
        block[p:p + 4 * G] = (s.astype(np.uint32) | (z.astype(np.uint32) << 16)).view(np.uint8)


def read_block(block, P, D):
    """Values held by a block: k, v fp64 [P, D]."""
    G = D // GROUP
    p = np.arange(P)[:, None]
    kb, ks = k_place(D)
    vb, vs = v_place(D)
    kc = (block[p * (D // 2) + kb] >> ks) & 15
    vc = (block[P * (D // 2) + p // 2 * D + p % 2 * 2 + vb] >> vs) & 15
    par = block[P * D:P * (D + 8 * G)].copy().view(np.uint32).reshape(P, 2, G)
    s = f32((par & 0xFFFF).astype(np.uint16)).astype(np.float64)
    z = f32((par >> 16).astype(np.uint16)).astype(np.float64)
    g = np.arange(D) // GROUP
    with np.errstate(invalid="ignore"):
        return z[:, 0, g] + s[:, 0, g] * kc, z[:, 1, g] + s[:, 1, g] * vc


def read_sequence(pool, P, D, pages, n):
    """Keys and values fp64 [n, Hkv, D] of a sequence, and which positions are on valid pages."""
    Hkv = pool.shape[1]
    k, v, ok = np.zeros((n, Hkv, D)), np.zeros((n, Hkv, D)), np.zeros(n, bool)
    for i in range((n + P - 1) // P):
        if i >= len(pages) or not 0 <= pages[i] < pool.shape[0]:
            continue
        m = min(P, n - i * P)
        ok[i * P:i * P + m] = True
        for h in range(Hkv):
            a, b = read_block(pool[pages[i], h], P, D)
            k[i * P:i * P + m, h], v[i * P:i * P + m, h] = a[:m], b[:m]
    return k, v, ok


# ---------------------------------------------------------------- rotation

def head_norm(x, w, eps):
    """fp32 [..., D], weight bits [D]: the definition's order, every operation rounded."""
    if w is None:
        return x
    D = x.shape[-1]
    q = x * x
    q = q[..., :D // 2] + q[..., D // 2:]
    q = q[..., 0::2] + q[..., 1::2]
    while q.shape[-1] > 1:
        q = q[..., :q.shape[-1] // 2] + q[..., q.shape[-1] // 2:]
    r = F(1) / np.sqrt(q / F(D) + F(eps))
    return (x * r) * f32(w)


def rotate(x, cs, rot, interleaved):
    """x [T, H, D] (fp32 or fp64), cs [T, rot / 2, 2]."""
    out = x.copy()
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    c, s = cs[:, None, :, 0].astype(x.dtype), cs[:, None, :, 1].astype(x.dtype)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


# ---------------------------------------------------------------- attention

def attention(q, k, v, ok, first, scale):
    """q fp64 [n, Hq, D] of positions first .. first + n - 1; k, v [S, Hkv, D].  Returns o, the mean of |v| under the
    same weights, and a bound of the scores' sums of magnitudes, all fp64."""
    n, Hq, D = q.shape
    S, Hkv = k.shape[:2]
    G = Hq // Hkv
    o, mag, big = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq, 1))
    for i in range(n):
        m = min(S, first + i + 1)
        if m <= 0 or not ok[:m].any():
            continue
        for h in range(Hq):
            kk, vv = k[:m, h // G][ok[:m]], v[:m, h // G][ok[:m]]
            s = kk @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h], mag[i, h] = p @ vv, p @ np.abs(vv)
            big[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return o, mag, big


# ---------------------------------------------------------------- logits

def logits_process(logits, V, ids=None, begin=None, mid=None, end=None, repetition=None, presence=None, frequency=None,
                   bias_ids=None, bias=None, mask=None):
    x = f32(logits)[:, :V].copy()
    M = x.shape[0]
    best = np.full(M, -1, np.int32)
    for m in range(M):
        if ids is not None:
            held = {int(t) for t in ids[begin[m]:end[m]] if 0 <= t < V}
            count = {}
            for t in ids[max(mid[m], begin[m]):end[m]]:
                if 0 <= t < V:
                    count[int(t)] = count.get(int(t), 0) + 1
            rep = F(1) if repetition is None else repetition[m]
            for t in held:
                x[m, t] = x[m, t] / rep if x[m, t] > 0 else x[m, t] * rep
            for t, c in count.items():
                fr = F(0) if frequency is None else frequency[m]
                pr = F(0) if presence is None else presence[m]
                x[m, t] = F(F(x[m, t]) - F(fr * F(c))) - pr
        if bias_ids is not None:
            last = {int(t): b for t, b in zip(bias_ids[m], bias[m]) if 0 <= t < V}
            for t, b in last.items():
                x[m, t] = F(x[m, t]) + F(b)
        if mask is not None:
            v = np.arange(V)
            x[m, ((mask[m].view(np.uint32)[v >> 5] >> (v & 31).astype(np.uint32)) & 1) == 0] = -np.inf
        y = np.where(np.isnan(x[m]), -np.inf, x[m])
        if y.max() > -np.inf:
            best[m] = int(np.argmax(y))
    return x, best
