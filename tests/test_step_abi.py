"""Host-side checks of the decoder-step operators: sizes, and the refusals of
every argument rule, before anything is launched (fake pointers that are never
dereferenced), and the references' own layout."""
import ctypes

import numpy as np
import pytest
import torch

from tests import step_ref as ref

FAKE = 1 << 32          # 16-byte aligned, never dereferenced
FAR = 1 << 40           # overlaps no small buffer at FAKE


@pytest.fixture(scope="module")
def bi():
    import __graft_entry__
    __graft_entry__.build()
    import invariant_quantized_linear_gb300 as m
    return m


def test_block_bytes(bi):
    for P in (16, 32, 64, 128):
        for D in (64, 128):
            assert bi.bi_kv4_block_bytes(P, D) == ref.block_bytes(P, D)
    for P, D in ((0, 64), (24, 64), (8, 128), (256, 128), (16, 96), (16, 256), (-16, 64)):
        assert bi.bi_kv4_block_bytes(P, D) == 0


def norm(bi, **o):
    a = dict(h=FAKE, ldh=1024, y=2 * FAR, ldy=1024, w=3 * FAR, eps=1e-6, M=4, K=1024, h_out=FAKE, ldo=1024, q=4 * FAR,
             s=5 * FAR)
    a.update(o)
    return bi.lib.bi_rmsnorm_quantize(a["h"], a["ldh"], a["y"], a["ldy"], a["w"], a["eps"], a["M"], a["K"], a["h_out"],
                                      a["ldo"], a["q"], a["s"], 0, None)


def test_norm_refusals(bi):
    inv, ali = bi.BI_ERR_INVALID_ARG, bi.BI_ERR_ALIGNMENT
    for o in ({"h": None}, {"w": None}, {"q": None}, {"s": None}, {"y": None}, {"h_out": None}, {"M": 0}, {"M": 65536},
              {"ldh": 1016}, {"ldy": 512}, {"ldo": 8}, {"K": 1000}, {"K": 0}, {"eps": -1e-6}, {"eps": float("nan")},
              {"eps": float("inf")}, {"h_out": FAKE + 16}, {"ldo": 1032}, {"h_out": 2 * FAR}, {"q": FAKE},
              {"s": FAKE + 64}, {"q": 2 * FAR}, {"q": 3 * FAR}, {"s": 4 * FAR}):
        assert norm(bi, **o) == inv, o
    for o in ({"h": FAKE + 8, "h_out": FAKE + 8}, {"y": 2 * FAR + 2}, {"w": 3 * FAR + 4}, {"q": 4 * FAR + 8},
              {"s": 5 * FAR + 2}, {"ldh": 1028, "ldo": 1028}, {"ldy": 1030}):
        assert norm(bi, **o) == ali, o
    assert norm(bi, K=133152, ldh=133152, ldy=133152, ldo=133152) == bi.BI_ERR_INT32_BOUND


def cache(bi, **o):
    a = dict(pool=FAKE, page_stride=4 * ref.block_bytes(16, 128), num_pages=10, page_size=16, Hkv=4, D=128)
    a.update(o)
    return bi.bi_kv4_cache(*[a[f] for f, _ in bi.bi_kv4_cache._fields_])


def batch(bi, **o):
    a = dict(cu_q=FAKE, kv_len=FAKE, pages=FAKE, ld_pages=8, B=2, T=6, max_q=5, max_kv=100)
    a.update(o)
    return bi.bi_kv4_batch(*[a[f] for f, _ in bi.bi_kv4_batch._fields_])


BAD_CACHE = [({"pool": None}, 1), ({"num_pages": 0}, 1), ({"Hkv": 0}, 1), ({"Hkv": 1025}, 1), ({"page_size": 48}, 1),
             ({"page_size": 256}, 1), ({"D": 96}, 1), ({"D": 256}, 1), ({"page_stride": 4 * ref.block_bytes(16, 128) - 16}, 1),
             ({"pool": FAKE + 8}, 2), ({"page_stride": 4 * ref.block_bytes(16, 128) + 8}, 2)]
BAD_BATCH = [({"cu_q": None}, 1), ({"kv_len": None}, 1), ({"pages": None}, 1), ({"ld_pages": 0}, 1), ({"B": 0}, 1),
             ({"B": 65536}, 1), ({"T": 0}, 1), ({"T": (1 << 20) + 1}, 1), ({"max_q": 0}, 1), ({"max_q": 65536}, 1),
             ({"max_kv": 0}, 1), ({"max_kv": (1 << 22) + 1}, 1), ({"cu_q": FAKE + 2}, 2), ({"kv_len": FAKE + 1}, 2),
             ({"pages": FAKE + 3}, 2)]


def calls(bi):
    """The three entry points that take a cache and a batch."""
    L = bi.lib
    return {
        "append": lambda c, b, **o: (lambda a: L.bi_rope_append_kv4(
            a["q"], a["ldq"], a["Hq"], a["k"], a["ldk"], a["v"], a["ldv"], a["qn"], a["kn"], a["eps"], a["rope"], a["n_pos"],
            a["rot"], a["layout"], a["out"], c, b, 0, None))(
            {**dict(q=FAR, ldq=2048, Hq=8, k=FAR + 2048, ldk=2048, v=FAR + 2048 + 1024, ldv=2048, qn=None, kn=None, eps=1e-6,
                    rope=FAKE, n_pos=100, rot=64, layout=0, out=2 * FAR), **o}),
        "gather": lambda c, b, **o: (lambda a: L.bi_kv4_gather(c, b, a["k"], a["v"], None))(
            {**dict(k=FAR, v=2 * FAR), **o}),
        "attention": lambda c, b, **o: (lambda a: L.bi_attention_kv4(
            a["q"], a["ldq"], a["Hq"], c, b, a["scale"], a["o"], a["ws"], a["n"], 0, None))(
            {**dict(q=FAR, ldq=1024, Hq=8, scale=0.1, o=2 * FAR, ws=3 * FAR, n=1 << 40), **o}),
    }


@pytest.mark.parametrize("name", ["append", "gather", "attention"])
def test_cache_and_batch_refusals(bi, name):
    f = calls(bi)[name]
    for o, want in BAD_CACHE:
        assert f(cache(bi, **o), batch(bi)) == want, o
    for o, want in BAD_BATCH:
        assert f(cache(bi), batch(bi, **o)) == want, o
    assert f(None, batch(bi)) == bi.BI_ERR_INVALID_ARG
    assert f(cache(bi), None) == bi.BI_ERR_INVALID_ARG


def test_append_refusals(bi):
    f = calls(bi)["append"]
    for o in ({"q": None}, {"k": None}, {"v": None}, {"out": None}, {"rope": None}, {"Hq": 0}, {"Hq": 1025}, {"ldq": 1016},
              {"ldk": 504}, {"ldv": 0}, {"n_pos": 0}, {"rot": -4}, {"rot": 132}, {"rot": 6}, {"layout": 2}, {"eps": -1.0},
              {"out": FAR}, {"out": FAR + 4096}):
        assert f(cache(bi), batch(bi), **o) == bi.BI_ERR_INVALID_ARG, o
    for o in ({"q": FAR + 8}, {"k": FAR + 2050}, {"v": FAR + 4}, {"out": 2 * FAR + 2}, {"rope": FAKE + 4}, {"qn": FAKE + 2},
              {"kn": FAKE + 8}, {"ldq": 2052}, {"ldk": 2050}, {"ldv": 2049}):
        assert f(cache(bi), batch(bi), **o) == bi.BI_ERR_ALIGNMENT, o


def test_gather_refusals(bi):
    f = calls(bi)["gather"]
    assert f(cache(bi), batch(bi), k=None) == bi.BI_ERR_INVALID_ARG
    assert f(cache(bi), batch(bi), v=FAR) == bi.BI_ERR_INVALID_ARG
    assert f(cache(bi), batch(bi), v=FAR + 16) == bi.BI_ERR_INVALID_ARG
    assert f(cache(bi), batch(bi), k=FAR + 4) == bi.BI_ERR_ALIGNMENT


def test_attention_refusals(bi):
    f = calls(bi)["attention"]
    for o in ({"q": None}, {"o": None}, {"Hq": 0}, {"Hq": 6}, {"ldq": 1016}, {"scale": 0.0}, {"scale": -1.0},
              {"scale": float("nan")}, {"scale": float("inf")}, {"o": FAR + 16}):
        assert f(cache(bi), batch(bi), **o) == bi.BI_ERR_INVALID_ARG, o
    for o in ({"q": FAR + 8}, {"o": 2 * FAR + 8}, {"ldq": 1028}):
        assert f(cache(bi), batch(bi), **o) == bi.BI_ERR_ALIGNMENT, o
    need = bi.bi_attention_kv4_workspace_size(8, cache(bi), batch(bi))
    assert need > 0
    for o in ({"ws": None}, {"n": need - 1}, {"ws": 3 * FAR + 8}):
        assert f(cache(bi), batch(bi), **o) == bi.BI_ERR_WORKSPACE, o
    assert bi.bi_attention_kv4_workspace_size(6, cache(bi), batch(bi)) == 0
    assert bi.bi_attention_kv4_workspace_size(8, cache(bi, D=96), batch(bi)) == 0
    assert bi.bi_attention_kv4_workspace_size(8, cache(bi), batch(bi, T=0)) == 0


def test_attention_workspace_grows_with_the_call(bi):
    """One workspace of the largest size serves smaller calls: the size never falls when a bound grows."""
    size = lambda **o: bi.bi_attention_kv4_workspace_size(32, cache(bi, Hkv=8), batch(bi, **o))
    base = dict(B=4, T=16, max_q=4, max_kv=3000)
    for k, v in (("B", 9), ("T", 64), ("max_q", 16), ("max_kv", 100000)):
        assert size(**{**base, k: v}) >= size(**base)


def logits(bi, r=None, **o):
    a = dict(x=FAKE, ldl=1000, M=4, V=1000, out=FAR, ldo=1000, am=2 * FAR, ws=3 * FAR, n=1 << 20)
    a.update(o)
    rules = dict(ids=None, begin=None, mid=None, end=None, repetition=None, presence=None, frequency=None, bias_ids=None,
                 bias=None, n_bias=0, mask=None, ld_mask=0)
    rules.update(r or {})
    s = bi.bi_logits_rules(*[rules[f] for f, _ in bi.bi_logits_rules._fields_])
    return bi.lib.bi_logits_process(a["x"], a["ldl"], a["M"], a["V"], s, a["out"], a["ldo"], a["am"], a["ws"], a["n"], 0,
                                    None)


def test_logits_refusals(bi):
    for o in ({"x": None}, {"M": 0}, {"M": 65536}, {"V": 0}, {"V": (1 << 24) + 1, "ldl": 1 << 25, "ldo": 1 << 25},
              {"ldl": 999}, {"ldo": 999}, {"out": None, "am": None}, {"out": FAKE}):
        assert logits(bi, **o) == bi.BI_ERR_INVALID_ARG, o
    for r in ({"ids": FAKE}, {"ids": FAKE, "begin": FAKE, "mid": FAKE}, {"n_bias": -1}, {"n_bias": 65537}, {"n_bias": 3},
              {"n_bias": 3, "bias_ids": FAKE}, {"mask": FAKE, "ld_mask": 31}):
        assert logits(bi, r) == bi.BI_ERR_INVALID_ARG, r
    for o in ({"x": FAKE + 1}, {"out": FAR + 2}, {"am": 2 * FAR + 1}):
        assert logits(bi, **o) == bi.BI_ERR_ALIGNMENT, o
    for k in ("ids", "begin", "mid", "end", "repetition", "presence", "frequency", "mask", "bias", "bias_ids"):
        r = dict(ids=FAKE, begin=FAKE, mid=FAKE, end=FAKE, ld_mask=32)
        r[k] = FAKE + 2
        assert logits(bi, r) == bi.BI_ERR_ALIGNMENT, k
    for o in ({"ws": None}, {"ws": 3 * FAR + 4}, {"n": bi.bi_logits_workspace_size(4) - 1}):
        assert logits(bi, **o) == bi.BI_ERR_WORKSPACE, o
    assert bi.bi_logits_workspace_size(0) == 0 and bi.bi_logits_workspace_size(65536) == 0
    assert bi.lib.bi_logits_process(FAKE, 10, 1, 10, None, FAR, 10, None, FAR, 1 << 20, 0, None) == bi.BI_ERR_INVALID_ARG


def test_rope_table_refusals(bi):
    T = bi.lib.bi_rope_table
    for a in ((None, 4, 1.0, 4, FAKE), (FAKE, 0, 1.0, 4, FAKE), (FAKE, 4, float("nan"), 4, FAKE), (FAKE, 4, 1.0, 0, FAKE),
              (FAKE, 4, 1.0, (1 << 22) + 1, FAKE), (FAKE, 4, 1.0, 4, None)):
        assert T(*a, None) == bi.BI_ERR_INVALID_ARG
    assert T(FAKE + 4, 4, 1.0, 4, FAKE, None) == bi.BI_ERR_ALIGNMENT
    assert T(FAKE, 4, 1.0, 4, FAKE + 4, None) == bi.BI_ERR_ALIGNMENT


@pytest.mark.parametrize("P,D", [(16, 64), (32, 128)])
def test_reference_layout_round_trip(P, D):
    """Every element has a place of its own, and what is written is what is read, within half a step."""
    rng = np.random.default_rng(3)
    x = ref.bf16_round(rng.normal(size=(2, P, D)).astype(np.float32))
    block = np.full(ref.block_bytes(P, D), 0xA5, np.uint8)
    for slot in rng.permutation(P):
        ref.write_position(block, P, D, int(slot), x[0, slot], x[1, slot])
    k, v = ref.read_block(block, P, D)
    for got, want in ((k, x[0]), (v, x[1])):
        s = ref.f32(ref.quantise(want)[1]).astype(np.float64).repeat(ref.GROUP, -1)
        # half a step; the top code may fall short by the rounding of s (2^-8 of 15 steps)
        assert (np.abs(got - want) <= s * (0.5 + 15 * 2.0 ** -8 + 2.0 ** -16)).all()


def test_half_rotation_is_in_steps_of_eight(bi):
    f = calls(bi)["append"]
    for rot in (4, 12, 124):
        assert f(cache(bi), batch(bi), rot=rot, layout=bi.BI_ROPE_HALF) == bi.BI_ERR_INVALID_ARG, rot
    for rot in (2, 6, 14):
        assert f(cache(bi), batch(bi), rot=rot, layout=bi.BI_ROPE_INTERLEAVED) == bi.BI_ERR_INVALID_ARG, rot


def test_attention_workspace_has_a_status(bi):
    """Small calls' workspaces too are large enough for bi_workspace_status."""
    need = bi.bi_linear_workspace_size(1, 1, 16)
    assert bi.bi_attention_kv4_workspace_size(1, cache(bi, Hkv=1, D=64), batch(bi, B=1, T=1, max_q=1, max_kv=1)) >= need
    assert bi.bi_attention_kv4_workspace_size(8, cache(bi), batch(bi)) >= need


def test_mask_of_one_row_for_all_is_refused(bi):
    """A mask whose rows are one and the same (stride 0) is not read past its end."""
    words = torch.zeros((1, 32), dtype=torch.int32)
    assert bi.logits_rules(mask=words).ld_mask == 32
    r = bi.logits_rules(mask=words.expand(4, 32))
    assert bi.lib.bi_logits_process(FAKE, 1000, 4, 1000, r, FAR, 1000, 2 * FAR, 3 * FAR, 1 << 20, 0,
                                    None) == bi.BI_ERR_INVALID_ARG


def test_bindings_refuse_heads_that_are_not_side_by_side(bi):
    c, b = cache(bi), batch(bi)
    q = torch.zeros((6, 8, 128), dtype=torch.bfloat16)
    for bad in (q.transpose(0, 1).contiguous().transpose(0, 1), q.float(), q[:5], q[..., :64]):
        with pytest.raises(AssertionError):
            bi.bi_attention_kv4(bad, c, b, 1.0, torch.zeros_like(q), torch.zeros(1), stream=0)
    k = torch.zeros((6, 4, 128), dtype=torch.bfloat16)
    rope = torch.zeros((10, 64, 2))
    for qq, kk, vv in ((q, k[:, :3], k[:, :3]), (q, k[:5], k), (q, k, k.float())):
        with pytest.raises(AssertionError):
            bi.bi_rope_append_kv4(qq, kk, vv, rope, 128, 0, torch.zeros_like(q), c, b, stream=0)
    with pytest.raises(AssertionError):
        bi.bi_kv4_gather(c, b, k, k[:, :2], stream=0)


def test_ctypes_structs_match_the_header(bi):
    assert ctypes.sizeof(bi.bi_kv4_cache) == 32
    assert ctypes.sizeof(bi.bi_kv4_batch) == 48
    assert ctypes.sizeof(bi.bi_logits_rules) == 96
