"""What the Python bindings of the decoder-step operators check and hold, on the CPU: nothing is launched."""
import gc
import weakref

import pytest
import torch


@pytest.fixture(scope="module")
def bi():
    import __graft_entry__
    __graft_entry__.build()
    import invariant_quantized_linear_gb300 as m
    return m


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_structures_hold_their_tensors(bi):
    """Cache, batch and rules are addresses: the tensors behind them live as long as they do."""
    def lives(make, *tensors):
        return [weakref.ref(t) for t in tensors], make(*tensors)
    for make in (lambda: lives(lambda p: bi.kv4_cache(p, 16, 64),
                               torch.zeros((2, 1, bi.bi_kv4_block_bytes(16, 64)), dtype=torch.uint8)),
                 lambda: lives(lambda c, n, p: bi.kv4_batch(c, n, p, 3, 3, 40), ints(3), ints(2), ints(2, 4)),
                 lambda: lives(lambda i, b, m, e, k: bi.logits_rules(ids=i, begin=b, mid=m, end=e, mask=k), ints(9), ints(2),
                               ints(2), ints(2), ints(2, 32)),
                 lambda: lives(lambda r, p, f, i, b: bi.logits_rules(repetition=r, presence=p, frequency=f, bias_ids=i, bias=b),
                               torch.ones(2), torch.ones(2), torch.ones(2), ints(2, 5), torch.ones(2, 5))):
        refs, s = make()
        gc.collect()
        assert all(r() is not None for r in refs)
        del s
        gc.collect()
        assert all(r() is None for r in refs)


def test_append_checks_the_table_and_the_norms(bi):
    """A table narrower than rot / 2 or of another type, and norms of another length, are not read past their end."""
    T, Hq, Hkv, D = 6, 4, 2, 64
    pool = torch.zeros((2, Hkv, bi.bi_kv4_block_bytes(16, D)), dtype=torch.uint8)
    cache, batch = bi.kv4_cache(pool, 16, D), bi.kv4_batch(ints(3), ints(2), ints(2, 4), T, 3, 40)
    half = dict(dtype=torch.bfloat16)
    q, k, v, out = (torch.zeros((T, h, D), **half) for h in (Hq, Hkv, Hkv, Hq))
    norm = torch.ones(D, **half)

    def call(rope=torch.zeros((40, 16, 2)), rot=32, q_norm=norm, k_norm=norm, q_out=out):
        bi.bi_rope_append_kv4(q, k, v, rope, rot, bi.BI_ROPE_HALF, q_out, cache, batch, q_norm=q_norm, k_norm=k_norm, stream=0)
    for bad in (dict(rope=torch.zeros((40, 15, 2))), dict(rope=torch.zeros((40, 32, 2))), dict(rope=torch.zeros((40, 16, 1))),
                dict(rope=torch.zeros((40, 32))), dict(rope=torch.zeros((40, 16, 2), dtype=torch.float64)),
                dict(rope=torch.zeros((40, 2, 16)).transpose(1, 2)), dict(rope=torch.zeros((40, 16, 2)).bfloat16()),
                dict(q_norm=norm[:32]), dict(k_norm=norm[:63]), dict(q_norm=norm.float()), dict(k_norm=torch.ones(2 * D, **half)[::2]),
                dict(q_out=out[:5])):
        with pytest.raises(AssertionError):
            call(**bad)
    # the shapes that are right reach the library, which finds no device (or unaligned memory) here
    with pytest.raises(bi.BiError):
        call(rot=36, rope=torch.zeros((40, 18, 2)))            # half layout: a multiple of 8


def test_norm_checks_shapes_and_types(bi):
    M, K = 3, 64
    half = dict(dtype=torch.bfloat16)
    good = dict(h=torch.zeros((M, K), **half), y=torch.zeros((M, K), **half), w=torch.zeros(K, **half), eps=1e-6,
                h_out=torch.zeros((M, K), **half), q=torch.zeros((M, K), dtype=torch.int8), s_a=torch.zeros(M))

    def call(**o):
        a = {**good, **o}
        bi.bi_rmsnorm_quantize(a["h"], a["y"], a["w"], a["eps"], a["h_out"], a["q"], a["s_a"], stream=0)
    wide = torch.zeros((M, 2 * K), **half)
    for bad in (dict(h=wide[:2]), dict(h=wide[:, :K - 8]), dict(h=wide[:, ::2]), dict(h=torch.zeros((M, K))), dict(h=wide[0]),
                dict(y=wide[:2]), dict(y=wide[:, :K - 1]), dict(y=torch.zeros((M, K))), dict(w=wide[0, :K - 1]),
                dict(w=torch.zeros(K)), dict(w=wide[0, ::2]), dict(h_out=wide[:2]), dict(h_out=wide[:, :8]),
                dict(h_out=torch.zeros((M, K))), dict(q=torch.zeros((M, 2 * K), dtype=torch.int8)[:, :K]),
                dict(q=torch.zeros((M, K), dtype=torch.int16)), dict(s_a=torch.zeros(M - 1)),
                dict(s_a=torch.zeros(M, dtype=torch.float64)), dict(s_a=torch.zeros(2 * M)[::2])):
        with pytest.raises(AssertionError):
            call(**bad)
    for refused in (dict(y=None), dict(h_out=None), dict(eps=-1.0)):
        with pytest.raises(bi.BiError):
            call(**refused)


def test_logits_checks_rows_and_results(bi):
    M, V = 3, 100
    x, out, ws = torch.zeros((M, V), dtype=torch.bfloat16), torch.zeros((M, V)), torch.zeros(1, dtype=torch.uint8)

    def call(rules, out=out, argmax=ints(M)):
        bi.bi_logits_process(x, rules, out, argmax, ws, stream=0)
    none = bi.logits_rules()
    ids = dict(ids=ints(9), begin=ints(M), mid=ints(M), end=ints(M))
    for bad in (bi.logits_rules(**{**ids, "begin": ints(M - 1)}), bi.logits_rules(**{**ids, "end": ints(1)}),
                bi.logits_rules(**ids, repetition=torch.ones(M - 1)), bi.logits_rules(presence=torch.ones(1)),
                bi.logits_rules(frequency=torch.ones(2)), bi.logits_rules(bias_ids=ints(2, 4), bias=torch.ones(2, 4)),
                bi.logits_rules(mask=ints(M - 1, 4)), bi.logits_rules(mask=ints(M, 3)), bi.logits_rules(mask=ints(M, 9)[:, :3])):
        with pytest.raises(AssertionError):
            call(bad)
    with pytest.raises(AssertionError):
        bi.logits_rules(bias_ids=ints(M, 4), bias=torch.ones(M, 3))
    for o in (out[:2], out[:, :99], torch.zeros((M, V), dtype=torch.bfloat16), out.double(), out.t().contiguous().t()):
        with pytest.raises(AssertionError):
            call(none, out=o)
    for a in (ints(M - 1), ints(2 * M)[::2], ints(M).long(), torch.zeros(M)):
        with pytest.raises(AssertionError):
            call(none, argmax=a)
    with pytest.raises(bi.BiError):                             # more rows than the logits will do; the workspace will not
        call(bi.logits_rules(**{k: v if k == "ids" else ints(M + 2) for k, v in ids.items()}, mask=ints(M + 1, 4)))


def test_rope_table_checks_its_frequencies(bi):
    """Frequencies that are not side by side are not read as if they were."""
    f, rope = torch.ones(16, dtype=torch.float64), torch.zeros((5, 8, 2))
    for bad in (dict(inv_freq=f[::2]), dict(inv_freq=f[:8].float()), dict(inv_freq=f[:7]), dict(rope=torch.zeros((5, 9, 2))),
                dict(rope=rope.double()), dict(rope=torch.zeros((5, 2, 8)).transpose(1, 2))):
        a = {**dict(inv_freq=f[:8], rope=rope), **bad}
        with pytest.raises(AssertionError):
            bi.bi_rope_table(a["inv_freq"], a["rope"], stream=0)
    with pytest.raises(bi.BiError):
        bi.bi_rope_table(f[:8], rope, float("nan"), stream=0)
