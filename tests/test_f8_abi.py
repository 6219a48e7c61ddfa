"""Host-side checks of the e4m3 linears and the mixture of experts: sizes, the refusals of every argument rule before
anything is launched (fake pointers that are never dereferenced), and what the bindings check."""
import pytest
import torch

FAKE = 1 << 32          # 16-byte aligned, never dereferenced
FAR = 1 << 40           # overlaps no small buffer at FAKE


@pytest.fixture(scope="module")
def bi():
    import __graft_entry__
    __graft_entry__.build()
    import invariant_quantized_linear_gb300 as m
    return m


def refused(call, rules, status):
    for o in rules:
        assert call(**o) == status, o


def quantize(bi, gate=None):
    def call(**o):
        a = dict(x=FAKE, ldx=2048, M=4, K=1024, gate=gate, q=2 * FAR, s=3 * FAR)
        a.update(o)
        if gate is None:
            return bi.lib.bi_quantize_act_f8(a["x"], a["ldx"], a["M"], a["K"], a["q"], a["s"], 0, None)
        return bi.lib.bi_gated_quantize_f8(a["x"], a["ldx"], a["M"], a["K"], a["gate"], a["q"], a["s"], 0, None)
    return call


@pytest.mark.parametrize("gate", [None, 0, 1])
def test_quantize_refusals(bi, gate):
    call = quantize(bi, gate)
    refused(call, [{"x": None}, {"q": None}, {"s": None}, {"M": 0}, {"M": (1 << 20) + 1}, {"K": 0}, {"K": 1000}, {"K": -16},
                   {"K": (1 << 20) + 16}, {"ldx": 1016}, {"q": FAKE}, {"q": FAKE + 3 * 4096 + 2032}, {"s": FAKE + 16},
                   {"s": 2 * FAR + 4092}, {"q": 3 * FAR + 112}], bi.BI_ERR_INVALID_ARG)
    refused(call, [{"x": FAKE + 8}, {"q": 2 * FAR + 4}, {"s": 3 * FAR + 2}, {"ldx": 2052}], bi.BI_ERR_ALIGNMENT)
    if gate is not None:
        refused(call, [{"gate": 2}, {"gate": -1}, {"ldx": 2040}], bi.BI_ERR_INVALID_ARG)


def test_quantize_weight_refusals(bi):
    def call(**o):
        a = dict(w=FAKE, ldw=1024, N=300, K=1024, q=2 * FAR, s=3 * FAR)
        a.update(o)
        return bi.lib.bi_quantize_weight_f8(a["w"], a["ldw"], a["N"], a["K"], a["q"], a["s"], None)
    refused(call, [{"w": None}, {"q": None}, {"s": None}, {"N": 0}, {"N": (1 << 24) + 1}, {"K": 8}, {"ldw": 1020}, {"q": FAKE},
                   {"s": FAKE + 4}, {"s": 2 * FAR}], bi.BI_ERR_INVALID_ARG)
    refused(call, [{"w": FAKE + 4}, {"q": 2 * FAR + 8}, {"s": 3 * FAR + 1}, {"ldw": 1026}], bi.BI_ERR_ALIGNMENT)


def linear(bi):
    n = bi.bi_f8_workspace_size()

    def call(**o):
        a = dict(q=FAKE, s=FAR, M=6, K=1024, w=2 * FAR, sw=3 * FAR, N=300, y=4 * FAR, ws=5 * FAR, n=n)
        a.update(o)
        return bi.lib.bi_linear_f8(a["q"], a["s"], a["M"], a["K"], a["w"], a["sw"], a["N"], a["y"], a["ws"], a["n"], 0, None)
    return call


def test_linear_refusals(bi):
    call, n = linear(bi), bi.bi_f8_workspace_size()
    refused(call, [{"q": None}, {"s": None}, {"w": None}, {"sw": None}, {"y": None}, {"M": 0}, {"M": (1 << 20) + 1}, {"K": 0}, {"K": 1032},
                   {"N": 0}, {"N": (1 << 24) + 1}, {"y": FAKE}, {"y": FAR + 188}, {"y": 2 * FAR + 16}, {"y": 3 * FAR},
                   {"y": 5 * FAR + 64}, {"ws": FAKE}, {"ws": 2 * FAR - n + 16}], bi.BI_ERR_INVALID_ARG)
    refused(call, [{"q": FAKE + 8}, {"w": 2 * FAR + 8}, {"s": FAR + 2}, {"sw": 3 * FAR + 1}, {"y": 4 * FAR + 1}], bi.BI_ERR_ALIGNMENT)
    refused(call, [{"ws": None}, {"n": n - 1}, {"ws": 5 * FAR + 8}], bi.BI_ERR_WORKSPACE)


def test_grouped_refusals(bi):
    n = bi.bi_f8_workspace_size()

    def call(**o):
        a = dict(q=FAKE, s=FAR, rows=6, K=1024, src=6 * FAR, R=12, off=7 * FAR, E=4, w=2 * FAR, sw=3 * FAR, N=300, y=4 * FAR, ws=5 * FAR,
                 n=n)
        a.update(o)
        return bi.lib.bi_linear_f8_grouped(a["q"], a["s"], a["rows"], a["K"], a["src"], a["R"], a["off"], a["E"], a["w"], a["sw"], a["N"],
                                           a["y"], a["ws"], a["n"], 0, None)
    refused(call, [{"q": None}, {"off": None}, {"rows": 0}, {"R": 0}, {"R": (1 << 20) + 1}, {"E": 0}, {"E": 1025}, {"src": None},
                   {"E": 1024, "N": 1 << 22}, {"y": 6 * FAR + 44}, {"y": 7 * FAR + 16}, {"ws": 7 * FAR}, {"ws": 6 * FAR},
                   {"y": 2 * FAR + 3 * 300 * 1024}], bi.BI_ERR_INVALID_ARG)
    refused(call, [{"src": 6 * FAR + 2}, {"off": 7 * FAR + 1}], bi.BI_ERR_ALIGNMENT)
    refused(call, [{"ws": None}, {"n": 0}], bi.BI_ERR_WORKSPACE)


def test_route_sizes_and_refusals(bi):
    assert bi.bi_moe_route_workspace_size(1, 1) > 0
    for M, E in ((0, 4), (65536, 4), (4, 0), (4, 1025)):
        assert bi.bi_moe_route_workspace_size(M, E) == 0
    for M, E in ((1, 1024), (8192, 128), (65535, 1024)):       # counts of each chunk of tokens
        assert bi.bi_moe_route_workspace_size(M, E) >= 4 * E
    n = bi.bi_moe_route_workspace_size(5, 40)

    def call(**o):
        a = dict(x=FAKE, ld=40, type=0, M=5, E=40, k=3, score=0, renorm=1, scale=1.0, ids=FAR, w=2 * FAR, off=3 * FAR, src=4 * FAR,
                 pos=5 * FAR, ws=6 * FAR, n=n)
        a.update(o)
        return bi.lib.bi_moe_route(a["x"], a["ld"], a["type"], a["M"], a["E"], a["k"], a["score"], a["renorm"], a["scale"], a["ids"],
                                   a["w"], a["off"], a["src"], a["pos"], a["ws"], a["n"], 0, None)
    refused(call, [{"x": None}, {"ids": None}, {"w": None}, {"off": None}, {"src": None}, {"pos": None}, {"M": 0}, {"M": 65536}, {"E": 0},
                   {"E": 1025, "ld": 1025}, {"k": 0}, {"k": 41}, {"E": 64, "ld": 64, "k": 33}, {"ld": 39}, {"type": 2}, {"score": 2},
                   {"score": -1}, {"scale": float("inf")}, {"scale": float("nan")}, {"ids": FAKE}, {"w": FAR + 56}, {"off": FAKE + 796},
                   {"src": 3 * FAR + 160}, {"pos": 4 * FAR}, {"ws": 5 * FAR}, {"ws": FAKE}], bi.BI_ERR_INVALID_ARG)
    refused(call, [{"x": FAKE + 2}, {"x": FAKE + 1, "type": 1}, {"ids": FAR + 2}, {"w": 2 * FAR + 1}, {"off": 3 * FAR + 2},
                   {"src": 4 * FAR + 3}, {"pos": 5 * FAR + 2}], bi.BI_ERR_ALIGNMENT)
    refused(call, [{"ws": None}, {"n": n - 1}, {"ws": 6 * FAR + 4}], bi.BI_ERR_WORKSPACE)


def test_combine_refusals(bi):
    def call(**o):
        a = dict(rows=FAKE, R=10, pos=FAR, w=2 * FAR, M=5, k=2, N=64, base=3 * FAR, y=4 * FAR)
        a.update(o)
        return bi.lib.bi_moe_combine(a["rows"], a["R"], a["pos"], a["w"], a["M"], a["k"], a["N"], a["base"], a["y"], 0, None)
    refused(call, [{"rows": None}, {"pos": None}, {"w": None}, {"y": None}, {"R": 0}, {"R": (1 << 21) + 1}, {"M": 0}, {"M": 65536}, {"k": 0},
                   {"k": 33}, {"N": 0}, {"N": (1 << 24) + 1}, {"y": FAKE + 1278}, {"y": FAR}, {"y": 2 * FAR + 36}, {"y": 3 * FAR + 2}],
            bi.BI_ERR_INVALID_ARG)
    refused(call, [{"rows": FAKE + 1}, {"pos": FAR + 2}, {"w": 2 * FAR + 2}, {"base": 3 * FAR + 1}, {"y": 4 * FAR + 1}],
            bi.BI_ERR_ALIGNMENT)


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_bindings_check_shapes(bi):
    """What the C entry points cannot see; a call that passes reaches the library, which finds no device here."""
    half = dict(dtype=torch.bfloat16)
    ws = torch.zeros(bi.bi_f8_workspace_size(), dtype=torch.uint8)

    def quant(x=torch.zeros((3, 272), **half), q=codes(3, 272), s=torch.zeros(3, 3)):
        bi.bi_quantize_act_f8(x, q, s, stream=0)

    def gated(x=torch.zeros((3, 544), **half), q=codes(3, 272), s=torch.zeros(3, 3)):
        bi.bi_gated_quantize_f8(x, bi.BI_GATE_SILU, q, s, stream=0)

    def weight(w=torch.zeros(200, 272), q=codes(200, 272), s=torch.zeros(2, 3)):
        bi.bi_quantize_weight_f8(w, q, s, stream=0)

    def lin(q=codes(3, 272), s=torch.zeros(3, 3), w=codes(200, 272), sw=torch.zeros(2, 3), y=torch.zeros((3, 200), **half)):
        bi.bi_linear_f8(q, s, w, sw, y, ws, stream=0)

    def group(q=codes(3, 272), s=torch.zeros(3, 3), src=ints(6), off=ints(5), w=codes(4, 200, 272), sw=torch.zeros(4, 2, 3),
              y=torch.zeros((6, 200), **half)):
        bi.bi_linear_f8_grouped(q, s, src, off, w, sw, y, ws, stream=0)

    def route(x=torch.zeros(3, 8), ids=ints(3, 2), w=torch.zeros(3, 2), off=ints(9), src=ints(6), pos=ints(3, 2)):
        bi.bi_moe_route(x, bi.BI_ROUTE_SOFTMAX, True, 1.0, ids, w, off, src, pos, ws, stream=0)

    def combine(rows=torch.zeros((6, 64), **half), pos=ints(3, 2), w=torch.zeros(3, 2), base=None, y=torch.zeros((3, 64), **half)):
        bi.bi_moe_combine(rows, pos, w, base, y, stream=0)
    for call, bad in ((quant, [dict(x=torch.zeros((2, 272), **half)), dict(x=torch.zeros((3, 256), **half)), dict(s=torch.zeros(3, 2)),
                               dict(x=torch.zeros(3, 272)), dict(q=codes(272, 3).t()), dict(s=torch.zeros(3, 3).double())]),
                      (gated, [dict(x=torch.zeros((3, 528), **half)), dict(s=torch.zeros(2, 3))]),
                      (weight, [dict(w=torch.zeros((200, 272), **half)), dict(s=torch.zeros(2, 2)), dict(w=torch.zeros(199, 272))]),
                      (lin, [dict(s=torch.zeros(3, 2)), dict(w=codes(200, 256)), dict(sw=torch.zeros(1, 3)), dict(sw=torch.zeros(3, 2).t()),
                             dict(y=torch.zeros((3, 199), **half)), dict(y=torch.zeros(3, 200)), dict(y=torch.zeros((3, 400), **half)[:, ::2])]),
                      (group, [dict(src=ints(5)), dict(src=ints(6).long()), dict(off=ints(4)), dict(off=ints(5).float()),
                               dict(w=codes(4, 200, 256)), dict(sw=torch.zeros(4, 3, 2)), dict(y=torch.zeros((6, 201), **half))]),
                      (route, [dict(ids=ints(2, 2)), dict(w=torch.zeros(3, 3)), dict(w=torch.zeros(3, 2).int()), dict(off=ints(8)),
                               dict(src=ints(5)), dict(pos=ints(2, 3)), dict(x=torch.zeros(3, 8).half()), dict(x=torch.zeros(8, 3).t())]),
                      (combine, [dict(w=torch.zeros(2, 3)), dict(pos=ints(3, 2).long()), dict(base=torch.zeros((3, 65), **half)),
                                 dict(y=torch.zeros((3, 65), **half)), dict(rows=torch.zeros(6, 64))])):
        for o in bad:
            with pytest.raises((AssertionError, bi.BiError)) as e:
                call(**o)
            assert e.type is AssertionError, (call.__name__, {k: v.shape for k, v in o.items()})
        with pytest.raises(bi.BiError):
            call()
