"""What the bindings of the e4m3 linears and the mixture of experts refuse before they call the library, on the CPU and
with a stand-in for the library: nothing is launched, whatever the machine."""
import pytest
import torch


@pytest.fixture(scope="module")
def bi():
    import __graft_entry__
    __graft_entry__.build()
    import invariant_quantized_linear_gb300 as m
    return m


class Library:
    """In place of the library: every call succeeds, and is noted."""

    def __init__(self):
        self.names = []

    def bi_status_string(self, status):
        return b"status"

    def __getattr__(self, name):
        return lambda *args: self.names.append(name) or 0


class On(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    at = 0

    def get_device(self):
        return self.at


class OnOther(On):
    at = 1


M, K, N, E, TOP = 3, 272, 200, 4, 2


def tensors(bi):
    """The tensors of each call, by their names in it."""
    half, ints, codes = dict(dtype=torch.bfloat16), dict(dtype=torch.int32), dict(dtype=torch.uint8)
    z, ws = torch.zeros, torch.zeros(4096, dtype=torch.uint8)
    return dict(
        bi_quantize_act_f8=dict(x=z((M, K), **half), q=z((M, K), **codes), s_a=z(M, 3)),
        bi_gated_quantize_f8=dict(gu=z((M, 2 * K), **half), gate=bi.BI_GATE_SILU, q=z((M, K), **codes), s_a=z(M, 3)),
        bi_quantize_weight_f8=dict(w=z(N, K), w_q=z((N, K), **codes), s_w=z(2, 3)),
        bi_linear_f8=dict(q=z((M, K), **codes), s_a=z(M, 3), w=z((N, K), **codes), s_w=z(2, 3), y=z((M, N), **half), ws=ws),
        bi_linear_f8_grouped=dict(q=z((M, K), **codes), s_a=z(M, 3), src=z(6, **ints), offsets=z(E + 1, **ints),
                                  w=z((E, N, K), **codes), s_w=z(E, 2, 3), y=z((6, N), **half), ws=ws),
        bi_moe_route=dict(logits=z(M, E), score=0, renorm=True, scale=1.0, ids=z((M, TOP), **ints), weights=z(M, TOP),
                          offsets=z(E + 1, **ints), src=z(M * TOP, **ints), pos=z((M, TOP), **ints), ws=ws),
        bi_moe_combine=dict(rows=z((6, N), **half), pos=z((M, TOP), **ints), weights=z(M, TOP), base=z((M, N), **half),
                            y=z((M, N), **half)))


def on(kind, args):
    return {k: v.as_subclass(kind) if torch.is_tensor(v) else v for k, v in args.items()}


def call(bi, name, args):
    getattr(bi, name)(**args, stream=0)


NAMES = ["bi_quantize_act_f8", "bi_gated_quantize_f8", "bi_quantize_weight_f8", "bi_linear_f8", "bi_linear_f8_grouped",
         "bi_moe_route", "bi_moe_combine"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_off_the_gpu_reach_no_kernel(bi, monkeypatch, name):
    """Host tensors, all or one, and tensors on another GPU than the current one."""
    lib = Library()
    monkeypatch.setattr(bi, "lib", lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    args = tensors(bi)[name]
    bad = [args, on(OnOther, args)]
    for k, v in args.items():
        if torch.is_tensor(v):
            bad += [{**on(On, args), k: v}, {**on(On, args), k: v.as_subclass(OnOther)}]
    for b in bad:
        with pytest.raises(bi.BiError) as e:
            call(bi, name, b)
        assert e.value.status == bi.BI_ERR_INVALID_ARG
    assert not lib.names
    call(bi, name, on(On, args))
    assert lib.names == [name]


# other types of the same size, which would be read as if they were the right one
WRONG = {torch.bfloat16: (torch.float16, torch.int16), torch.float32: (torch.int32,), torch.int32: (torch.float32,),
         torch.uint8: (torch.int8, torch.float8_e5m2, torch.bool)}


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_other_types_reach_no_kernel(bi, monkeypatch, name):
    lib = Library()
    monkeypatch.setattr(bi, "lib", lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    args = on(On, tensors(bi)[name])
    for k, v in args.items():
        if not torch.is_tensor(v) or k == "ws":
            continue
        for dtype in WRONG[v.dtype]:
            with pytest.raises(AssertionError):
                call(bi, name, {**args, k: torch.zeros(v.shape, dtype=dtype).as_subclass(On)})
    assert not lib.names
    for k, v in args.items():                        # codes are taken as such too, and logits as bf16
        if torch.is_tensor(v) and v.dtype == torch.uint8 and k != "ws":
            args[k] = v.view(torch.float8_e4m3fn)
    if name == "bi_moe_route":
        args["logits"] = args["logits"].bfloat16()
    call(bi, name, args)
    assert lib.names == [name]


@pytest.mark.parametrize("gate", [None, 0, 1])
def test_quantisers_count_their_blocks_in_32_bits(bi, gate):
    """2^31 blocks are more than any memory holds, and refused; one row less gets past the limit, to an unaligned pointer."""
    def quantise(M):
        K, at = 1 << 20, (1 << 44) + 8
        if gate is None:
            return bi.lib.bi_quantize_act_f8(at, K, M, K, 1 << 50, 1 << 52, 0, None)
        return bi.lib.bi_gated_quantize_f8(at, 2 * K, M, K, gate, 1 << 50, 1 << 52, 0, None)
    assert quantise(1 << 18) == bi.BI_ERR_INVALID_ARG
    assert quantise((1 << 18) - 1) == bi.BI_ERR_ALIGNMENT
