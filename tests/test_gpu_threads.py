"""The first call that a host thread makes: nothing has made the device current in it before."""
import threading

import pytest
import torch

from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bi():
    import invariant_quantized_linear_gb300 as m
    return m


def same_in_a_thread(call, y):
    """y after `call` in a thread of its own, on a stream that was made before, is y after it here."""
    call(None)
    want, stream, errors = y.clone(), torch.cuda.Stream(), []
    y.zero_()
    torch.cuda.synchronize()

    def first():
        try:
            call(stream)
        except Exception as e:
            errors.append(str(e))
    t = threading.Thread(target=first)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("grouped", [False, True])
def test_e4m3_linear(bi, grouped):
    g = torch.Generator().manual_seed(1)
    q, w = (torch.randint(0, 120, s, generator=g, dtype=torch.uint8).to(DEV) for s in ((5, 144), (1, 40, 144)))
    s_a, s_w = torch.ones((5, 2), device=DEV), torch.ones((1, 1, 2), device=DEV)
    y, ws = torch.empty((5, 40), dtype=torch.bfloat16, device=DEV), bi.new_f8_workspace()
    offsets = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    if grouped:
        same_in_a_thread(lambda s: bi.bi_linear_f8_grouped(q, s_a, None, offsets, w, s_w, y, ws, stream=s), y)
    else:
        same_in_a_thread(lambda s: bi.bi_linear_f8(q, s_a, w[0], s_w[0], y, ws, stream=s), y)


@pytest.mark.parametrize("M", [1, 40, 600])
def test_w8a8_linear(bi, M):
    g = torch.Generator().manual_seed(2)
    q, w = (torch.randint(-127, 128, s, generator=g, dtype=torch.int8).to(DEV) for s in ((M, 256), (128, 256)))
    s_a, s_w = torch.ones(M, device=DEV), torch.ones(128, device=DEV)
    y = torch.empty((M, 128), dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(bi.bi_linear_workspace_size(M, 128, 256), dtype=torch.uint8, device=DEV)
    same_in_a_thread(lambda s: bi.bi_linear_w8a8(q, s_a, w, s_w, y, ws, stream=s), y)


@pytest.mark.parametrize("M", [3, 16])
def test_program(bi, M):
    """Built and run in the thread."""
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, 256), generator=g).bfloat16().to(DEV)
    w, s_w = torch.randint(-127, 128, (128, 256), generator=g, dtype=torch.int8).to(DEV), torch.ones(128, device=DEV)
    q, s = torch.empty((M, 256), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    y = torch.empty((M, 128), dtype=torch.bfloat16, device=DEV)
    ops = [bi.op_quantize_act(x, q, s), bi.op_linear(q, s, w, s_w, y)]
    prog, ws = bi.new_program(len(ops)), torch.zeros(bi.bi_program_workspace_size(), dtype=torch.uint8, device=DEV)

    def call(stream):
        bi.bi_program_build(ops, prog)
        bi.bi_program_run(prog, M, ws, stream=stream)
    same_in_a_thread(call, y)
