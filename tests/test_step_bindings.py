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
