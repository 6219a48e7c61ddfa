"""Launches of the e4m3 linears and the routing whose shared memory differs from call to call: right after any earlier
call, and with several host threads at once."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def check_top1(M, E):
    """Routing of M tokens to one of E experts each, against torch."""
    import invariant_quantized_linear_gb300 as bi
    x = torch.rand((M, E), device=DEV)
    x.scatter_(1, torch.randint(0, E, (M, 1), device=DEV), 2.0)
    want = x.argmax(1).int()
    ids, offsets, src, pos = (torch.empty(s, dtype=torch.int32, device=DEV) for s in ((M, 1), (E + 1,), (M,), (M, 1)))
    bi.bi_moe_route(x, bi.BI_ROUTE_SOFTMAX, True, 1.0, ids, torch.empty((M, 1), device=DEV), offsets, src, pos,
                    bi.new_moe_route_workspace(M, E))
    assert torch.equal(ids[:, 0], want)
    assert torch.equal(src.long(), torch.sort(want, stable=True).indices)
    assert torch.equal(offsets[1:].long(), torch.bincount(want, minlength=E).cumsum(0))
    assert torch.equal(src[pos[:, 0].long()].long(), torch.arange(M, device=DEV))


# 12 bytes an expert and 4 more for each 32 tokens of a chunk: from just below 48 KB to just above it
@pytest.mark.parametrize("M, E", [(40000, 1024), (43776, 1024), (60000, 768), (38912, 1024), (43777, 1024), (45000, 943)])
def test_route_in_a_fresh_process(M, E):
    """No earlier call has raised what the kernels may use."""
    code = "from tests.test_gpu_f8_launch import check_top1; check_top1(%d, %d)" % (M, E)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("threads", [2, 4])
def test_threads_with_few_and_many_experts(threads):
    """Host threads on streams of their own, whose calls differ in their number of experts, so in their shared memory.  The
    library is called without the binding, which would hold the threads apart."""
    import invariant_quantized_linear_gb300 as bi
    ws, refused, turns = bi.new_f8_workspace(), [], 16000 // threads
    g = torch.Generator().manual_seed(3)

    def setup(E):
        q, w = (torch.randint(0, 120, s, generator=g, dtype=torch.uint8).to(DEV) for s in ((4, 16), (E, 32, 16)))
        s_a, s_w = torch.ones((4, 1), device=DEV), torch.ones((E, 1, 1), device=DEV)
        offsets = torch.full((E + 1,), 4, dtype=torch.int32, device=DEV)
        offsets[:E] = 0
        return q, s_a, offsets, w, s_w, torch.empty((4, 32), dtype=torch.bfloat16, device=DEV), torch.cuda.Stream()

    def work(q, s_a, offsets, w, s_w, y, stream):
        args = (q.data_ptr(), s_a.data_ptr(), 4, 16, None, 4, offsets.data_ptr(), w.shape[0], w.data_ptr(), s_w.data_ptr(), 32,
                y.data_ptr(), ws.data_ptr(), ws.nbytes, 0, stream.cuda_stream)
        for i in range(turns):
            if bi.lib.bi_linear_f8_grouped(*args) != bi.BI_OK:
                refused.append((w.shape[0], i))
            if i % 20 == 19:
                stream.synchronize()                 # no full queue behind which the threads would wait for one another
    calls = [setup(E) for E in (1024, 1, 700, 3)[:threads]]
    wants = []
    for q, s_a, offsets, w, s_w, y, _ in calls:
        bi.bi_linear_f8_grouped(q, s_a, None, offsets, w, s_w, y, ws)
        wants.append(y.clone())
        y.zero_()
    torch.cuda.synchronize()
    running = [threading.Thread(target=work, args=c) for c in calls]
    for t in running:
        t.start()
    for t in running:
        t.join()
    torch.cuda.synchronize()
    assert not refused, (len(refused), refused[:4])
    for c, want in zip(calls, wants):
        assert torch.equal(c[5].view(torch.int16), want.view(torch.int16))
    assert bi.bi_workspace_status(ws) == bi.BI_OK
