"""Launches of the routing whose shared memory differs from call to call."""
import os
import subprocess
import sys

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
